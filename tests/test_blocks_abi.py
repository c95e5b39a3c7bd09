"""What the calls of rotary axes, norms around a block, block selection and attention over blocks refuse, before any
CUDA call, and the block of a row of lists (compiled for the host)."""
import ctypes
import os
import subprocess

import pytest

import nvfp4_activation_quantize_gb300 as h3q
from nvfp4_activation_quantize_gb300 import build as libbuild

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return h3q.library()


def refuses(f, names, good, cases):
    for kw, what in cases:
        a = list(good)
        for name, value in kw.items():
            a[names.index(name)] = value
        assert f(*a) == h3q.H3Q_ERR_INVALID_ARGUMENT, kw
        assert what in h3q.h3q_last_error(), (kw, h3q.h3q_last_error())


def test_block_rows_on_the_host(tmp_path):
    exe = str(tmp_path / "block_rows")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    os.path.join(HERE, "host", "block_rows.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout + out.stderr
    assert int(out.stdout) > 10000


def _doubles(*v):
    return (ctypes.c_double * len(v))(*v)


def _dims(*v):
    return (ctypes.c_int64 * len(v))(*v)


AXES = ["q", "ld_q", "k", "ld_k", "v", "ld_v", "bq", "bk", "bv", "wq", "wk", "positions", "axes", "dims", "theta", "scale",
        "sections", "interleaved", "norm", "rows", "heads", "kv_heads", "dim", "eps", "qo", "ko", "vo", "stream"]


def test_axes_refusals(lib):
    good = [0x1000000, 512, 0x1100000, 256, 0x1200000, 256, None, None, None, None, None, 0x1300000, 3, _dims(44, 42, 42),
            _doubles(1e4, 1e4, 1e4), _doubles(1, 1, 1), 0, 0, 1, 10, 4, 2, 128, 1e-6, 0x2000000, 0x2100000, 0x2200000, None]
    refuses(lib.h3q_qkv_epilogue_axes, AXES, good, (
        ({"rows": -1}, "rows"), ({"rows": 1 << 41}, "2^40"), ({"dim": 96}, "head_dim"), ({"heads": 0}, "heads"),
        ({"heads": 3}, "multiple of kv_heads"), ({"kv_heads": 0}, "kv_heads"), ({"heads": 1 << 18}, "2^24"),
        ({"axes": 0}, "axes"), ({"axes": 5}, "axes"), ({"dims": None}, "axis_dims"), ({"theta": None}, "axis_dims"),
        ({"scale": None}, "axis_dims"), ({"dims": _dims(44, 41, 43)}, "even"), ({"dims": _dims(0, 64, 64)}, "positive"),
        ({"dims": _dims(44, 42, 58)}, "at most head_dim"), ({"dims": _dims(44, 42, 44)}, "multiple of 16"),
        ({"dims": _dims(20, 20, 20)}, "multiple of 16"), ({"dims": _dims(-2, 66, 64)}, "positive"),
        ({"theta": _doubles(1e4, 0, 1)}, "theta"), ({"theta": _doubles(1e4, float("nan"), 1)}, "theta"),
        ({"scale": _doubles(1, float("inf"), 1)}, "scale"), ({"theta": _doubles(5e-324, 1, 1), "scale": _doubles(1e300, 1, 1)}, "not finite"),
        ({"sections": 2}, "0 or 1"), ({"interleaved": -1}, "0 or 1"), ({"norm": 3}, "0 or 1"),
        ({"norm": 0, "wq": 0x1400000}, "weights need"), ({"eps": -1.0}, "eps"), ({"eps": float("nan")}, "eps"),
        ({"q": None}, "q is NULL"), ({"k": 0x1100010}, "32-byte"), ({"ld_q": 500}, "ld of q"), ({"ld_v": 128}, "ld of v"),
        ({"bq": 0x1400008}, "bias_q"), ({"wk": 0x1400002}, "weight_k"), ({"positions": None}, "positions"),
        ({"positions": 0x1300002}, "positions"), ({"qo": None}, "16-byte"), ({"vo": 0x2200008}, "16-byte"),
        ({"ko": 0x1100000}, "overlap"), ({"ko": 0x2000000 + 1024}, "overlap"), ({"vo": 0x1300000}, "overlap")))
    assert lib.h3q_qkv_epilogue_axes(*[0 if n == "rows" else a for n, a in zip(AXES, good)]) == h3q.H3Q_OK


POST = ["h", "ld_h", "o", "ld_o", "bias", "post", "gate", "keep", "gamma", "table", "frames", "row_frame", "rpf", "eps", "rows",
        "cols", "gsf", "codes", "scales", "rstd", "stream"]


def test_postnorm_refusals(lib):
    good = [0x1000000, 256, 0x1100000, 256, None, 0x1200000, 0x1210000, 1.0, 0x1220000, 0x1230000, 2, None, 5, 1e-6, 10, 256,
            0x1240000, 0x2000000, 0x2100000, None, None]
    refuses(lib.h3q_postnorm_residual_adaln_nvfp4, POST, good, (
        ({"rows": -1}, "rows"), ({"cols": 100}, "multiple of 64"), ({"cols": 8256, "ld_h": 8256, "ld_o": 8256}, "8,192"),
        ({"eps": -1.0}, "eps"), ({"keep": float("inf")}, "residual_scale"), ({"keep": float("nan")}, "residual_scale"),
        ({"frames": 0}, "num_frames"), ({"h": None}, "h must"), ({"h": 0x1000010}, "32-byte"), ({"ld_h": 252}, "ld of h"),
        ({"ld_h": 260}, "multiple of 8"), ({"o": None}, "o is NULL"), ({"ld_o": 264}, "ld of o"), ({"bias": 0x1200002}, "bias"),
        ({"post": None}, "gamma_post"), ({"gamma": None}, "gamma"), ({"gate": 0x1210008}, "gate_table"),
        ({"table": 0x1230010}, "mod_table"), ({"codes": None}, "codes"), ({"scales": 0x2100008}, "16-byte"),
        ({"gsf": None}, "global_scale"), ({"row_frame": 0x1250001}, "row_frame"), ({"rpf": 0}, "rows_per_frame"),
        ({"rpf": 4}, "past the tables"), ({"rstd": 0x1260002}, "row_rstd"), ({"codes": 0x1100000}, "overlaps an input"),
        ({"o": 0x1000000}, "overlaps an input"), ({"scales": 0x2000000}, "overlap each other"),
        ({"rstd": 0x1000000}, "overlap")))
    if lib.h3q_postnorm_residual_adaln_nvfp4(*[0 if n == "rows" else a for n, a in zip(POST, good)]) != h3q.H3Q_OK:
        raise AssertionError(h3q.h3q_last_error())


SELECT = ["q", "ld_q", "k", "ld_k", "cu_q", "cu_k", "batch", "rows_q", "rows_k", "heads", "kv_heads", "dim", "bq", "bk", "top",
          "causal", "first", "blocks", "scores", "ws", "ws_bytes", "stream"]
SHARED = (({"dim": 96}, "head_dim"), ({"dim": 256}, "head_dim"), ({"kv_heads": 0}, "kv_heads"), ({"heads": 3}, "multiple of kv_heads"),
          ({"heads": 1 << 18}, "2^24"), ({"bq": 32}, "block_q"), ({"bq": 96}, "block_q"), ({"bk": 512}, "block_k"),
          ({"bk": 0}, "block_k"), ({"top": 0}, "top"), ({"top": 4097}, "top"), ({"rows_q": -1}, "rows_q"),
          ({"rows_q": 1 << 31}, "rows_q"), ({"rows_k": (1 << 25) + 1}, "rows_k"), ({"batch": -1}, "batch"),
          ({"batch": (1 << 24) + 1}, "batch"), ({"causal": 2}, "causal"), ({"q": None}, "q is NULL"), ({"ld_q": 96}, "ld of q"),
          ({"k": 0x1100010}, "32-byte"), ({"cu_q": None}, "cu_q"), ({"cu_k": 0x1210002}, "cu_q and cu_k"),
          ({"blocks": None}, "blocks"), ({"blocks": 0x2000002}, "blocks"))


def test_select_refusals(lib):
    good = [0x1000000, 512, 0x1100000, 256, 0x1200000, 0x1210000, 2, 300, 500, 4, 2, 128, 64, 64, 8, 1, 1, 0x2000000, None,
            0x3000000, 1 << 20, None]
    refuses(lib.h3q_select_blocks, SELECT, good, SHARED + (
        ({"rows_k": 16_001 * 64}, "16,000"), ({"first": -1}, "first"), ({"first": 9}, "first"),
        ({"top": 2, "first": 1}, "no room"), ({"bq": 256, "top": 5, "first": 1}, "no room"),
        ({"scores": 0x2100002}, "scores"), ({"ws": None}, "workspace"), ({"ws": 0x3000080}, "256-byte"),
        ({"ws_bytes": 1000}, "workspace_bytes"), ({"blocks": 0x1000000}, "overlaps an input"),
        ({"scores": 0x2000000}, "overlap each other"), ({"ws": 0x2000000}, "overlap"),
        ({"batch": 1 << 24, "kv_heads": 256, "heads": 256, "dim": 64, "ld_q": 1 << 14, "ld_k": 1 << 14}, "2^31 lists")))
    none = [0 if n in ("rows_q", "batch") else a for n, a in zip(SELECT, good)]
    assert lib.h3q_select_blocks(*none) == h3q.H3Q_OK


def test_workspace_bytes_of_the_binding(tmp_path):
    """The binding's formula is the header's."""
    src = tmp_path / "w.c"
    src.write_text('#include "h3q.h"\n#include <stdio.h>\nint main(void) { printf("%lld\\n", (long long)'
                   "h3q_select_blocks_workspace_bytes(1033, 90000, 7, 8, 128, 128, 64)); return 0; }\n")
    exe = str(tmp_path / "w")
    subprocess.run(["gcc", "-I", os.path.dirname(libbuild.HEADER), str(src), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    assert int(out) == h3q.select_blocks_workspace_bytes(1033, 90000, 7, 8, 128, 128, 64)


ATTEND = ["q", "ld_q", "k", "ld_k", "v", "ld_v", "cu_q", "cu_k", "batch", "rows_q", "rows_k", "heads", "kv_heads", "dim", "bq",
          "bk", "blocks", "top", "causal", "scale", "o", "lse", "stream"]


def test_attention_refusals(lib):
    good = [0x1000000, 512, 0x1100000, 256, 0x1180000, 256, 0x1200000, 0x1210000, 2, 300, 500, 4, 2, 128, 64, 64, 0x2000000, 8,
            1, 0.1, 0x3000000, None, None]
    refuses(lib.h3q_attention_blocks, ATTEND, good, SHARED + (
        ({"scale": 0.0}, "scale"), ({"scale": float("nan")}, "scale"), ({"v": None}, "v is NULL"), ({"ld_v": 250}, "ld of v"),
        ({"o": None}, "o must"), ({"o": 0x3000008}, "16-byte"), ({"lse": 0x4000002}, "lse"),
        ({"o": 0x1100000}, "overlaps an input"), ({"o": 0x2000000}, "overlaps an input"), ({"lse": 0x3000000}, "o and lse")))
    for name in ("rows_q", "batch"):
        assert lib.h3q_attention_blocks(*[0 if n == name else a for n, a in zip(ATTEND, good)]) == h3q.H3Q_OK


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    x = torch.zeros((4, 128), dtype=torch.bfloat16)
    with pytest.raises((ValueError, RuntimeError)):
        h3q.h3q_qkv_epilogue_axes(x, x, x, torch.zeros((4, 1), dtype=torch.int32), (128,), 1)
    with pytest.raises((ValueError, RuntimeError)):
        h3q.h3q_postnorm_residual_adaln_nvfp4(x.float(), x, x[0], x[0], torch.ones(1))
    y, cu = x.view(4, 1, 128), torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises((ValueError, RuntimeError)):
        h3q.h3q_select_blocks(y, y, cu, cu, 3)
    with pytest.raises((ValueError, RuntimeError)):
        h3q.h3q_attention_blocks(y, y, y, cu, cu, torch.zeros((1, 1, 1), dtype=torch.int32))
