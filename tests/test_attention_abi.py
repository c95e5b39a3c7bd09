"""The paged cache's and the attention calls' checks on the host: what they refuse, before any CUDA
call, and the place of a position in the cache (compiled for the host)."""
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


def caller(f, names, good):
    def call(**kw):
        a = list(good)
        for name, value in kw.items():
            a[names.index(name)] = value
        return f(*a)

    return call


def test_cache_rows_on_the_host(tmp_path):
    exe = str(tmp_path / "cache_rows")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    os.path.join(HERE, "host", "cache_rows.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout + out.stderr
    assert int(out.stdout) > 10000


WRITE = ["k", "ld_k", "v", "ld_v", "rows", "cu", "len", "table", "batch", "max_pages", "kg", "vg", "kc", "ks", "vc",
         "vs", "pages", "page", "heads", "dim", "stream"]
# 10 rows of 2 heads of 128 for 3 sequences; a cache of 16 pages of 16 rows
WRITE_GOOD = [0x1000000, 256, 0x1100000, 256, 10, 0x1200000, 0x1201000, 0x1202000, 3, 4, 0x1203000, 0x1203004,
              0x2000000, 0x2100000, 0x2200000, 0x2300000, 16, 16, 2, 128, None]


def test_write_refusals(lib):
    call = caller(lib.h3q_kv_cache_write_nvfp4, WRITE, WRITE_GOOD)
    assert call() in (0, 2)
    for kw, what in (({"dim": 96}, "head_dim"), ({"dim": 0}, "head_dim"), ({"heads": 0}, "kv_heads"),
                     ({"heads": 1 << 18}, "2^24"), ({"page": 8}, "page_size"), ({"page": 48}, "page_size"),
                     ({"page": 256}, "page_size"), ({"pages": 0}, "num_pages"), ({"pages": 1 << 31}, "num_pages"),
                     ({"rows": -1}, "rows"), ({"batch": -1}, "batch"), ({"max_pages": 0}, "max_pages"),
                     ({"max_pages": 1 << 40}, "2^40"), ({"cu": None}, "cu_rows"), ({"len": None}, "kv_len"),
                     ({"table": None}, "block_table"), ({"cu": 0x1200002}, "aligned"), ({"k": None}, "k is NULL"),
                     ({"v": 0x1100010}, "32-byte"), ({"ld_k": 255}, "ld of k"), ({"ld_v": 128}, "ld of v"),
                     ({"ks": None}, "16-byte"), ({"vc": 0x2200008}, "16-byte"), ({"kg": None}, "global_scale"),
                     ({"vg": 0x1203002}, "global_scale"), ({"kc": 0x1000100}, "overlaps"),
                     ({"vs": 0x1202004}, "16-byte"), ({"vs": 0x1202010}, "overlaps"),
                     ({"vc": 0x2000000 + 1024}, "overlap")):
        assert call(**kw) == h3q.H3Q_ERR_INVALID_ARGUMENT, kw
        assert what in h3q.h3q_last_error(), (kw, h3q.h3q_last_error())
    assert call(rows=0, k=None, v=None) == h3q.H3Q_OK
    assert call(batch=0, cu=None, len=None, table=None) == h3q.H3Q_OK


READ = ["kc", "ks", "vc", "vs", "pages", "page", "heads", "dim", "kg", "vg", "rows", "cu", "len", "table", "batch",
        "max_pages", "ko", "vo", "stream"]
READ_GOOD = [0x2000000, 0x2100000, 0x2200000, 0x2300000, 16, 16, 2, 128, 0x1203000, 0x1203004, 10, 0x1200000,
             0x1201000, 0x1202000, 3, 4, 0x1000000, 0x1100000, None]


def test_read_refusals(lib):
    call = caller(lib.h3q_kv_cache_read_nvfp4, READ, READ_GOOD)
    assert call() in (0, 2)
    for kw, what in (({"dim": 32}, "head_dim"), ({"page": 0}, "page_size"), ({"pages": -1}, "num_pages"),
                     ({"rows": -3}, "rows"), ({"table": 0x1202001}, "aligned"), ({"kc": None}, "16-byte"),
                     ({"ko": None}, "k_out"), ({"vo": 0x1100010}, "32-byte"), ({"vo": 0x1000000 + 5088}, "overlap"),
                     ({"ko": 0x2000000}, "overlaps"), ({"vg": None}, "global_scale")):
        assert call(**kw) == h3q.H3Q_ERR_INVALID_ARGUMENT, kw
        assert what in h3q.h3q_last_error(), (kw, h3q.h3q_last_error())
    assert call(rows=0, ko=None, vo=None) == h3q.H3Q_OK


def test_python_binding_refuses_host_tensors():
    import torch

    cache = h3q.kv_cache_nvfp4(4, 2, 16, 64, device="cpu")
    assert [tuple(t.shape) for t in cache] == [(4, 2, 16, 32), (4, 2, 16, 4)] * 2
    lists = torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros((1, 1), dtype=torch.int32)
    x = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    g = torch.ones(1)
    with pytest.raises(ValueError, match="CUDA tensor"):
        h3q.h3q_kv_cache_write_nvfp4(x, x, cache, *lists, g, g)
    with pytest.raises(ValueError, match="CUDA tensor"):
        h3q.h3q_kv_cache_read_nvfp4(cache, *lists, g, g, rows=1)


CACHED = ["q", "ld_q", "rows", "heads", "max_rows", "cu", "len", "table", "batch", "max_pages", "mask", "kc", "ks", "vc",
          "vs", "pages", "page", "kv_heads", "dim", "kg", "vg", "scale", "o", "lse", "ws", "wsb", "stream"]
CACHED_GOOD = [0x1000000, 1024, 10, 8, 4, 0x1200000, 0x1201000, 0x1202000, 3, 4, None, 0x2000000, 0x2100000, 0x2200000,
               0x2300000, 16, 16, 2, 128, 0x1203000, 0x1203004, 0.1, 0x3000000, None, 0x10000000,
               h3q.attention_cache_workspace_bytes(4, 8, 2, 128), None]


def test_cache_attention_refusals(lib):
    call = caller(lib.h3q_attention_cache_nvfp4, CACHED, CACHED_GOOD)
    assert call() in (0, 2)
    for kw, what in (({"dim": 96}, "head_dim"), ({"heads": 7}, "multiple of kv_heads"), ({"heads": 0}, "multiple"),
                     ({"heads": 1 << 18}, "2^24"), ({"max_rows": 0}, "max_rows"), ({"max_rows": 65}, "max_rows"),
                     ({"scale": 0.0}, "scale"), ({"scale": -1.0}, "scale"), ({"scale": float("nan")}, "scale"),
                     ({"scale": float("inf")}, "scale"), ({"rows": -1}, "rows"), ({"batch": -1}, "batch"),
                     ({"q": None}, "q is NULL"), ({"q": 0x1000010}, "32-byte"), ({"ld_q": 1000}, "ld of q"),
                     ({"ld_q": 512}, "ld of q"), ({"mask": 0x1300004}, "8-byte"), ({"o": 0x3000008}, "16-byte"),
                     ({"o": None}, "16-byte"), ({"lse": 0x3100002}, "4-byte"), ({"ws": None}, "256-byte"),
                     ({"ws": 0x10000080}, "256-byte"), ({"wsb": CACHED_GOOD[-2] - 1}, "workspace_bytes"),
                     ({"o": 0x1000000 + 2048}, "overlaps"), ({"lse": 0x3000000}, "overlap"),
                     ({"ws": 0x2fff000 // 256 * 256}, "overlap"), ({"page": 40}, "page_size"),
                     ({"table": None}, "block_table"), ({"kg": None}, "global_scale")):
        assert call(**kw) == h3q.H3Q_ERR_INVALID_ARGUMENT, kw
        assert what in h3q.h3q_last_error(), (kw, h3q.h3q_last_error())
    assert call(rows=0, q=None, o=None) == h3q.H3Q_OK
    assert call(batch=0, cu=None, len=None, table=None) == h3q.H3Q_OK


def test_workspace_bytes_of_header_and_binding_agree(tmp_path):
    src = tmp_path / "ws.c"
    src.write_text('#include <stdio.h>\n#include "h3q.h"\nint main(void){\n'
                   'int64_t a[][4]={{1,8,8,64},{1,32,8,128},{4,8,2,128},{9,8,2,128},{16,32,8,256},{64,64,1,64}};\n'
                   'for(int i=0;i<6;++i)printf("%lld\\n",(long long)h3q_attention_cache_workspace_bytes('
                   'a[i][0],a[i][1],a[i][2],a[i][3]));return 0;}\n')
    exe = str(tmp_path / "ws")
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(os.path.dirname(HERE), "include"), str(src), "-o", exe],
                   check=True)
    got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    want = [h3q.attention_cache_workspace_bytes(*a) for a in ((1, 8, 8, 64), (1, 32, 8, 128), (4, 8, 2, 128),
                                                             (9, 8, 2, 128), (16, 32, 8, 256), (64, 64, 1, 64))]
    assert got == want


VARLEN = ["q", "ld_q", "k", "ld_k", "v", "ld_v", "cu_q", "cu_k", "batch", "rows_q", "rows_k", "heads", "kv_heads", "dim",
          "causal", "scale", "o", "lse", "stream"]
VARLEN_GOOD = [0x1000000, 1024, 0x1100000, 256, 0x1200000, 256, 0x1300000, 0x1301000, 3, 10, 12, 8, 2, 128, 1, 0.1,
               0x2000000, None, None]


def test_varlen_refusals(lib):
    call = caller(lib.h3q_attention_varlen, VARLEN, VARLEN_GOOD)
    assert call() in (0, 2)
    for kw, what in (({"dim": 80}, "head_dim"), ({"heads": 3}, "multiple of kv_heads"), ({"kv_heads": 0}, "kv_heads"),
                     ({"heads": 1 << 18}, "2^24"), ({"rows_q": -1}, "rows_q"), ({"rows_k": 1 << 31}, "rows_k"),
                     ({"batch": -2}, "batch"), ({"causal": 2}, "causal"), ({"scale": 0.0}, "scale"),
                     ({"scale": float("inf")}, "scale"), ({"q": None}, "q is NULL"), ({"k": 0x1100010}, "32-byte"),
                     ({"v": None}, "v is NULL"), ({"ld_q": 1000}, "ld of q"), ({"ld_k": 264}, "ld of k"),
                     ({"cu_q": None}, "cu_q"), ({"cu_k": 0x1301002}, "4-byte"), ({"o": None}, "16-byte"),
                     ({"o": 0x2000008}, "16-byte"), ({"lse": 0x2100001}, "4-byte"), ({"o": 0x1000000}, "overlaps"),
                     ({"lse": 0x2000000 + 16}, "overlap"), ({"lse": 0x1300000}, "overlaps")):
        assert call(**kw) == h3q.H3Q_ERR_INVALID_ARGUMENT, kw
        assert what in h3q.h3q_last_error(), (kw, h3q.h3q_last_error())
    assert call(rows_q=0, q=None) == h3q.H3Q_OK
    assert call(batch=0, cu_q=None) == h3q.H3Q_OK
    assert call(rows_k=0, k=None, v=None) in (0, 2)
