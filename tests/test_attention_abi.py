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
