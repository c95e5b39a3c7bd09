"""GPU: attention over blocks whose waits run out.  The kernel is compiled with limits that ordinary waits pass, so that
every role of a CTA gives up at one moment or another; the call then ends, the error flag tells, what was stored is right
or was there before, rows of no sequence are untouched, and the GPU's next calls are as ever."""
import ctypes
import os
import subprocess

import pytest
import torch

import block_cases as bc
import nvfp4_activation_quantize_gb300 as h3q
from nvfp4_activation_quantize_gb300 import build as libbuild

pytestmark = pytest.mark.gpu

SOURCE = "attention_blocks.cu"
LIMITS = [0, 3000]   # ns: at the first wait that is not met at once, and somewhere on the way


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


@pytest.fixture(scope="module")
def libraries(dev, tmp_path_factory):
    libbuild.build()
    out = tmp_path_factory.mktemp("short_waits")
    flags = [f for f in libbuild.NVCC_FLAGS if f not in ("-Xptxas", "-v", "-lineinfo")]
    libs = {}
    for limit in LIMITS:
        obj, path = str(out / f"blocks.{limit}.o"), str(out / f"libh3q_{limit}.so")
        subprocess.run([libbuild._nvcc(), *flags, f"-DH3Q_SHORT_WAITS={limit}", "-c",
                        os.path.join(libbuild.CSRC, SOURCE), "-o", obj], check=True, capture_output=True)
        objs = [obj] + [os.path.join(libbuild.BUILD_DIR, s.replace(".cu", ".o")) for s in libbuild.SOURCES if s != SOURCE]
        subprocess.run([libbuild._nvcc(), *libbuild.ARCH, "-shared", "-o", path, *objs], check=True, capture_output=True)
        lib = ctypes.CDLL(path)
        for name, args in h3q._SIGNATURES.items():
            getattr(lib, name).argtypes, getattr(lib, name).restype = args, ctypes.c_int
        lib.h3q_last_error.argtypes, lib.h3q_last_error.restype = [], ctypes.c_char_p
        libs[limit] = lib
    return libs


def _use(lib):
    h3q._lib, h3q._torch, h3q._native = lib, None, None
    h3q._load_torch()


CASES = [  # (queries, keys), query heads, key heads, dim, block_q, block_k, top, causal
    ([(900, 900), (300, 1500), (64, 64)], 8, 2, 128, 64, 64, 8, True),      # a list for both tiles
    ([(900, 900), (300, 1500), (64, 64)], 2, 2, 128, 128, 128, 6, False),   # a list for each
    ([(900, 900), (300, 1500)], 3, 3, 64, 256, 64, 20, True),
    ([(1, 900), (1, 300), (1, 64)], 8, 2, 64, 64, 64, 14, True),            # single tokens
    ([(n, n) for n in range(1, 200, 3)], 2, 2, 64, 128, 64, 2, True),       # many short units
]


@pytest.mark.parametrize("limit", LIMITS)
@pytest.mark.parametrize("case", range(len(CASES)))
def test_calls_that_give_up(dev, libraries, case, limit):
    seqs, heads, kv_heads, dim, block_q, block_k, top, causal = CASES[case]
    c = bc.sequences(dev, seqs, heads, kv_heads, dim, seed=case)
    lists = bc.random_lists(c, kv_heads, block_q, block_k, top, case)
    rows = int(c["cu_q"][-1])

    def call():
        out = torch.full(c["q"].shape, 5.0, dtype=torch.bfloat16, device=dev)
        lse = torch.full((heads, c["q"].shape[0]), 6.0, device=dev)
        h3q.h3q_attention_blocks(c["q"], c["k"], c["v"], c["cu_q"], c["cu_k"], lists, block_q=block_q, block_k=block_k,
                                 causal=causal, out=out, lse=lse)
        return out, lse

    regular = h3q.library()
    want = call()
    assert h3q.h3q_kernel_error_flag() == 0
    gave_up = 0
    try:
        _use(libraries[limit])
        for _ in range(6):
            out, lse = call()
            flag = h3q.h3q_kernel_error_flag()
            gave_up += flag
            assert bool((out[rows:] == 5.0).all()) and bool((lse[:, rows:] == 6.0).all()), "rows of no sequence"
            assert bool(((out == want[0]) | (out == 5.0)).all()) and bool(((lse == want[1]) | (lse == 6.0)).all())
            if flag == 0:
                assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    finally:
        _use(regular)
    if limit == 0:
        assert gave_up == 6
    again = call()
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
    assert h3q.h3q_kernel_error_flag() == 0
