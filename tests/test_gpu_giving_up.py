"""GPU: attention kernels whose waits run out.  They are compiled with limits that ordinary waits pass, so that every
role of a CTA gives up at one moment or another; the call then ends, the error flag tells, what was stored is right or
was there before, rows of no sequence are untouched, and the GPU's next calls are as ever."""
import ctypes
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import nvfp4_activation_quantize_gb300 as h3q
import test_gpu_attention_cache as cached
import test_gpu_attention_varlen as varlen
from nvfp4_activation_quantize_gb300 import build as libbuild

pytestmark = pytest.mark.gpu

SOURCES = ["attention.cu", "attention_cache.cu", "attention_cache_wide.cu"]
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
    nvcc = libbuild._nvcc()

    def compile_one(job):
        src, limit = job
        obj = str(out / f"{src}.{limit}.o")
        define = [] if limit is None else [f"-DH3Q_SHORT_WAITS={limit}"]
        subprocess.run([nvcc, *flags, *define, "-c", os.path.join(libbuild.CSRC, src), "-o", obj], check=True,
                       capture_output=True)
        return obj

    kept = {s: os.path.join(libbuild.BUILD_DIR, s.replace(".cu", ".o")) for s in libbuild.SOURCES if s not in SOURCES}
    jobs = [(s, limit) for limit in LIMITS for s in SOURCES] + [(s, None) for s, o in kept.items() if not os.path.exists(o)]
    with ThreadPoolExecutor(len(jobs)) as pool:
        built = dict(zip(jobs, pool.map(compile_one, jobs)))
    libs = {}
    for limit in LIMITS:
        path = str(out / f"libh3q_{limit}.so")
        objs = [built[s, limit] for s in SOURCES] + [built.get((s, None), o) for s, o in kept.items()]
        subprocess.run([nvcc, *libbuild.ARCH, "-shared", "-o", path, *objs], check=True, capture_output=True)
        lib = ctypes.CDLL(path)
        for name, args in h3q._SIGNATURES.items():
            getattr(lib, name).argtypes, getattr(lib, name).restype = args, ctypes.c_int
        lib.h3q_last_error.argtypes, lib.h3q_last_error.restype = [], ctypes.c_char_p
        libs[limit] = lib
    return libs


def _use(lib):
    h3q._lib, h3q._torch, h3q._native = lib, None, None
    h3q._load_torch()


LONG = 300000   # positions that keep the cache's copies behind the arithmetic
CASES = {   # the call, and whether nothing is joined after the kernel
    "prompt 64": (lambda d: _prompt(d, 64, True), True),
    "prompt 128": (lambda d: _prompt(d, 128, False), True),
    "prompt 256": (lambda d: _prompt(d, 256, True), True),
    "short prompts": (lambda d: _prompt(d, 128, True, [(n, n) for n in range(1, 200, 3)]), True),
    "1 token": (lambda d: _cache(d, 1, 128, LONG), False),
    "4 tokens": (lambda d: _cache(d, 4, 128, LONG), False),
    "6 tokens": (lambda d: _cache(d, 6, 128, LONG), False),
    "8 tokens": (lambda d: _cache(d, 8, 128, LONG), False),
    "8 tokens, head_dim 64": (lambda d: _cache(d, 8, 64, LONG), False),
    "4 tokens, head_dim 256": (lambda d: _cache(d, 4, 256, LONG), False),
    "12 tokens": (lambda d: _cache(d, 12, 128, 3000), False),
    "20 tokens": (lambda d: _cache(d, 20, 128, 3000), False),
    "20 tokens, head_dim 64": (lambda d: _cache(d, 20, 64, 3000), False),
    "12 tokens, one tile": (lambda d: _cache(d, 12, 128, 120), True),
    "20 tokens, one tile": (lambda d: _cache(d, 20, 64, 120), True),
    "1 token, one tile": (lambda d: _cache(d, 1, 128, 200), True),
}
MET = ("1 token, one tile",)   # the copies may have landed before the queries are there


def _prompt(dev, dim, causal, seqs=((900, 900), (300, 1500), (64, 64))):
    c = varlen._case(dev, list(seqs), 8, 2, dim, seed=50)
    return lambda: varlen._run(c, causal), int(c["cu_q"][-1])


def _cache(dev, new, dim, keys):
    c = cached._case(dev, [(new, keys), (new, keys // 2 + new), (1, keys // 3 + 1)], 8, 2, dim, 64, seed=51)
    c["table"] = c["table"][:, :-(-keys // 64)].contiguous()
    return lambda: cached._run(c), int(c["cu"][-1])


@pytest.mark.parametrize("limit", LIMITS)
@pytest.mark.parametrize("name", list(CASES))
def test_calls_that_give_up(dev, libraries, name, limit):
    make, whole = CASES[name]
    call, rows = make(dev)
    regular = h3q.library()
    want = [t.clone() for t in call()]
    assert h3q.h3q_kernel_error_flag() == 0
    gave_up = 0
    try:
        _use(libraries[limit])
        for _ in range(8):
            out, lse = call()
            flag = h3q.h3q_kernel_error_flag()
            gave_up += flag
            assert bool((out[rows:] == 5.0).all()) and bool((lse[:, rows:] == 6.0).all()), "rows of no sequence"
            if flag == 0:
                assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
            elif whole:
                assert bool(((out == want[0]) | (out == 5.0)).all()) and bool(((lse == want[1]) | (lse == 6.0)).all())
    finally:
        _use(regular)
    if limit == 0 and name not in MET:
        assert gave_up == 8
    for _ in range(2):
        again = call()
        assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
    assert h3q.h3q_kernel_error_flag() == 0
