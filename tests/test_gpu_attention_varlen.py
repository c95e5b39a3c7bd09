"""GPU: softmax attention over packed sequences, against the formula in 64 bits: head sizes and groups (a row
tile holds tokens x heads), lengths around the tiles of rows and keys, more keys than queries and fewer, sequences
of nothing, strides, values that are no numbers where they are not seen and where they are, graphs and streams,
and the same bits every time."""
import numpy as np
import pytest
import torch

import cache_cases as cc
import nvfp4_activation_quantize_gb300 as h3q

pytestmark = pytest.mark.gpu

WEIGHT = 2.0 ** -8  # weights are rounded to bf16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


def _case(dev, seqs, heads, kv_heads, dim, seed=0, packed=False, tail=3):
    """Inputs for sequences of (queries, keys); the last `tail` rows belong to none."""
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def rows(n, h):
        x = torch.randn((n, (2 if packed else 1) * h * dim), generator=g, device=dev).bfloat16()
        return (x[:, h * dim:] if packed else x).unflatten(1, (h, dim))

    nq, nk = [a for a, _ in seqs], [b for _, b in seqs]
    return {"q": rows(sum(nq) + tail, heads), "k": rows(sum(nk) + tail, kv_heads), "v": rows(sum(nk) + tail, kv_heads),
            "cu_q": cc.ints(cc.offsets(nq).tolist(), dev), "cu_k": cc.ints(cc.offsets(nk).tolist(), dev)}


def _run(c, causal, **kw):
    rows, heads, dim = c["q"].shape
    out = torch.full((rows, heads, dim), 5.0, dtype=torch.bfloat16, device=c["q"].device)
    lse = torch.full((heads, rows), 6.0, dtype=torch.float32, device=c["q"].device)
    assert h3q.h3q_attention_varlen(c["q"], c["k"], c["v"], c["cu_q"], c["cu_k"], causal=causal, out=out, lse=lse,
                                    **kw) is out
    return out, lse


def _check(c, causal, out, lse, scale=None, what=""):
    cu_q, cu_k = c["cu_q"].tolist(), c["cu_k"].tolist()
    scale = c["q"].shape[2] ** -0.5 if scale is None else scale
    for b in range(len(cu_q) - 1):
        n, keys = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        if n == 0:
            continue
        seen = torch.ones((n, keys), dtype=torch.bool, device=out.device)
        if causal:
            seen = seen.tril(keys - n)
        ref = cc.attention64(c["q"][cu_q[b]:cu_q[b + 1]], c["k"][cu_k[b]:cu_k[b + 1]], c["v"][cu_k[b]:cu_k[b + 1]], seen,
                             scale)
        cc.check_attention(out[cu_q[b]:cu_q[b + 1]], lse[:, cu_q[b]:cu_q[b + 1]], ref, keys, WEIGHT,
                           f"{what} sequence {b}")
    assert bool((out[cu_q[-1]:] == 5.0).all()) and bool((lse[:, cu_q[-1]:] == 6.0).all()), f"{what}: rows of no sequence"


CASES = [  # (queries, keys) of the sequences, query heads, key heads, dim
    ([(1, 1)], 1, 1, 128),
    ([(128, 128)], 1, 1, 128),
    ([(256, 256)], 1, 1, 64),
    ([(37, 37)], 8, 2, 64),
    ([(n, n) for n in (1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300)], 2, 2, 128),
    ([(n, n) for n in (1, 31, 32, 33, 64, 65, 129, 200)], 4, 1, 128),
    ([(500, 500), (0, 70), (130, 0), (700, 700)], 8, 2, 128),
    ([(1, 300), (5, 1000), (200, 333), (128, 640), (64, 128)], 8, 2, 128),
    ([(300, 100), (129, 128), (500, 499)], 3, 3, 64),                # queries that see nothing
    ([(200, 200), (90, 1500)], 14, 2, 128),                          # 7 heads: 126 rows of a tile
    ([(77, 77), (150, 151)], 40, 8, 64),                             # 5 heads
    ([(33, 500)], 48, 1, 128),                                       # 48 heads a key head: 16 of them a tile
    ([(3, 200), (40, 41)], 128, 1, 64),
    ([(2, 70)], 131, 1, 64),                                         # a prime group: one head a tile
    ([(1, 1), (200, 200), (65, 320), (129, 129)], 4, 2, 256),
    ([(300, 170), (64, 64)], 1, 1, 256),
    ([(2500, 2500), (1023, 1029)], 4, 4, 128),
    ([(3000, 3000)], 6, 3, 64),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("causal", [True, False])
def test_against_the_formula(dev, case, causal):
    seqs, heads, kv_heads, dim = CASES[case]
    c = _case(dev, seqs, heads, kv_heads, dim, seed=case, packed=case % 2 == 1)
    out, lse = _run(c, causal)
    assert h3q.h3q_kernel_error_flag() == 0
    _check(c, causal, out, lse, what=f"case {case}")
    again = _run(c, causal)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1]), "other bits the second time"


@pytest.mark.parametrize("scale", [1.0, 0.004, 3.0])
def test_scale(dev, scale):
    """Sharp softmaxes move the reference maximum often, flat ones never."""
    c = _case(dev, [(300, 700), (256, 256)], 4, 2, 128, seed=40)
    for causal in (True, False):
        out, lse = _run(c, causal, scale=scale)
        _check(c, causal, out, lse, scale=scale)


def test_maxima_that_grow_and_fall(dev):
    """Scores that rise along the keys (the output is rescaled at every tile) and that fall."""
    for dim, heads in ((128, 2), (64, 2), (256, 1)):
        c = _case(dev, [(200, 1000), (200, 1000)], heads, heads, dim, seed=41)
        ramp = torch.linspace(0, 30, 1000, device=dev)
        c["q"][:, :, 0] = 4.0
        c["k"][:1000, :, 0] = ramp[:, None].bfloat16()
        c["k"][1000:2000, :, 0] = ramp.flip(0)[:, None].bfloat16()
        for causal in (True, False):
            out, lse = _run(c, causal)
            _check(c, causal, out, lse, what=f"dim {dim}")


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_values_that_are_no_numbers(dev, dim):
    """NaN and infinities in keys and values reach exactly the rows that see them."""
    c = _case(dev, [(300, 300), (200, 200), (90, 250)], 4, 2, dim, seed=42)
    out, _ = _run(c, True)
    clean = out.clone()
    bad = {name: c[name].clone() for name in "kv"}
    bad["v"][150, 0, 7] = float("nan")       # sequence 0, position 150, key head 0
    bad["v"][299, 1, 60] = float("inf")      # its last position
    bad["k"][300 + 130, 1, 3] = float("nan")  # sequence 1, position 130
    bad["v"][500 + 200, 0, 1] = float("-inf")  # sequence 2, position 200: seen by queries 40 on
    got, _ = _run({**c, **bad}, True)
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[150:300, 0:2, 7] = True
    hit[299, 2:4, 60] = True
    hit[300 + 130:500, 2:4, :] = True
    hit[500 + 40:590, 0:2, 1] = True
    assert torch.equal(got[~hit], clean[~hit])
    assert bool(torch.isnan(got[150:300, 0:2, 7]).all()) and bool(torch.isnan(got[430:500, 2:4]).all())
    assert bool((got[299, 2:4, 60] == float("inf")).all())
    assert bool((got[540:590, 0:2, 1] == float("-inf")).all())
    # without the causal mask every row of the sequence sees them, and no other sequence's
    clean, _ = _run(c, False)
    got, _ = _run({**c, **bad}, False)
    assert bool(torch.isnan(got[:300, 0:2, 7]).all()) and bool(torch.isnan(got[300:500, 2:4]).all())
    assert torch.equal(got[300:500, 0:2], clean[300:500, 0:2]) and torch.equal(got[500:, 2:4], clean[500:, 2:4])
    # and behind the last sequence nobody does
    c["v"][-3:] = float("nan")
    c["k"][-3:] = float("nan")
    for causal, want in ((True, out), (False, clean)):
        assert torch.equal(_run(c, causal)[0], want)


def test_queries_that_are_no_numbers(dev):
    c = _case(dev, [(200, 200)], 2, 1, 128, seed=43)
    out, _ = _run(c, True)
    q = c["q"].clone()
    q[50, 1, 0] = float("nan")
    q[60, 0, 5] = float("inf")
    got, _ = _run({**c, "q": q}, True)
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[50, 1] = hit[60, 0] = True
    assert torch.equal(got[~hit], out[~hit]) and bool(torch.isnan(got[hit]).all())


def test_lists_out_of_order(dev):
    """Lists that decrease or point past the rows: the good sequences' outputs stay right."""
    c = _case(dev, [(100, 100), (200, 200), (50, 50)], 4, 2, 128, seed=44)
    good, _ = _run(c, True)
    for cu_q, cu_k in (([0, 100, 50, 2 ** 31 - 1], [0, 100, 300, 350]), ([0, 100, -7, -7], [0, 100, 40, -9]),
                       ([0, 100, 300, 350], [0, 100, -5, 2 ** 31 - 1])):
        got, _ = _run({**c, "cu_q": cc.ints(cu_q, dev), "cu_k": cc.ints(cu_k, dev)}, True)
        assert torch.equal(got[:50], good[:50])
    assert h3q.h3q_kernel_error_flag() == 0


def test_no_keys_at_all(dev):
    c = _case(dev, [(70, 0)], 2, 1, 64, seed=45, tail=0)
    for causal in (True, False):
        out, lse = _run(c, causal)
        assert bool((out == 0).all()) and bool((lse == -np.inf).all())


def test_graph_replay_follows_the_lists(dev):
    c = _case(dev, [(300, 400), (100, 100)], 8, 2, 128, seed=46, tail=0)
    _run(c, True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = _run(c, True)
    for cu_q, cu_k in (([0, 300, 400], [0, 400, 500]), ([0, 1, 400], [0, 60, 500]), ([0, 200, 390], [0, 200, 400])):
        c["cu_q"].copy_(cc.ints(cu_q, dev))
        c["cu_k"].copy_(cc.ints(cu_k, dev))
        graph.replay()
        _check(c, True, out, lse, what=str(cu_q))


def test_two_streams_and_a_full_gpu(dev):
    """Calls on two streams that compete for the SMs with each other and with the block-scaled GEMM's TMEM."""
    cases = [_case(dev, [(900, 900), (600, 1500)], 8, 2, d, seed=47 + d) for d in (128, 64)]
    want = [_run(c, True) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for c, s in zip(cases, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(_run(c, True))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])


def test_between_its_neighbours(dev):
    """The calls as a prefill step makes them: QKV epilogue, cache write, attention over the prefix read back,
    quantize of the output; then a decoding step over the same cache agrees with the prompt's attention."""
    heads, dim, page, rows = 4, 128, 64, 333
    g = torch.Generator(device=dev)
    g.manual_seed(3)
    x = torch.randn((rows, 3 * heads * dim), generator=g, device=dev).bfloat16()
    bias = [torch.randn(heads * dim, generator=g, device=dev).bfloat16() for _ in range(3)]
    cos, sin = (torch.randn((rows, 64), generator=g, device=dev).bfloat16() for _ in range(2))
    q, k, v = h3q.h3q_qkv_epilogue(*x.split(heads * dim, 1), bias, cos, sin, heads, 1e-6)
    cache = h3q.kv_cache_nvfp4(12, heads, page, dim, dev)
    table = torch.randperm(12, device=dev).to(torch.int32)[None].contiguous()
    cu, length = cc.ints([0, rows], dev), cc.ints([rows], dev)
    gs = [torch.tensor([448.0 * 6 / float(t.float().abs().max())], device=dev) for t in (k, v)]
    h3q.h3q_kv_cache_write_nvfp4(k, v, cache, cu, length, table, *gs)
    kr, vr = h3q.h3q_kv_cache_read_nvfp4(cache, cu, length, table, *gs, rows=rows)
    assert float((kr.float() - k.float()).norm() / k.float().norm()) < 0.2
    out = h3q.h3q_attention_varlen(q, kr, vr, cu, cu, causal=True)
    codes, scales = h3q.h3q_quantize_nvfp4(out.view(rows, heads * dim), torch.tensor([100.0], device=dev))
    assert codes.shape == (rows, heads * dim // 2) and scales.shape[0] == 384
    last = h3q.h3q_attention_cache_nvfp4(q[-5:], cache, cc.ints([0, 5], dev), length, table, *gs, max_rows=5)
    # the same sums from bf16(k), bf16(v) and bf16 weights, and from the cache's exact values and fp16 weights
    k32, v32 = kr.float(), vr.float()
    w = torch.softmax(torch.einsum("nhd,khd->hnk", q[-5:].float(), k32) * dim ** -0.5, -1)
    spread = torch.einsum("hnk,khd->nhd", w, v32.abs())
    # bf16 keys and values are off by 2^-8 each, the scores by 2^-8 of a sum of magnitudes
    size = float(torch.einsum("nhd,khd->hnk", q[-5:].float().abs(), k32.abs()).max()) * dim ** -0.5
    tol = 2 * (2.0 ** -8 * (3 + size)) * spread + 2.0 ** -7 * last.float().abs()
    assert bool(((last.float() - out[-5:].float()).abs() <= tol).all())
