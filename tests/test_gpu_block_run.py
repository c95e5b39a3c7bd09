"""GPU: the calls of one transformer block of a video as they follow each other -- the QKV epilogue with rotary axes, the
blocks that are selected, attention over them, its output quantized, and the norms around the block with the gated
residual -- each step against its definition on what the step before gave, eagerly and from a graph that is replayed."""
import numpy as np
import pytest
import torch

import block_cases as bc
import cache_cases as cc
import nvfp4_activation_quantize_gb300 as h3q
import oracle
import test_gpu_postnorm as norms
import test_gpu_qkv_axes as axes
from parity import bits, check_rows, gsf_tensor

pytestmark = pytest.mark.gpu

HEADS, DIM, DIMS, FRAMES, HIGH, WIDE = 4, 128, (44, 42, 42), 5, 10, 12
ROWS = FRAMES * HIGH * WIDE


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


def _inputs(dev, seed):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device=dev).bfloat16()  # noqa: E731
    d = HEADS * DIM
    n = torch.arange(ROWS, device=dev)
    return {"qkv": r(ROWS, 3 * d), "biases": (r(d), r(d), r(d)), "weights": (r(DIM), r(DIM)),
            "positions": torch.stack((n // (HIGH * WIDE), n // WIDE % HIGH, n % WIDE), 1).int().contiguous(),
            "h": torch.randn((ROWS, d), generator=g, device=dev), "post": r(d), "gamma": r(d), "bias": r(d),
            "gate": r(FRAMES, d), "table": r(FRAMES, 2, d), "cu": cc.ints([0, ROWS], dev),
            "gsf": gsf_tensor(300.0, dev), "gsf2": gsf_tensor(250.0, dev)}


def _block(w):
    """The run of calls; h is updated in place."""
    d = HEADS * DIM
    qkv = w["qkv"]
    q, k, v = h3q.h3q_qkv_epilogue_axes(qkv[:, :d], qkv[:, d:2 * d], qkv[:, 2 * d:], w["positions"], DIMS, HEADS,
                                        biases=w["biases"], weights=w["weights"], interleaved=True)
    lists = h3q.h3q_select_blocks(q, k, w["cu"], w["cu"], 4, block_q=128, block_k=64, first=1)
    lse = torch.empty((HEADS, ROWS), device=qkv.device)
    o = h3q.h3q_attention_blocks(q, k, v, w["cu"], w["cu"], lists, block_q=128, block_k=64, lse=lse)
    codes, scales = h3q.h3q_quantize_nvfp4(o.view(ROWS, d), w["gsf"])
    # (the output projection is the library user's; its result is taken to be the attention's)
    after = h3q.h3q_postnorm_residual_adaln_nvfp4(w["h"], o.view(ROWS, d), w["post"], w["gamma"], w["gsf2"],
                                                  bias=w["bias"], gate_table=w["gate"], mod_table=w["table"],
                                                  residual_scale=0.5, rows_per_frame=HIGH * WIDE)
    return {"q": q, "k": k, "v": v, "lists": lists, "o": o, "lse": lse, "codes": codes, "scales": scales, "after": after}


def _check(w, h, got):
    d = HEADS * DIM
    for i, name in enumerate("qk"):
        want, size = axes._want(w["qkv"][:, i * d:(i + 1) * d], w["biases"][i], w["weights"][i], w["positions"], DIMS,
                                [1e4] * 3, [1.0] * 3, False, True, True, 1e-6, HEADS)
        axes._check(got[name], want, size, name)
    c = {"q": got["q"], "k": got["k"], "v": got["v"], "cu_q": w["cu"], "cu_k": w["cu"]}
    want, _ = bc.selected(c, 4, 128, 64, False, 1)
    assert (got["lists"].cpu().numpy() == want).all()
    bc.check_blocks(c, got["lists"], 128, 64, False, got["o"], got["lse"])
    codes, sf = oracle.quantize_rows(bits(got["o"]).reshape(ROWS, d), 300.0)
    check_rows(got["codes"], got["scales"], np.arange(ROWS), d, codes, sf, "attention's output")
    n = dict(w, h=h, o=got["o"].view(ROWS, d))
    want_h, codes, sf, _ = norms._want(n, np.arange(ROWS) // (HIGH * WIDE), 0.5, 1e-6, 250.0)
    assert (w["h"].cpu().numpy().view(np.uint32) == want_h.view(np.uint32)).all()
    check_rows(*got["after"], np.arange(ROWS), d, codes, sf, "after the norms")


def test_a_run_of_calls(dev):
    w = _inputs(dev, 1)
    h = w["h"].clone()
    _check(w, h, _block(w))
    assert h3q.h3q_kernel_error_flag() == 0


def test_the_run_in_a_graph(dev):
    w = _inputs(dev, 2)
    stream = torch.cuda.Stream(dev)
    stream.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(stream):
        _block(w)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            got = _block(w)
    torch.cuda.synchronize()
    for seed in (3, 4):
        other = _inputs(dev, seed)
        for name, t in other.items():
            for a, b in zip(w[name], t) if isinstance(t, tuple) else ((w[name], t),):
                a.copy_(b)
        h = w["h"].clone()
        graph.replay()
        torch.cuda.synchronize()
        _check(w, h, got)


def test_graphs_that_share_a_workspace(dev):
    """Two captured selections with one workspace, replayed in turn."""
    cases = [bc.sequences(dev, [(300 + 50 * s, 1500)], 2, 2, 128, seed=s) for s in (5, 6)]
    ws = torch.empty(max(h3q.select_blocks_workspace_bytes(c["q"].shape[0], c["k"].shape[0], 1, 2, 128, 64, 64)
                         for c in cases), dtype=torch.uint8, device=dev)
    graphs = []
    for c in cases:
        lists = torch.empty((2, h3q.block_rows(c["q"].shape[0], 1, 64), 6), dtype=torch.int32, device=dev)
        call = lambda c=c, lists=lists: h3q.h3q_select_blocks(  # noqa: E731
            c["q"], c["k"], c["cu_q"], c["cu_k"], 6, block_q=64, block_k=64, causal=True, blocks=lists, workspace=ws)
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        graphs.append((graph, c, lists))
    for graph, _, lists in graphs * 2:
        lists.fill_(-9)
        graph.replay()
    torch.cuda.synchronize()
    for _, c, lists in graphs:
        want, _ = bc.selected(c, 6, 64, 64, True, 0)
        assert (lists.cpu().numpy() == want).all()


CYCLES = 40_000_000   # some 20 ms


def test_outputs_on_another_stream(dev):
    """Outputs and a workspace that the binding allocates for a call on a stream given as an argument: their memory may
    still be used by work queued on the current stream."""
    w = _inputs(dev, 7)
    d = HEADS * DIM
    q = w["qkv"][:, :d].unflatten(1, (HEADS, DIM))
    k = w["qkv"][:, d:2 * d].unflatten(1, (HEADS, DIM))
    lists = h3q.h3q_select_blocks(q, k, w["cu"], w["cu"], 3)
    calls = {
        "axes": lambda s: h3q.h3q_qkv_epilogue_axes(w["qkv"][:, :d], w["qkv"][:, d:2 * d], w["qkv"][:, 2 * d:],
                                                    w["positions"], DIMS, HEADS, stream=s),
        "select": lambda s: [h3q.h3q_select_blocks(q, k, w["cu"], w["cu"], 3, stream=s)],
        "blocks": lambda s: [h3q.h3q_attention_blocks(q, k, k, w["cu"], w["cu"], lists, stream=s)],
        "postnorm": lambda s: h3q.h3q_postnorm_residual_adaln_nvfp4(
            torch.zeros_like(w["h"]) if s is None else zero, w["qkv"][:, :d], w["post"], w["gamma"], w["gsf"], stream=s),
    }
    stream = torch.cuda.Stream(dev)
    for name, call in calls.items():
        zero = torch.zeros_like(w["h"])
        want = [t.clone() for t in call(None)]
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        size = max(t.numel() * t.element_size() for t in want)
        junk = [torch.empty(size, dtype=torch.uint8, device=dev) for _ in range(6)]
        torch.cuda._sleep(CYCLES)
        for t in junk:   # written late, after the memory has been given back
            t.fill_(255)
        del junk, t
        got = call(stream)
        stream.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name
        torch.cuda.synchronize()
