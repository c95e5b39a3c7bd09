"""GPU: calls on a stream given as an argument, with outputs (and a workspace) that the binding allocates: the
memory may be what work queued on the current stream still uses, and is not given away while the call runs."""
import pytest
import torch

import cache_cases as cc
import nvfp4_activation_quantize_gb300 as h3q

pytestmark = pytest.mark.gpu

CYCLES = 40_000_000   # some 20 ms


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


@pytest.fixture(scope="module")
def calls(dev):
    """name -> call(stream), each returning its allocated outputs."""
    g = torch.Generator(device=dev)
    g.manual_seed(5)

    def rand(*shape):
        return torch.randn(shape, generator=g, device=dev).bfloat16()

    x, up, gamma, table = rand(512, 512), rand(512, 512), rand(512), rand(4, 2, 512)
    one = torch.ones(1, device=dev)
    codes, scales = h3q.h3q_quantize_nvfp4(x, one)
    weight = torch.randint(0, 256, (512, 256), generator=g, device=dev, dtype=torch.uint8)
    weight_scales = torch.randint(0, 120, (512, 32), generator=g, device=dev, dtype=torch.uint8)
    amax, rstd = torch.full((1,), 3.0, device=dev), torch.ones(512, device=dev)
    h, gate = torch.randn((512, 512), generator=g, device=dev), rand(4, 512)
    biases = [rand(512) for _ in range(3)]
    q, k, v = rand(400, 8, 128), rand(400, 2, 128), rand(400, 2, 128)
    cache = h3q.kv_cache_nvfp4(16, 2, 64, 128, dev)
    cu, length = cc.ints([0, 400], dev), cc.ints([400], dev)
    pages = torch.randperm(16, device=dev)[:7].to(torch.int32)[None].contiguous()
    h3q.h3q_kv_cache_write_nvfp4(k, v, cache, cu, length, pages, one, one)
    last, ones = q[-40:], (cc.ints([0, 40], dev), length, pages, one, one)
    ws = torch.empty(h3q.attention_cache_workspace_bytes(40, 8, 2, 128), dtype=torch.uint8, device=dev)
    torch.cuda.synchronize()
    frames = {"rows_per_frame": 128}
    return {
        "quantize": lambda s: h3q.h3q_quantize_nvfp4(x, one, stream=s),
        "adaln": lambda s: h3q.h3q_rmsnorm_adaln_nvfp4(x, gamma, table, one, **frames, stream=s),
        "swiglu": lambda s: h3q.h3q_swiglu_nvfp4(x, up, one, stream=s),
        "dequantize": lambda s: [h3q.h3q_dequantize_nvfp4(codes, scales, one, stream=s)],
        "amax": lambda s: [h3q.h3q_amax_bf16(x, stream=s)],
        "adaln amax": lambda s: [h3q.h3q_rmsnorm_adaln_amax(x, gamma, table, **frames, stream=s)],
        "from rstd": lambda s: h3q.h3q_rmsnorm_adaln_nvfp4_from_rstd(x, gamma, table, rstd, one, **frames, stream=s),
        "swiglu amax": lambda s: [h3q.h3q_swiglu_amax(x, up, stream=s)],
        "scale": lambda s: [h3q.h3q_global_scale_from_amax(amax, stream=s)],
        "dynamic": lambda s: h3q.h3q_quantize_nvfp4_dynamic(x, stream=s),
        "residual": lambda s: h3q.h3q_residual_rmsnorm_adaln_nvfp4(h, torch.zeros_like(x), gate, gamma, table, one,
                                                                   **frames, stream=s),
        "packed": lambda s: h3q.h3q_swiglu_packed_nvfp4(x, one, stream=s),
        "qkv": lambda s: h3q.h3q_qkv_epilogue(x, x, x, biases, None, None, 4, 1e-6, stream=s),
        "gemm": lambda s: h3q.h3q_gemm_swiglu_nvfp4(codes, scales, weight, weight_scales, one, one, stream=s),
        "read": lambda s: h3q.h3q_kv_cache_read_nvfp4(cache, cu, length, pages, one, one, rows=400, stream=s),
        "cached": lambda s: [h3q.h3q_attention_cache_nvfp4(last, cache, *ones, max_rows=40, stream=s)],
        "cached, own workspace": lambda s: [h3q.h3q_attention_cache_nvfp4(last, cache, *ones, max_rows=40, workspace=ws,
                                                                          stream=s)],
        "varlen": lambda s: [h3q.h3q_attention_varlen(q, k, v, cu, cu, stream=s)],
    }


NAMES = ["quantize", "adaln", "swiglu", "dequantize", "amax", "adaln amax", "from rstd", "swiglu amax", "scale", "dynamic",
         "residual", "packed", "qkv", "gemm", "read", "cached", "cached, own workspace", "varlen"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("given", ["object", "handle"])
def test_memory_that_queued_work_still_uses(dev, calls, name, given):
    call = calls[name]
    want = [t.clone() for t in call(None)]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    old = [torch.empty_like(t) for t in want]
    torch.cuda._sleep(CYCLES)
    for t in old:   # queued on the current stream, behind the wait
        t.fill_(77)
    del old, t      # so the next allocations of these sizes may be the same memory
    got = call(stream if given == "object" else stream.cuda_stream)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b), name


@pytest.mark.parametrize("name", NAMES)
def test_memory_is_kept_while_the_call_runs(dev, calls, name):
    call = calls[name]
    shapes = [(t.shape, t.dtype) for t in call(None)]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(CYCLES)
    got = call(stream)
    del got
    other = [torch.full(shape, 33, dtype=dtype, device=dev) for shape, dtype in shapes]
    torch.cuda.synchronize()
    for t in other:
        assert bool((t == 33).all()), name


def test_streams_inside_a_graph(dev, calls):
    """The stream of a capture given as the argument, and one that the capture has forked to."""
    want = [t.clone() for t in calls["quantize"](None) + calls["read"](None)]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        got = [*calls["quantize"](main), *calls["read"](side)]
        main.wait_stream(side)
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("number", [0, 1, 2])
def test_the_default_streams_by_number(dev, calls, number):
    """0 and 1 are the legacy default stream, 2 is the thread's own."""
    want = [t.clone() for t in calls["quantize"](None)]
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = calls["quantize"](number)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
