"""GPU: the kernels that allocate an SM's tensor memory (the block-scaled GEMM, prompt attention, cache attention of
many rows) on streams of their own beside each other and beside the library's products, which use it too: the same
bits as one after the other, and no wait runs out."""
import pytest
import torch

import cache_cases as cc
import nvfp4_activation_quantize_gb300 as h3q

pytestmark = pytest.mark.gpu


def test_all_at_once():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(2)

    def rand(*shape):
        return torch.randn(shape, generator=g, device=dev).bfloat16()

    one = torch.ones(1, device=dev)
    a, b = (h3q.h3q_quantize_nvfp4(rand(n, 1024), one) for n in (2048, 4096))
    q, k, v = rand(2100, 16, 128), rand(2100, 4, 128), rand(2100, 4, 128)
    cu = cc.ints([0, 900, 2100], dev)
    cache = h3q.kv_cache_nvfp4(40, 4, 64, 128, dev)
    table = torch.randperm(40, device=dev)[:38].to(torch.int32).view(2, 19).contiguous()
    length = cc.ints([900, 1200], dev)
    h3q.h3q_kv_cache_write_nvfp4(k, v, cache, cu, length, table, one, one)
    chains = cc.ints([0, 40, 100], dev)
    x, y = rand(4096, 4096), rand(4096, 4096)
    z = torch.empty((4096, 4096), dtype=torch.bfloat16, device=dev)
    calls = [
        lambda: h3q.h3q_gemm_swiglu_nvfp4(*a, *b, one, one),
        lambda: [h3q.h3q_attention_varlen(q, k, v, cu, cu)],
        lambda: [h3q.h3q_attention_cache_nvfp4(q[:100], cache, chains, length, table, one, one, max_rows=60)],
        lambda: [h3q.h3q_attention_cache_nvfp4(q[:100, :4], cache, chains, length, table, one, one, max_rows=60)],
        lambda: [torch.mm(x, y, out=z)],
    ]
    want = [[t.clone() for t in call()] for call in calls[:-1]]
    assert h3q.h3q_kernel_error_flag() == 0
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for i, (call, stream) in enumerate(zip(calls, streams)):
            with torch.cuda.stream(stream):
                outs = call()
                if i < len(want):
                    got.append((i, outs))
    torch.cuda.synchronize()
    assert h3q.h3q_kernel_error_flag() == 0
    for i, outs in got:
        for w, o in zip(want[i], outs):
            assert torch.equal(w, o), f"call {i}"
