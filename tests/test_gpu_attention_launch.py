"""GPU: launches of the prompt kernel that are mostly blocks without a unit: many sequences of nothing."""
import pytest
import torch

import cache_cases as cc
import nvfp4_activation_quantize_gb300 as h3q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


@pytest.mark.parametrize("dim, heads, kv_heads", [(64, 8, 8), (128, 8, 2), (256, 3, 3)])
@pytest.mark.parametrize("where", [0, 700, 1999])
def test_sequences_of_nothing(dev, dim, heads, kv_heads, where):
    """One sequence of rows among 2,000 of none: 0 to 8 units in up to 8 x 2,000 blocks."""
    n, batch = 300, 2000
    g = torch.Generator(device=dev)
    g.manual_seed(where)
    q, k, v = (torch.randn((n, h, dim), generator=g, device=dev).bfloat16() for h in (heads, kv_heads, kv_heads))
    cu = torch.zeros(batch + 1, dtype=torch.int32, device=dev)
    cu[where + 1:] = n
    want = h3q.h3q_attention_varlen(q, k, v, cc.ints([0, n], dev), cc.ints([0, n], dev))
    for _ in range(3):
        out = torch.full_like(want, 9.0)
        h3q.h3q_attention_varlen(q, k, v, cu, cu, out=out)
        assert torch.equal(out, want)
    assert h3q.h3q_kernel_error_flag() == 0


def test_many_heads_and_many_empty_sequences(dev):
    """Blocks are launched for the pairs of row tiles that a row can be in: one row of 2^18 heads among 8,256
    sequences is 2^18 of them, not 2^31."""
    heads, dim, batch = 1 << 18, 64, 8256
    q, k, v = (torch.randn((1, heads, dim), device=dev).bfloat16() for _ in range(3))
    cu = torch.zeros(batch + 1, dtype=torch.int32, device=dev)
    cu[5000:] = 1
    assert torch.equal(h3q.h3q_attention_varlen(q, k, v, cu, cu), v)   # (one key: its weight is 1)
    assert h3q.h3q_kernel_error_flag() == 0


def test_as_many_sequences_as_are_allowed(dev):
    batch = 1 << 24
    q, k, v = (torch.randn((1, 1, 64), device=dev).bfloat16() for _ in range(3))
    cu = torch.zeros(batch + 1, dtype=torch.int32, device=dev)
    cu[-1] = 1
    assert torch.equal(h3q.h3q_attention_varlen(q, k, v, cu, cu), v)
    cache = h3q.kv_cache_nvfp4(2, 1, 16, 64, dev)
    length = torch.zeros(batch, dtype=torch.int32, device=dev)
    length[-1] = 1
    table = torch.ones((batch, 1), dtype=torch.int32, device=dev)
    one = torch.ones(1, device=dev)
    h3q.h3q_kv_cache_write_nvfp4(k, v, cache, cu, length, table, one, one)
    _, back = h3q.h3q_kv_cache_read_nvfp4(cache, cu, length, table, one, one, rows=1)
    assert torch.equal(h3q.h3q_attention_cache_nvfp4(q, cache, cu, length, table, one, one), back)
    assert h3q.h3q_kernel_error_flag() == 0
