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
