"""GPU: attention over blocks and block selection where there are no keys, no queries, or no sequences at all."""
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


@pytest.mark.parametrize("rows_q, rows_k, ends_q, ends_k", [
    (200, 0, [0, 150, 190], [0, 0, 0]), (0, 200, [0, 0, 0], [0, 150, 190]), (0, 0, [0], [0]), (200, 200, [0], [0]),
    (1, 1, [0, 0, 1], [0, 1, 1])])
@pytest.mark.parametrize("dim", [64, 128])
def test_nothing_to_see(dev, rows_q, rows_k, ends_q, ends_k, dim):
    q = torch.randn((rows_q, 4, dim), device=dev).bfloat16()
    k = torch.full((rows_k, 2, dim), float("nan"), device=dev).bfloat16()
    cu_q, cu_k = cc.ints(ends_q, dev), cc.ints(ends_k, dev)
    lists = h3q.h3q_select_blocks(q, k, cu_q, cu_k, 3, block_q=64, block_k=64)
    assert lists.shape == (2, rows_q // 64 + len(ends_q) - 1, 3) and bool((lists == -1).all())
    lists.zero_()
    out = torch.full((rows_q, 4, dim), 5.0, device=dev, dtype=torch.bfloat16)
    lse = torch.full((4, rows_q), 6.0, device=dev)
    h3q.h3q_attention_blocks(q, k, k, cu_q, cu_k, lists, block_q=64, block_k=64, out=out, lse=lse)
    assert h3q.h3q_kernel_error_flag() == 0
    end = ends_q[-1]
    assert bool((out[:end] == 0).all()) and bool((lse[:, :end] == -float("inf")).all())
    assert bool((out[end:] == 5.0).all()) and bool((lse[:, end:] == 6.0).all())
