"""The cache's attention without max_rows takes one new token a sequence: more rows than sequences are refused, not
left uncomputed."""
import pytest
import torch

import cache_cases as cc
import nvfp4_activation_quantize_gb300 as h3q


def _call(dev, rows, batch, **kw):
    cache = h3q.kv_cache_nvfp4(4, 2, 16, 64, dev)
    q = torch.ones((rows, 4, 64), dtype=torch.bfloat16, device=dev)
    one = torch.ones(1, device=dev)
    cu = cc.ints([min(rows, i * -(-rows // batch)) for i in range(batch + 1)], dev)
    table = cc.ints([[i] for i in range(batch)], dev)
    return h3q.h3q_attention_cache_nvfp4(q, cache, cu, cc.ints([16] * batch, dev), table, one, one, **kw)


@pytest.mark.parametrize("rows, batch", [(2, 1), (5, 2), (64, 4)])
def test_chains_need_max_rows(rows, batch):
    with pytest.raises(ValueError, match="give max_rows"):
        _call("cpu", rows, batch)


@pytest.mark.gpu
def test_one_token_a_sequence_does_not():
    assert bool((_call("cuda:0", 3, 3) == 0).all())   # (values of an empty cache)
    assert bool((_call("cuda:0", 6, 3, max_rows=2) == 0).all())
    with pytest.raises(ValueError, match="give max_rows"):
        _call("cuda:0", 6, 3)


def test_heads_of_no_elements_are_refused_as_such():
    q, lists = torch.zeros((1, 2, 0), dtype=torch.bfloat16), cc.ints([0, 1], "cpu")
    with pytest.raises(ValueError, match="CUDA tensor"):
        h3q.h3q_attention_varlen(q, q, q, lists, lists)
    cache = h3q.kv_cache_nvfp4(2, 2, 16, 0, "cpu")
    with pytest.raises(ValueError, match="CUDA tensor"):
        h3q.h3q_attention_cache_nvfp4(q, cache, lists, cc.ints([1], "cpu"), cc.ints([[0]], "cpu"), torch.ones(1), torch.ones(1))


@pytest.mark.gpu
def test_heads_of_no_elements_on_the_gpu():
    q, lists = torch.zeros((1, 2, 0), dtype=torch.bfloat16, device="cuda:0"), cc.ints([0, 1], "cuda:0")
    with pytest.raises((ValueError, h3q.H3QError), match="head_dim"):
        h3q.h3q_attention_varlen(q, q, q, lists, lists)
