"""GPU: prompt attention of large values under scores that rise between the key tiles: the output is the values'
weighted mean, however far a tile's weights lie above those before it.  (At 59 a step the weights once reached 2^59
against the reference before, and 2^70 times that is no fp32 number.)"""
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


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("step", [7.0, 15.5, 16.5, 59.0, 63.5])
@pytest.mark.parametrize("size", [2.0 ** 70, 2.0 ** 86])
def test_large_values_and_rising_scores(dev, causal, dim, step, size):
    """Scores that rise by `step` (units of log2) from one 64-key stretch to the next.  All values of a column are
    the same, so that the output is that value: the weights, each rounded to bf16 (2^-8 of it), and their fp32
    sums cancel to 2^-8 + 2^-20, and the output is rounded to bf16 (2^-8)."""
    n, heads = 700, 2
    q = torch.zeros((n, heads, dim), device=dev)
    k = torch.zeros((n, heads, dim), device=dev)
    q[:, :, 0] = 1.0
    # (a score in two parts of at most 8 bits each, exact in bf16)
    rise = torch.arange(n, device=dev) // 64 * step
    high = rise.bfloat16()
    k[:, :, 0] = high.float()[:, None]
    q[:, :, 1] = 1.0
    k[:, :, 1] = (rise - high.float())[:, None]
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    column = (torch.rand((1, heads, dim), generator=g, device=dev) + 1).bfloat16() * (size / 2)
    v = column.expand(n, heads, dim).contiguous()
    cu = cc.ints([0, n], dev)
    out = h3q.h3q_attention_varlen(q.bfloat16(), k.bfloat16(), v, cu, cu, causal=causal, scale=0.6931471805599453)
    err = (out.double() - column.double()).abs() / column.double()
    assert float(err.max()) <= 2 * 2.0 ** -8 + 2.0 ** -16 + 2.0 ** -19


@pytest.mark.parametrize("v_scale", [3.0e38, 1.0e36, 1.0, 1.0e-34])
@pytest.mark.parametrize("new, heads, keys", [(1, 8, 6000), (1, 8, 40), (9, 8, 3000), (2, 16, 900)])
def test_values_near_the_ends_of_fp32(dev, v_scale, new, heads, keys):
    """Global scales of very small and of very large values: what the cache stands for is a number of fp32's range,
    and so is the mean, whatever the sum of the weights is."""
    page, kv_heads, dim = 64, 2, 128
    table, pages = cc.paged(dev, [keys], page, 3)
    cache = cc.random_cache(dev, pages, kv_heads, page, dim, 4)
    cache[2].fill_(0x77)           # values of 6 ...
    cache[3].copy_(cache[3] % 16 + 0x6f)   # ... under scales of 120 to 448: the mean is far above fp32's smallest
    g = torch.Generator(device=dev)
    g.manual_seed(6)
    q = torch.randn((new, heads, dim), generator=g, device=dev).bfloat16()
    lse = torch.empty((heads, new), device=dev)
    gs = (2688.0, float(torch.tensor(v_scale)))
    out = h3q.h3q_attention_cache_nvfp4(q, cache, cc.ints([0, new], dev), cc.ints([keys], dev), table,
                                        *(torch.tensor([x], device=dev) for x in gs), max_rows=new, lse=lse)
    k, v = cc.cache_values64(cache, gs, table[0], keys, page)
    seen = torch.ones((new, keys), dtype=torch.bool, device=dev).tril(keys - new)
    cc.check_attention(out, lse, cc.attention64(q, k, v, seen, dim ** -0.5), keys, 2.0 ** -11, f"scale {v_scale}")
    assert bool((out != 0).any())
