"""GPU: attention over the cache rounds each weight once, to fp16, also where the reference moves inside a tile after
some of the tile's weights were formed."""
import numpy as np
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


# Scores (sums of two bf16) of 32 keys of value 1, of one key of value -32 that nearly cancels them, and of a key
# of value 0 that moves the reference: chosen so that roundings of the first keys' weights, of the factor that
# takes them to the new reference and of the other key's weight all pull the same way.
SCORES = [
    ((4.90625, -0.0135498046875), (4.90625, -0.01361083984375), (8.3125, -0.02978515625)),
    ((4.875, -0.002197265625), (4.875, -0.0020599365234375), (7.59375, 0.01202392578125)),
    ((4.90625, -0.01544189453125), (4.90625, -0.01531982421875), (6.21875, 0.0093994140625)),
    ((4.90625, -0.01348876953125), (4.90625, -0.01361083984375), (6.90625, 0.01397705078125)),
    ((4.875, 0.00634765625), (4.875, 0.006500244140625), (7.59375, 0.01495361328125)),
    ((4.875, 0.00634765625), (4.875, 0.006500244140625), (20.0, 0.01495361328125)),    # factors below 2^-24
    ((4.875, 0.00634765625), (4.875, 0.006500244140625), (40.0, 0.01495361328125)),
]


@pytest.mark.parametrize("heads, dim", [(16, 64), (32, 64), (24, 64), (8, 64), (16, 128), (24, 128), (32, 128), (48, 128),
                                        (16, 256), (8, 256)])
@pytest.mark.parametrize("case", range(len(SCORES)))
def test_each_weight_is_rounded_once(dev, heads, dim, case):
    keys, page, one = 512, 64, 0x38   # scale byte of 1
    cache = h3q.kv_cache_nvfp4(keys // page, 1, page, dim, dev)
    kc, ks, vc, vs = (t.view(keys, -1) for t in cache)
    q = torch.zeros((1, heads, dim), device=dev)
    for i, (at, n) in enumerate(((256, 32), (288, 1), (289, 1))):   # the second tile's first 64 keys
        q[:, :, 2 * i], q[:, :, 2 * i + 1] = SCORES[case][i]
        kc[at:at + n, i] = 0x22      # elements 2 i and 2 i + 1 are 1
        ks[at:at + n, 0] = one
    vc[256:288], vs[256:288] = 0x22, one
    vc[288], vs[288] = 0xCC, 0x58    # -2 times 16
    q = q.bfloat16()
    table = torch.arange(keys // page, dtype=torch.int32, device=dev)[None].contiguous()
    unit = torch.ones(1, device=dev)
    lse = torch.empty((heads, 1), device=dev)
    out = h3q.h3q_attention_cache_nvfp4(q, cache, cc.ints([0, 1], dev), cc.ints([keys], dev), table, unit, unit, scale=1.0,
                                        lse=lse)
    k, v = cc.cache_values64(cache, (1.0, 1.0), table[0], keys, page)
    want, want_lse, spread, size = cc.attention64(q, k, v, torch.ones((1, keys), dtype=torch.bool, device=dev), 1.0)
    # The sum of the weights is formed before they are rounded: a weight's rounding (2^-11 of it, or half of fp16's
    # smallest step, 2^-25, beside a largest weight of 2^5 at least) moves the numerator alone.  Exponents, powers and
    # sums in fp32 as in cache_cases.check_attention.
    fp32 = 2.0 ** -19 * (size + 8) + 2.0 ** -22 * (keys / 16 + 8)
    tol = want.abs() * 2.0 ** -8 + spread * (2.0 ** -11 + 2 * fp32) + 2.0 ** -30 * float(v.abs().sum(0).max())
    err = (out.double() - want).abs()
    assert bool((err <= tol).all()), f"off by {float((err / tol).max()):.3g} of what is allowed"
    assert float((lse.double() - want_lse).abs().max()) <= 2 * fp32 + float(want_lse.abs().max()) * 2.0 ** -22
