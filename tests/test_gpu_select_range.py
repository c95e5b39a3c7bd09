"""GPU: block selection where sums are formed of large values that cancel, at ordinary sizes and near fp32's ends: the
lists are those of scores in 64 bits wherever the sums' lengths fit fp32."""
import pytest
import torch

import block_cases as bc
from test_gpu_select_many_lists import check, dev  # noqa: F401

pytestmark = pytest.mark.gpu


def cancelling(x, block, size, seed):
    """Blocks of rows that cancel but for two small rows of each, all values times 2^size."""
    g = torch.Generator(device=x.device)
    g.manual_seed(seed)
    half = block // 2 - 1
    for rows in x.split(block):
        if rows.shape[0] < block:
            continue
        large = torch.randn((half, *x.shape[1:]), generator=g, device=x.device).bfloat16()
        rows[:half] = large
        rows[half:2 * half] = -large[torch.randperm(half, generator=g, device=x.device)]
        rows[2 * half:] = (rows[2 * half:].float() * 2.0 ** -13).bfloat16()
    x.copy_((x.float() * 2.0 ** size).bfloat16())


CASES = [  # query heads, key heads, dim, block_q, block_k, which cancel, 2^ of q's values and of k's
    (2, 2, 64, 64, 64, "k", 0, 0), (2, 2, 64, 64, 64, "k", -100, 112), (4, 2, 128, 64, 256, "k", -90, 115),
    (2, 2, 128, 128, 64, "q", 112, -100), (6, 2, 64, 256, 128, "q", 116, -60), (2, 2, 64, 64, 64, "qk", 112, -90),
    (2, 2, 64, 64, 64, "k", 0, 120), (2, 2, 64, 64, 64, "k", 20, -110),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_large_values_that_cancel(dev, case):  # noqa: F811
    heads, kv_heads, dim, block_q, block_k, which, size_q, size_k = CASES[case]
    c = bc.sequences(dev, [(block_q * 6, block_k * 50)], heads, kv_heads, dim, seed=60 + case, tail=0)
    for name, block, size in (("q", block_q, size_q), ("k", block_k, size_k)):
        if name in which:
            cancelling(c[name], block, size, case)
        else:
            c[name].copy_((c[name].float() * 2.0 ** size).bfloat16())
    check(c, 20, block_q, block_k, False, 0)


def test_sums_that_pass_the_end_on_the_way(dev):  # noqa: F811
    """Partial sums beyond fp32, sums that fit."""
    c = bc.sequences(dev, [(64, 64 * 40)], 1, 1, 64, seed=70, tail=0)
    k = c["k"].view(40, 64, 64)
    k[:, :24] = 1.5 * 2.0 ** 126
    k[:, 24:48] = -1.5 * 2.0 ** 126
    k[:, 48:] *= 2.0 ** 112
    c["q"] *= 2.0 ** -100
    check(c, 10, 64, 64, False, 0)
