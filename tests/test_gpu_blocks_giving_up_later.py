"""GPU: attention over blocks whose waits run out in a unit that is not a CTA's first, and in halves of units."""
import pytest
import torch

import block_cases as bc
import nvfp4_activation_quantize_gb300 as h3q
from test_gpu_blocks_giving_up import LIMITS, _use, dev, libraries  # noqa: F401

pytestmark = pytest.mark.gpu

CASES = [  # (queries, keys), query heads, key heads, dim, block_q, block_k, top, causal
    ([(900, 900)] * 8 + [(300, 1500)] * 8, 16, 16, 128, 128, 128, 6, False),
    ([(900, 900)] * 8 + [(300, 1500)] * 8, 24, 6, 128, 64, 64, 9, True),
    ([(n, n) for n in range(1, 400)], 8, 2, 64, 64, 64, 4, True),
    ([(6900, 2000)], 24, 24, 128, 128, 64, 7, False),
]


@pytest.mark.parametrize("limit", LIMITS)
@pytest.mark.parametrize("case", range(len(CASES)))
def test_calls_that_give_up(dev, libraries, case, limit):  # noqa: F811
    seqs, heads, kv_heads, dim, block_q, block_k, top, causal = CASES[case]
    c = bc.sequences(dev, seqs, heads, kv_heads, dim, seed=case)
    lists = bc.random_lists(c, kv_heads, block_q, block_k, top, case)
    rows = int(c["cu_q"][-1])

    def call():
        out = torch.full(c["q"].shape, 5.0, dtype=torch.bfloat16, device=dev)
        lse = torch.full((heads, c["q"].shape[0]), 6.0, device=dev)
        h3q.h3q_attention_blocks(c["q"], c["k"], c["v"], c["cu_q"], c["cu_k"], lists, block_q=block_q, block_k=block_k,
                                 causal=causal, out=out, lse=lse)
        return out, lse

    regular = h3q.library()
    want = call()
    assert h3q.h3q_kernel_error_flag() == 0
    gave_up = 0
    try:
        _use(libraries[limit])
        for _ in range(4):
            out, lse = call()
            gave_up += h3q.h3q_kernel_error_flag()
            assert bool((out[rows:] == 5.0).all()) and bool((lse[:, rows:] == 6.0).all()), "rows of no sequence"
            assert bool(((out == want[0]) | (out == 5.0)).all()) and bool(((lse == want[1]) | (lse == 6.0)).all())
    finally:
        _use(regular)
    if limit == 0:
        assert gave_up == 4
    again = call()
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
    assert h3q.h3q_kernel_error_flag() == 0
