"""GPU: block selection writes its lists, scores and workspace alone, whatever the offsets hold."""
import pytest
import torch

import block_cases as bc
import cache_cases as cc
import nvfp4_activation_quantize_gb300 as h3q

pytestmark = pytest.mark.gpu

GUARD = 1024   # elements on both sides


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


OFFSETS = [([0, 200, 400], [0, 300, 600]), ([0, 200, 10_000], [0, 300, 20_000]), ([0, 200, -5], [0, 300, -7]),
           ([5, 3, 1], [9, 4, 2]), ([0, 400, 200], [0, 600, 100]), ([399, 400, 400], [599, 600, 600]),
           ([-(1 << 31), 7, (1 << 31) - 1], [-(1 << 31), 7, (1 << 31) - 1]), ([0, 0, 0], [0, 0, 0])]


@pytest.mark.parametrize("cu_q, cu_k", OFFSETS)
@pytest.mark.parametrize("block_q, block_k, causal, many", [(128, 64, True, False), (64, 256, False, False), (64, 64, True, True)])
def test_nothing_outside_is_written(dev, cu_q, cu_k, block_q, block_k, causal, many):
    top, kv_heads, dim = 6, 2, 128
    c = bc.sequences(dev, [(200, 300), (200, 300)], 4, kv_heads, dim, seed=27, tail=0)
    if many:   # more sequences than a warp has lanes
        cu_q, cu_k = cu_q + cu_q[-1:] * 40, cu_k + cu_k[-1:] * 40
    batch = len(cu_q) - 1
    shape = (kv_heads, h3q.block_rows(400, batch, block_q), top)
    nbytes = h3q.select_blocks_workspace_bytes(400, 600, batch, kv_heads, dim, block_q, block_k)
    n = shape[0] * shape[1] * shape[2]
    lists = torch.full((n + 2 * GUARD,), 1234567, dtype=torch.int32, device=dev)
    scores = torch.full((n + 2 * GUARD,), 77.0, device=dev)
    ws = torch.full((nbytes + 2 * GUARD,), 171, dtype=torch.uint8, device=dev)
    before = {name: t.clone() for name, t in c.items()}
    got = h3q.h3q_select_blocks(c["q"], c["k"], cc.ints(cu_q, dev), cc.ints(cu_k, dev), top, block_q=block_q, block_k=block_k,
                                causal=causal, blocks=lists[GUARD:GUARD + n].view(shape),
                                scores=scores[GUARD:GUARD + n].view(shape), workspace=ws[GUARD:GUARD + nbytes])
    for t, keep, size in ((lists, 1234567, n), (scores, 77.0, n), (ws, 171, nbytes)):
        assert bool((t[:GUARD] == keep).all()) and bool((t[GUARD + size:] == keep).all())
    for name in ("q", "k", "v"):
        assert torch.equal(c[name], before[name])
    # (each list: ascending numbers of blocks that there are, then -1)
    assert bool((got >= -1).all()) and bool((got <= 600 // block_k).all())
    later = got[:, :, 1:]
    assert bool(((later == -1) | (later > got[:, :, :-1])).all())
    assert bool(((got == -1) == (scores[GUARD:GUARD + n].view(shape) == -float("inf"))).all())
