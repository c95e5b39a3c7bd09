"""GPU: block selection, whose lists equal those of scores in 64 bits: head sizes and groups, sizes of blocks, ragged
lengths, ties, scores that fp32 cannot tell apart, blocks that are always kept, workspaces, graphs."""
import numpy as np
import pytest
import torch

import block_cases as bc
import cache_cases as cc
import nvfp4_activation_quantize_gb300 as h3q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


def _check(c, top, block_q, block_k, causal, first, what="", scores=True):
    lists = torch.full((c["k"].shape[1], h3q.block_rows(c["q"].shape[0], c["cu_q"].shape[0] - 1, block_q), top), 77,
                       dtype=torch.int32, device=c["q"].device)
    s = torch.full(lists.shape, 77.0, device=lists.device) if scores else None
    got = h3q.h3q_select_blocks(c["q"], c["k"], c["cu_q"], c["cu_k"], top, block_q=block_q, block_k=block_k, causal=causal,
                                first=first, blocks=lists, scores=s)
    assert got is lists
    want, want_scores = bc.selected(c, top, block_q, block_k, causal, first)
    bad = np.argwhere((lists.cpu().numpy() != want).any(-1))
    assert bad.size == 0, f"{what}: lists {bad[:4].tolist()}: {lists[tuple(bad[0])].tolist()} for " \
                          f"{want[tuple(bad[0])].tolist()}"
    if scores:
        # what the kernel allows a score to be off, 64 * 2^-24 of sum|mean q| max|mean k|: at most that of the largest values
        size = 0.0
        if min(c["q"].shape[0], c["k"].shape[0]) > 0:
            size = float(c["q"].float().abs().amax(0).sum(-1).max()) * float(c["k"].float().abs().amax())
        got = s.cpu().double().numpy()
        empty = want == -1
        assert (got[empty] == -np.inf).all() and np.abs(got[~empty] - want_scores[~empty]).max(initial=0) <= 2.0 ** -18 * size
    return lists


CASES = [  # (queries, keys) of the sequences, query heads, key heads, dim, block_q, block_k, top
    ([(1, 1)], 1, 1, 128, 64, 64, 3),
    ([(1, 1000), (1, 77), (1, 64), (1, 65)], 8, 2, 128, 64, 64, 5),
    ([(300, 1000)], 2, 2, 128, 128, 128, 4),
    ([(300, 3000)], 2, 2, 64, 128, 64, 12),
    ([(600, 5000)], 3, 1, 128, 256, 64, 33),
    ([(600, 5000)], 2, 2, 64, 64, 256, 6),
    ([(500, 500), (0, 70), (130, 0), (257, 1257)], 8, 2, 128, 64, 64, 5),
    ([(300, 100), (129, 128)], 3, 3, 64, 128, 64, 4),
    ([(n, n + 37) for n in (1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257)], 4, 2, 64, 64, 64, 4),
    ([(2000, 20_000)], 2, 1, 128, 128, 64, 64),                 # more key blocks than a tile of scores
    ([(100, 90_000)], 2, 2, 64, 64, 64, 100),                   # more than 16 query blocks' scores have room for
    ([(5, 40)] * 70, 2, 2, 128, 64, 64, 4),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("causal, first", [(False, 0), (False, 2), (True, 0), (True, 1)])
def test_against_the_definition(dev, case, causal, first):
    seqs, heads, kv_heads, dim, block_q, block_k, top = CASES[case]
    top = max(top, first + -(-block_q // block_k) + 1) if causal else top
    c = bc.sequences(dev, seqs, heads, kv_heads, dim, seed=case, packed=case % 2 == 1)
    _check(c, top, block_q, block_k, causal, first, f"case {case}", scores=case % 3 != 0)


def test_ties_go_to_the_lowest(dev):
    """Blocks with the same keys (in another order too), blocks of zeros, and queries of zero."""
    c = bc.sequences(dev, [(200, 64 * 40 + 10)], 2, 2, 128, seed=20)
    k = c["k"]
    for j in range(1, 40):
        src = k[(j % 5) * 64:(j % 5 + 1) * 64]
        k[j * 64:(j + 1) * 64] = src[torch.randperm(64, device=dev)] if j % 2 else src
    _check(c, 12, 64, 64, False, 0)
    _check(c, 12, 64, 64, True, 1)
    k[64 * 10:64 * 30] = 0
    _check(c, 17, 64, 64, False, 0)
    c["q"][64:] = 0
    _check(c, 17, 64, 64, False, 0)
    k[:] = 1.0
    _check(c, 7, 64, 64, False, 3)


def test_scores_that_fp32_cannot_tell_apart(dev):
    """Blocks that differ by little beside a large common part, and sums whose large parts cancel."""
    c = bc.sequences(dev, [(300, 64 * 60)], 2, 2, 128, seed=21, tail=0)
    noise = c["k"].float()
    base = torch.randn((1, 2, 128), device=dev) * 64
    c["k"][:] = (base + (noise * 0.01)).bfloat16()       # most of the noise is rounded away: many equal sums
    _check(c, 20, 64, 64, False, 0)
    c["k"][:] = noise.bfloat16() * 2.0 ** -10
    c["k"][0::2] += 1024.0                               # cancels within each block, up to the noise's rounding
    c["k"][1::2] -= 1024.0
    c["q"][:, :, 64:] *= 2.0 ** -12
    _check(c, 20, 64, 64, False, 0)
    c["k"][:] = (noise * 2.0 ** -60).bfloat16()          # products below fp32's smallest
    c["q"][:] = (c["q"].float() * 2.0 ** -80).bfloat16()
    _check(c, 20, 64, 64, False, 0, scores=False)


def test_numbers_that_are_none(dev):
    """Blocks of infinities and of no numbers: the latter are chosen last."""
    c = bc.sequences(dev, [(64, 64 * 20)], 1, 1, 64, seed=22, tail=0)
    c["k"][64 * 3] = float("nan")
    c["k"][64 * 7:64 * 8] = float("nan")
    for top in (5, 18, 19, 20):
        _check(c, top, 64, 64, False, 0, f"top {top}", scores=False)
    c["q"][5, 0, 0] = float("nan")
    _check(c, 6, 64, 64, False, 0, scores=False)


@pytest.mark.parametrize("dim", [64, 128])
def test_scores_are_as_near_as_the_choice_takes_them(dev, dim):
    """Large products that cancel beside small ones: each score within 176 * 2^-24 of |q| |k|, and the two roundings of
    what is stored."""
    c = bc.sequences(dev, [(64 * 20, 64 * 200)], 1, 1, dim, seed=31, tail=0)
    g = torch.Generator(device=dev)
    g.manual_seed(31)
    for name in "qk":
        size = torch.randint(-9, 10, (1, 1, dim // 2), generator=g, device=dev).float().exp2()
        c[name][:] = (c[name].float() * size.repeat_interleave(2, 2)).bfloat16()
    c["q"][:, :, 1::2] = c["q"][:, :, 0::2]
    c["k"][:, :, 1::2] = -c["k"][:, :, 0::2]
    c["k"][3::7, :, 1::2] *= 0.99                         # the rest of some rows' cancellation
    s = torch.empty((1, 20 + 1, 200), device=dev)
    h3q.h3q_select_blocks(c["q"], c["k"], c["cu_q"], c["cu_k"], 200, block_q=64, block_k=64, scores=s)
    q = c["q"].double().view(20, 64, dim).mean(1)
    k = c["k"].double().view(200, 64, dim).mean(1)
    off = (s[0, :20].double() - q @ k.T).abs()
    assert bool((off <= 2.0 ** -24 * (176 * q.norm(dim=1)[:, None] * k.norm(dim=1) + 2 * (q @ k.T).abs())).all())


@pytest.mark.parametrize("blocks", [40, 1500])   # scores kept in registers, formed again
def test_scores_that_are_infinite(dev, blocks):
    c = bc.sequences(dev, [(64, 64 * blocks)], 1, 1, 64, seed=29, tail=0)
    c["q"][:, :, 0] = 1.0                                 # (the mean of ones: the infinities' sign is the score's)
    c["k"][64 * 3 + 5, 0, 0], c["k"][64 * 30, 0, 0] = float("inf"), float("-inf")
    c["k"][64 * 9, 0, 0], c["k"][64 * 9 + 1, 0, 0] = float("inf"), float("-inf")
    s = torch.empty((1, 1 + 1, blocks), device=dev)
    lists = h3q.h3q_select_blocks(c["q"], c["k"], c["cu_q"], c["cu_k"], blocks, block_q=64, block_k=64, scores=s)
    want, want_scores = bc.selected(c, blocks, 64, 64, False, 0)
    assert (lists.cpu().numpy() == want).all()
    got = s.cpu().numpy()
    assert got[0, 0, 3] == np.inf and got[0, 0, 30] == -np.inf and np.isnan(got[0, 0, 9])
    rest = np.isfinite(want_scores[0, 0])
    assert rest.sum() == blocks - 3 and np.isfinite(got[0, 0][rest]).all()
    top = h3q.h3q_select_blocks(c["q"], c["k"], c["cu_q"], c["cu_k"], 5, block_q=64, block_k=64)
    assert 3 in top[0, 0].tolist() and 30 not in top[0, 0].tolist() and 9 not in top[0, 0].tolist()


def test_no_sequences_and_no_rows(dev):
    for seqs in ([], [(0, 0)], [(0, 100), (0, 0)]):
        c = bc.sequences(dev, seqs, 2, 1, 64, seed=23, tail=200)
        assert bool((_check(c, 3, 64, 64, True, 0) == -1).all())
    c = bc.sequences(dev, [(0, 100)], 2, 1, 64, seed=23, tail=0)
    assert bool((_check(c, 3, 64, 64, True, 0) == -1).all())


def test_rows_of_a_workspace_are_its_own(dev):
    """A workspace of any contents; the same lists from a graph that is replayed with other rows."""
    c = bc.sequences(dev, [(700, 3000), (200, 900)], 4, 2, 128, seed=24)
    nbytes = h3q.select_blocks_workspace_bytes(c["q"].shape[0], c["k"].shape[0], 2, 2, 128, 64, 64)
    ws = torch.full((nbytes,), 255, dtype=torch.uint8, device=dev)
    lists = torch.empty((2, h3q.block_rows(c["q"].shape[0], 2, 64), 9), dtype=torch.int32, device=dev)

    def call():
        h3q.h3q_select_blocks(c["q"], c["k"], c["cu_q"], c["cu_k"], 9, block_q=64, block_k=64, causal=True, first=1,
                              blocks=lists, workspace=ws)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (25, 26):
        other = bc.sequences(dev, [(500 + seed, 2000), (400 - seed, 1900)], 4, 2, 128, seed=seed)
        for name in c:
            c[name].copy_(other[name])
        ws.fill_(seed)
        graph.replay()
        want, _ = bc.selected(c, 9, 64, 64, True, 1)
        assert (lists.cpu().numpy() == want).all()


def test_many_sequences_give_the_same_lists(dev):
    """A sequence of its own, and behind 40 empty ones."""
    c = bc.sequences(dev, [(900, 3000)], 4, 2, 128, seed=32)
    want = _check(c, 9, 64, 64, True, 1)
    many = dict(c, cu_q=cc.ints([0] * 41 + [900], dev), cu_k=cc.ints([0] * 41 + [3000], dev))
    assert torch.equal(_check(many, 9, 64, 64, True, 1)[:, 40:], want)


def test_long_keys_past_32_bits(dev):
    """Keys whose place passes 2^31 elements."""
    heads, keys = 64, 300_000
    g = torch.Generator(device=dev)
    g.manual_seed(34)
    k = torch.empty((keys, heads, 128), dtype=torch.bfloat16, device=dev)
    for part in k.split(keys // 10):
        part.normal_(generator=g)
    q = torch.randn((100, heads, 128), generator=g, device=dev).bfloat16()
    got = h3q.h3q_select_blocks(q, k, cc.ints([0, 100], dev), cc.ints([0, keys], dev), 20)
    for head in (0, heads - 1):
        c = {"q": q[:, head:head + 1], "k": k[:, head:head + 1], "cu_q": cc.ints([0, 100], dev), "cu_k": cc.ints([0, keys], dev)}
        want, _ = bc.selected(c, 20, 128, 128, False, 0)
        assert (got[head].cpu().numpy() == want[0]).all()


def test_wrong_offsets_touch_nothing_outside(dev):
    c = bc.sequences(dev, [(200, 300), (200, 300)], 2, 2, 128, seed=27, tail=0)
    for cu_q, cu_k in (([0, 200, 10_000], [0, 300, 20_000]), ([0, 200, -5], [0, 300, -7]), ([5, 3, 1], [9, 4, 2]),
                       ([-(1 << 31), 7, (1 << 31) - 1], [-(1 << 31), 7, (1 << 31) - 1])):
        h3q.h3q_select_blocks(c["q"], c["k"], cc.ints(cu_q, dev), cc.ints(cu_k, dev), 5, block_k=64, causal=True)
        torch.cuda.synchronize()
