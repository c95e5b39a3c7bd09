"""GPU: block selection with as many lists as large calls have: many query blocks a CTA, of one sequence or several, in
both instances of the kernel, scores kept in registers and not, rows that do not fit beside each other.  The lists
equal those of scores in 64 bits, and each score is within what the header promises."""
import pytest
import torch

import block_cases as bc
import nvfp4_activation_quantize_gb300 as h3q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


def definition(c, top, block_q, block_k, causal, first):
    """The lists [kv_heads, rows, top] of the definition in 64 bits, their scores, and what each score may be off by."""
    kv_heads, dev = c["k"].shape[1], c["q"].device
    group = c["q"].shape[1] // kv_heads
    cu_q, cu_k = c["cu_q"].tolist(), c["cu_k"].tolist()
    rows = c["q"].shape[0] // block_q + len(cu_q) - 1
    lists = torch.full((kv_heads, rows, top), -1, dtype=torch.int64, device=dev)
    scores = torch.full(lists.shape, -torch.inf, dtype=torch.float64, device=dev)
    off = torch.zeros_like(scores)
    for b in range(len(cu_q) - 1):
        n, keys = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        if n == 0 or keys == 0:
            continue

        def means(x, size):   # [kv_heads, blocks, dim]
            return torch.stack([p.double().unflatten(1, (kv_heads, -1)).mean((0, 2)) for p in x.split(size)], 1)

        q, k = means(c["q"][cu_q[b]:cu_q[b + 1]], block_q), means(c["k"][cu_k[b]:cu_k[b + 1]], block_k)
        score = q @ k.transpose(1, 2)
        nq, nk = score.shape[1:]
        i, j = torch.arange(nq, device=dev)[:, None], torch.arange(nk, device=dev)[None]
        begin = keys - n + i * block_q                                     # position of the block's first query
        end = (begin + (n - i * block_q).clamp(max=block_q)).clamp(max=keys)   # one past its last
        there = j * block_k < end if causal else torch.ones((nq, nk), dtype=torch.bool, device=dev)
        always = (j < first) | (((j + 1) * block_k).clamp(max=keys) > begin) if causal else (j < first).expand(nq, nk)
        rank = score.masked_fill(always, torch.inf).masked_fill(~there, -torch.inf)
        count = there.sum(1).clamp(max=top)
        best = rank.sort(dim=2, descending=True, stable=True).indices      # (of equal ones the lowest numbers first)
        place = torch.arange(nk, device=dev)[None]
        best = best.masked_fill(place >= count[:, None], nk).sort(dim=2).values[:, :, :top]
        if best.shape[2] < top:
            best = torch.nn.functional.pad(best, (0, top - best.shape[2]), value=nk)
        at = slice(cu_q[b] // block_q + b, cu_q[b] // block_q + b + nq)
        none = best == nk
        mine = score.gather(2, best.clamp(max=nk - 1))
        lists[:, at] = best.masked_fill(none, -1)
        scores[:, at] = mine.masked_fill(none, -torch.inf)
        # 176 * 2^-24 of |q| |k| and the roundings of what is stored
        size = q.norm(dim=2)[:, :, None] * k.norm(dim=2).gather(1, best.clamp(max=nk - 1).flatten(1)).view(best.shape)
        off[:, at] = 2.0 ** -24 * (176 * size + 4 * mine.abs())
    assert group * kv_heads == c["q"].shape[1]
    return lists, scores, off


def check(c, top, block_q, block_k, causal, first):
    want, want_scores, off = definition(c, top, block_q, block_k, causal, first)
    scores = torch.full(want.shape, 77.0, device=want.device)
    lists = h3q.h3q_select_blocks(c["q"], c["k"], c["cu_q"], c["cu_k"], top, block_q=block_q, block_k=block_k, causal=causal,
                                  first=first, scores=scores)
    bad = (lists != want).any(2).nonzero()
    assert bad.shape[0] == 0, f"{bad.shape[0]} lists, the first {bad[0].tolist()}: {lists[tuple(bad[0])].tolist()} for " \
                              f"{want[tuple(bad[0])].tolist()}"
    none = want == -1
    assert bool((scores[none] == -torch.inf).all())
    assert bool(((scores.double() - want_scores).abs() <= off)[~none].all())
    again = h3q.h3q_select_blocks(c["q"], c["k"], c["cu_q"], c["cu_k"], top, block_q=block_q, block_k=block_k, causal=causal,
                                  first=first)
    assert torch.equal(lists, again)


SHORT = [(37 + 53 * i % 700, 41 + 97 * i % 900) for i in range(40)]
CASES = [  # (queries, keys) of the sequences, query heads, key heads, dim, block_q, block_k, top
    (SHORT, 32, 32, 64, 64, 64, 6),                                       # several sequences in a CTA
    ([(a, a + b) for a, b in SHORT] + [(0, 50), (300, 0)], 32, 16, 128, 64, 64, 9),
    ([(14_000, 14_000)], 32, 32, 128, 64, 64, 24),                        # one sequence, 16 query blocks a CTA
    ([(13_777, 20_011)], 64, 32, 64, 64, 128, 16),                        # a group of two
    ([(6000, 40_000)] + [(100, 100)] * 60, 32, 32, 64, 64, 64, 20),       # 625 key blocks where 512 are in registers
    ([(9000, 1000 * 64 - 9)], 20, 20, 64, 64, 64, 12),                    # 15 rows of 1,000 beside each other, one after
    ([(9001, 1090 * 64 + 3)], 20, 20, 64, 64, 64, 40),                    # more than registers hold, in 14 and 2
    ([(9001, 3000 * 64 + 3)], 20, 20, 64, 64, 64, 40),                    # 5 beside each other
    ([(20_000, 30_000), (900, 40_000)], 48, 12, 128, 128, 64, 33),        # 469 and 625 key blocks
    ([(40_000, 50_000)], 16, 16, 64, 256, 128, 300),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("causal, first", [(False, 0), (True, 2)])
def test_against_the_definition(dev, case, causal, first):
    seqs, heads, kv_heads, dim, block_q, block_k, top = CASES[case]
    check(bc.sequences(dev, seqs, heads, kv_heads, dim, seed=case, packed=case % 2 == 1), top, block_q, block_k, causal, first)


@pytest.mark.parametrize("blocks", [219, 1090])
def test_equal_blocks_go_to_the_lowest(dev, blocks):
    """Seven blocks and their copies, of which the lowest are kept, in CTAs of many query blocks."""
    c = bc.sequences(dev, [(14_000, 64 * blocks)], 32, 32, 64, seed=40, tail=0)
    for j in range(7, blocks):
        c["k"][64 * j:64 * (j + 1)] = c["k"][64 * (j % 7):64 * (j % 7 + 1)]
    lists = h3q.h3q_select_blocks(c["q"], c["k"], c["cu_q"], c["cu_k"], 40, block_q=64, block_k=64)
    q, k = (torch.stack([x.double().sum(0) for x in t.split(64)], 1) for t in (c["q"], c["k"][:7 * 64]))
    order = (q @ k.transpose(1, 2)).sort(dim=2, descending=True).indices.cpu()
    for head in range(32):
        for row in range(0, q.shape[1], 3):
            ranked = [j for p in order[head, row].tolist() for j in range(p, blocks, 7)][:40]
            assert lists[head, row].tolist() == sorted(ranked)
