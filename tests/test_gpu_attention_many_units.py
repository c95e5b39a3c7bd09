"""GPU: attention over blocks with several units of work a CTA: blocks taken over, what is carried from unit to unit,
halves of units behind whole ones, with a list for each row tile and one for both."""
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


def run(c, lists, block_q, block_k, causal):
    rows, heads, dim = c["q"].shape
    out = torch.full((rows, heads, dim), 5.0, dtype=torch.bfloat16, device=c["q"].device)
    lse = torch.full((heads, rows), 6.0, device=c["q"].device)
    h3q.h3q_attention_blocks(c["q"], c["k"], c["v"], c["cu_q"], c["cu_k"], lists, block_q=block_q, block_k=block_k,
                             causal=causal, out=out, lse=lse)
    assert h3q.h3q_kernel_error_flag() == 0
    end = int(c["cu_q"][-1])
    assert bool((out[end:] == 5.0).all()) and bool((lse[:, end:] == 6.0).all()), "rows of no sequence"
    return out, lse


def units_of(seqs, heads, kv_heads, block_q):
    """Pairs of row tiles of up to 128 rows, tokens x heads of one group, of each sequence and group."""
    group = heads // kv_heads
    per_tile = max((d for d in range(1, min(group, 128) + 1) if group % d == 0), key=lambda d: (128 // d * d, d))
    tokens = min(128 // per_tile, block_q)
    tiles = -(-block_q // tokens)   # of a query block

    def pairs(n):
        if tiles == 1:
            return -(--(-n // block_q) // 2)
        return n // block_q * -(-tiles // 2) + -(--(-(n % block_q) // tokens) // 2)

    return sum(pairs(n) for n, _ in seqs) * (heads // per_tile)


def check(c, lists, block_q, block_k, causal, out, lse, what):
    """As block_cases.check_blocks, all key heads of a query block at once."""
    dev, dim, (heads, kv_heads) = out.device, c["q"].shape[2], (c["q"].shape[1], c["k"].shape[1])
    cu_q, cu_k = c["cu_q"].tolist(), c["cu_k"].tolist()
    group, host, scale = heads // kv_heads, lists.cpu().tolist(), dim ** -0.5
    for r, b, first, last in bc.query_blocks(c, block_q):
        n, keys = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        at, blocks = slice(cu_q[b] + first, cu_q[b] + last), -(-keys // block_k)
        named = torch.zeros((kv_heads, blocks + 1), dtype=torch.bool)
        for h in range(kv_heads):
            named[h, bc.counted(host[h][r], blocks)] = True
        p = torch.arange(keys, device=dev)
        seen = named.to(dev)[:, p // block_k].repeat_interleave(group, 0)[:, None]
        t = torch.arange(first, last, device=dev)[:, None]
        seen = seen & (p <= t + (keys - n)) if causal else seen.expand(-1, last - first, -1)
        q, k, v = (x.double() for x in (c["q"][at], c["k"][cu_k[b]:cu_k[b + 1]], c["v"][cu_k[b]:cu_k[b + 1]]))
        k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
        x = (torch.einsum("nhd,khd->hnk", q, k) * scale).masked_fill(~seen, -torch.inf)
        sizes = torch.einsum("nhd,khd->hnk", q.abs(), k.abs())
        size = float(sizes.max()) * scale * 1.4427 if keys else 0.0
        sums = torch.logsumexp(x, -1) if keys else torch.full(x.shape[:2], -torch.inf, dtype=x.dtype, device=dev)
        w = torch.where(seen, torch.exp(x - sums[..., None].clamp(min=-1e300)), torch.zeros_like(x))
        ref = torch.einsum("hnk,khd->nhd", w, v), sums, torch.einsum("hnk,khd->nhd", w, v.abs()), size
        cc.check_attention(out[at], lse[:, at], ref, int(named.sum(1).max()) * block_k, 2.0 ** -8,
                           f"{what} sequence {b} queries {first}")


RAGGED = [(1 + 131 * i % 701, 1 + 197 * i % 1511) for i in range(24)]
CASES = [  # (queries, keys) of the sequences, query heads, key heads, dim, block_q, block_k, top, units
    (RAGGED, 20, 20, 128, 128, 128, 5, 600),                             # a list for each row tile
    (RAGGED + [(0, 70), (130, 0)], 24, 24, 64, 64, 64, 9, 600),
    (RAGGED, 24, 6, 128, 64, 64, 11, 600),                               # 4 heads: one list for both
    (RAGGED, 14, 14, 128, 256, 64, 13, 600),
    ([(a, a + b) for a, b in RAGGED], 35, 5, 64, 128, 128, 6, 600),      # 7 heads: one a row tile
    ([(1, 1 + 37 * i % 900) for i in range(200)], 16, 4, 128, 64, 64, 7, 600),   # single tokens
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("causal, junk", [(False, True), (True, False)])
def test_against_the_formula(dev, case, causal, junk):
    seqs, heads, kv_heads, dim, block_q, block_k, top, units = CASES[case]
    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    assert units_of(seqs, heads, kv_heads, block_q) >= units >= 3 * sms
    c = bc.sequences(dev, seqs, heads, kv_heads, dim, seed=case, packed=case % 2 == 1)
    lists = bc.random_lists(c, kv_heads, block_q, block_k, top, case, junk)
    lists[:, ::5] = -1   # (units with no keys between the others)
    out, lse = run(c, lists, block_q, block_k, causal)
    check(c, lists, block_q, block_k, causal, out, lse, f"case {case}")
    for _ in range(3):
        again = run(c, lists, block_q, block_k, causal)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1]), "other bits another time"


@pytest.mark.parametrize("pairs, heads, kv_heads, dim, block_q", [(27, 24, 24, 128, 128), (27, 24, 24, 64, 64),
                                                                  (27, 24, 24, 64, 256), (27, 48, 12, 128, 64)])
def test_halves_behind_whole_units(dev, pairs, heads, kv_heads, dim, block_q):
    """Units that fill the GPU more than once, the last turn's as two row tiles; whole behind 33 empty sequences."""
    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    per_tile = heads // kv_heads
    tokens = min(128 // per_tile, block_q)
    groups = heads // per_tile
    while not (pairs * groups > 2 * sms and 0 < 2 * (pairs * groups % sms) <= sms):
        pairs += 1
    rows = 2 * tokens * pairs - 5
    c = bc.sequences(dev, [(rows, rows + 300)], heads, kv_heads, dim, seed=50, tail=0)
    lists = bc.random_lists(c, kv_heads, block_q, 64, 9, 50)
    many = dict(c, cu_q=cc.ints([0] * 33 + [rows], dev), cu_k=cc.ints([0] * 33 + [rows + 300], dev))
    more = torch.full((kv_heads, lists.shape[1] + 32, 9), -1, dtype=torch.int32, device=dev)
    more[:, 32:] = lists
    for causal in (False, True):
        out, lse = run(c, lists, block_q, 64, causal)
        again, lse_again = run(many, more, block_q, 64, causal)
        assert torch.equal(out, again) and torch.equal(lse, lse_again)
    check(c, lists, block_q, 64, True, out, lse, "halves")


def test_large_values_between_ordinary_ones(dev):
    """Units whose values hold infinities, in turn with units that see none of them."""
    c = bc.sequences(dev, [(300, 300), (260, 260)] * 20, 8, 8, 128, seed=51)
    clean = {name: t.clone() for name, t in c.items()}
    at = c["cu_k"].tolist()
    for b in range(0, 40, 2):
        c["v"][at[b] + 170, :, 3] = float("inf")
    lists = torch.arange(5, device=dev, dtype=torch.int32).repeat(8, h3q.block_rows(c["q"].shape[0], 40, 128), 1).contiguous()
    out, lse = run(c, lists, 128, 64, True)
    want, want_lse = run(clean, lists, 128, 64, True)
    hit = torch.zeros(out.shape[0], dtype=torch.bool, device=dev)
    for b in range(0, 40, 2):
        hit[at[b] + 170:at[b + 1]] = True
    assert torch.equal(lse, want_lse) and torch.equal(out[~hit], want[~hit])
    other = torch.arange(128, device=dev) != 3
    assert torch.equal(out[:, :, other], want[:, :, other])
    assert not bool(torch.isfinite(out[hit][:, :, 3]).any())
