"""GPU: attention over listed blocks of keys, against the formula in 64 bits: head sizes and groups, sizes of blocks,
lengths around the tiles, lists of nothing and of everything, lists with numbers of no block, keys that are
masked or past a sequence's end and hold no numbers, graphs and streams, and the same bits every time."""
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


def _run(c, lists, block_q, block_k, causal, **kw):
    rows, heads, dim = c["q"].shape
    out = torch.full((rows, heads, dim), 5.0, dtype=torch.bfloat16, device=c["q"].device)
    lse = torch.full((heads, rows), 6.0, dtype=torch.float32, device=c["q"].device)
    assert h3q.h3q_attention_blocks(c["q"], c["k"], c["v"], c["cu_q"], c["cu_k"], lists, block_q=block_q, block_k=block_k,
                                    causal=causal, out=out, lse=lse, **kw) is out
    assert h3q.h3q_kernel_error_flag() == 0
    end = int(c["cu_q"][-1])
    assert bool((out[end:] == 5.0).all()) and bool((lse[:, end:] == 6.0).all()), "rows of no sequence"
    return out, lse


CASES = [  # (queries, keys) of the sequences, query heads, key heads, dim, block_q, block_k, top
    ([(1, 1)], 1, 1, 128, 64, 64, 1),
    ([(1, 1000), (1, 77), (1, 64)], 8, 2, 128, 64, 64, 5),            # single tokens
    ([(128, 1000)], 1, 1, 128, 128, 128, 3),                          # a block is a tile
    ([(300, 1000)], 2, 2, 128, 128, 128, 4),                          # three blocks: two a pair, one alone
    ([(300, 1000)], 2, 2, 128, 128, 64, 7),                           # an odd number of runs
    ([(300, 1000)], 2, 2, 64, 128, 256, 2),
    ([(600, 900)], 2, 2, 128, 256, 128, 4),                           # a block is two tiles with one list
    ([(600, 900)], 2, 2, 64, 256, 64, 9),
    ([(64, 500), (65, 500), (63, 200)], 1, 1, 64, 64, 64, 3),         # half-filled tiles
    ([(200, 700), (0, 70), (130, 0), (257, 257)], 8, 2, 128, 64, 64, 6),   # 4 heads: two tiles a block
    ([(500, 800)], 8, 2, 128, 128, 128, 3),                           # 4 heads: four tiles a block
    ([(300, 100), (129, 128)], 3, 3, 64, 128, 64, 2),                 # queries that see nothing
    ([(200, 200), (90, 1500)], 14, 2, 128, 64, 128, 3),               # 7 heads: 18 tokens a tile, four a block
    ([(77, 177), (150, 151)], 40, 8, 64, 128, 64, 3),                 # 5 heads
    ([(33, 500)], 48, 1, 128, 64, 64, 4),
    ([(70, 200), (40, 41)], 128, 1, 64, 64, 64, 2),
    ([(2, 70)], 131, 1, 64, 64, 64, 2),                               # a prime group: one head a tile
    ([(n, n + 37) for n in (1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257)], 2, 2, 128, 128, 64, 3),
    ([(n, n + 37) for n in (1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257)], 4, 2, 64, 64, 128, 2),
    ([(700, 5000)], 4, 2, 128, 128, 64, 70),                          # lists of more than 64 entries
    ([(1500, 2000)], 3, 3, 128, 128, 128, 16),                        # every block
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("junk", [False, True])
def test_against_the_formula(dev, case, causal, junk):
    seqs, heads, kv_heads, dim, block_q, block_k, top = CASES[case]
    c = bc.sequences(dev, seqs, heads, kv_heads, dim, seed=case, packed=case % 2 == 1)
    lists = bc.random_lists(c, kv_heads, block_q, block_k, top, case, junk)
    out, lse = _run(c, lists, block_q, block_k, causal)
    bc.check_blocks(c, lists, block_q, block_k, causal, out, lse, what=f"case {case}")
    again = _run(c, lists, block_q, block_k, causal)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1]), "other bits the second time"


@pytest.mark.parametrize("block_q, heads", [(64, 8), (128, 2), (256, 2)])
def test_all_blocks_are_dense_attention(dev, block_q, heads):
    """Lists of every block: the answer of h3q_attention_varlen, within what two roundings differ by."""
    c = bc.sequences(dev, [(700, 1000), (333, 333)], heads, 2, 128, seed=3, tail=0)
    rows = h3q.block_rows(1033, 2, block_q)
    lists = torch.arange(16, device=dev, dtype=torch.int32).repeat(2, rows, 1).contiguous()
    for causal in (False, True):
        out, lse = _run(c, lists, block_q, 64, causal)
        dense = torch.empty_like(lse)
        want = h3q.h3q_attention_varlen(c["q"], c["k"], c["v"], c["cu_q"], c["cu_k"], causal=causal, lse=dense)
        # the same tiles of keys in the same order, weights against references that follow the same rule
        assert torch.equal(out, want) and torch.equal(lse, dense)


def test_empty_lists(dev):
    c = bc.sequences(dev, [(300, 500), (5, 70)], 2, 2, 128, seed=4)
    rows = h3q.block_rows(c["q"].shape[0], 2, 128)
    for fill in (-1, 1 << 30):
        lists = torch.full((2, rows, 33), fill, dtype=torch.int32, device=dev)
        out, lse = _run(c, lists, 128, 64, False)
        assert bool((out[:305] == 0).all()) and bool((lse[:, :305] == -float("inf")).all())
    lists[0, :, 32] = 0   # one entry, the last, of one head
    out, lse = _run(c, lists, 128, 64, False)
    bc.check_blocks(c, lists, 128, 64, False, out, lse)


def test_one_tile_of_a_pair_alone(dev):
    """Neighbouring query blocks with lists of very different lengths."""
    c = bc.sequences(dev, [(512, 3000)], 1, 1, 128, seed=5)
    rows = h3q.block_rows(c["q"].shape[0], 1, 128)
    for lengths in ((0, 40, 40, 0), (1, 40, 40, 1), (40, 39, 2, 3), (3, 2, 17, 40)):
        lists = torch.full((1, rows, 40), -1, dtype=torch.int32, device=dev)
        for r, n in enumerate(lengths):
            lists[0, r, :n] = torch.arange(n, dtype=torch.int32, device=dev)
        for causal in (False, True):
            out, lse = _run(c, lists, 128, 64, causal)
            bc.check_blocks(c, lists, 128, 64, causal, out, lse, what=str(lengths))


@pytest.mark.parametrize("scale", [1.0, 0.004, 3.0])
def test_scale(dev, scale):
    """Sharp softmaxes move the reference maximum often, flat ones never."""
    c = bc.sequences(dev, [(300, 900)], 2, 2, 128, seed=6)
    lists = bc.random_lists(c, 2, 128, 64, 8, 6)
    out, lse = _run(c, lists, 128, 64, True, scale=scale)
    bc.check_blocks(c, lists, 128, 64, True, out, lse, scale=scale)


def test_maxima_that_grow(dev):
    c = bc.sequences(dev, [(300, 1000)], 2, 2, 128, seed=7)
    c["q"][:, :, 0] = 4.0
    c["k"][:1000, :, 0] = torch.linspace(0, 30, 1000, device=dev)[:, None].bfloat16()
    for block_q in (128, 256):
        lists = bc.random_lists(c, 2, block_q, 64, 12, 7)
        out, lse = _run(c, lists, block_q, 64, False)
        bc.check_blocks(c, lists, block_q, 64, False, out, lse)


@pytest.mark.parametrize("block_q, heads, dim", [(128, 1, 128), (256, 1, 64), (64, 4, 128)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_values_that_are_no_numbers(dev, block_q, heads, dim, value):
    """Past the end of a sequence (the next one's) and at keys to come they reach nobody; at keys that
    are seen they reach exactly the rows that see them."""
    c = bc.sequences(dev, [(300, 300), (200, 200)], heads, 1, dim, seed=8)
    clean = {k: t.clone() for k, t in c.items()}
    rows = h3q.block_rows(c["q"].shape[0], 2, block_q)
    lists = torch.arange(5, device=dev, dtype=torch.int32).repeat(1, rows, 1).contiguous()
    at = (299, 150, 300 + 199, 300 + 64)
    for p in at:
        c["v"][p, 0, 3] = value
    c["k"][500:] = value
    c["v"][500:] = value
    out, _ = _run(c, lists, block_q, 64, True)
    want, _ = _run(clean, lists, block_q, 64, True)
    hit = torch.zeros(503, dtype=torch.bool, device=dev)
    for first, end, start in ((150, 300, 0), (300 + 64, 500, 300)):
        hit[first:end] = True
    same = torch.ones(dim, dtype=torch.bool, device=dev)
    same[3] = False
    assert torch.equal(out[:500][:, :, same], want[:500][:, :, same])
    assert bool(torch.isfinite(out[:500, :, 3][~hit[:500]]).all())
    assert not bool(torch.isfinite(out[:500, :, 3][hit[:500]]).any())
    assert torch.equal(out[:500][~hit[:500]], want[:500][~hit[:500]])


def test_graph_follows_lists(dev):
    """A captured call replayed with other lists, offsets and inputs."""
    c = bc.sequences(dev, [(300, 700), (100, 300)], 4, 2, 128, seed=9)
    lists = bc.random_lists(c, 2, 64, 64, 4, 9)
    out = torch.zeros(c["q"].shape, dtype=torch.bfloat16, device=dev)
    lse = torch.zeros((4, c["q"].shape[0]), device=dev)

    def call():
        h3q.h3q_attention_blocks(c["q"], c["k"], c["v"], c["cu_q"], c["cu_k"], lists, block_q=64, block_k=64, causal=True,
                                 out=out, lse=lse)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (10, 11):
        other = bc.sequences(dev, [(50 + seed, 400), (350 - seed, 600)], 4, 2, 128, seed=seed)
        for name in c:
            c[name].copy_(other[name])
        lists.copy_(bc.random_lists(c, 2, 64, 64, 4, seed))
        graph.replay()
        torch.cuda.synchronize()
        bc.check_blocks(c, lists, 64, 64, True, out, lse)


def test_two_streams_at_once(dev):
    cases = [bc.sequences(dev, [(900, 2000)], 4, 4, 128, seed=s) for s in (12, 13)]
    lists = [bc.random_lists(c, 4, 128, 128, 6, s) for s, c in enumerate(cases)]
    want = [_run(c, m, 128, 128, True)[0] for c, m in zip(cases, lists)]
    streams = [torch.cuda.Stream(dev) for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            c = cases[i]
            got[i].append(h3q.h3q_attention_blocks(c["q"], c["k"], c["v"], c["cu_q"], c["cu_k"], lists[i], causal=True,
                                                   stream=s))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(o[:900], want[i][:900]) for o in got[i])


def test_wrong_offsets_touch_nothing_outside(dev):
    """Offsets that fall, are negative or pass the rows: no fault, and sequences that are right stay right."""
    c = bc.sequences(dev, [(200, 300), (200, 300)], 2, 2, 128, seed=14, tail=0)
    lists = bc.random_lists(c, 2, 128, 64, 3, 14)
    want, _ = _run(c, lists, 128, 64, True)
    for cu_q, cu_k in (([0, 200, 10_000], [0, 300, 20_000]), ([0, 200, -5], [0, 300, -7]), ([0, 200, 100], [0, 300, 200])):
        bad = dict(c, cu_q=cc.ints(cu_q, dev), cu_k=cc.ints(cu_k, dev))
        out = torch.zeros_like(want)
        h3q.h3q_attention_blocks(bad["q"], bad["k"], bad["v"], bad["cu_q"], bad["cu_k"], lists, block_k=64, causal=True,
                                 out=out)
        assert h3q.h3q_kernel_error_flag() == 0
        assert torch.equal(out[:200], want[:200])


@pytest.mark.parametrize("heads, kv_heads, dim, block_q", [(8, 8, 128, 128), (8, 8, 64, 64), (6, 6, 128, 256), (16, 4, 128, 64)])
@pytest.mark.parametrize("causal", [False, True])
def test_units_in_halves_give_the_same_bits(dev, heads, kv_heads, dim, block_q, causal):
    """The last units run as two row tiles where there are few sequences, as one beside 32 empty sequences."""
    c = bc.sequences(dev, [(1100, 1500)], heads, kv_heads, dim, seed=33)
    lists = bc.random_lists(c, kv_heads, block_q, 64, 9, 33)
    out, lse = _run(c, lists, block_q, 64, causal)
    many = dict(c, cu_q=cc.ints([0] * 33 + [1100], dev), cu_k=cc.ints([0] * 33 + [1500], dev))
    more = torch.full((kv_heads, lists.shape[1] + 32, 9), -1, dtype=torch.int32, device=dev)
    more[:, 32:] = lists
    again, lse_again = _run(many, more, block_q, 64, causal)
    assert torch.equal(out, again) and torch.equal(lse, lse_again)
    bc.check_blocks(c, lists, block_q, 64, causal, out, lse)


def test_long_keys_past_32_bits(dev):
    """Keys whose place passes 2^31 elements."""
    heads, dim, keys = 8, 128, 2_200_000
    g = torch.Generator(device=dev)
    g.manual_seed(15)
    k = torch.empty((keys, heads, dim), dtype=torch.bfloat16, device=dev)
    k.view(-1, dim)[:] = torch.randn((keys // 100, dim), generator=g, device=dev).bfloat16().repeat(100 * heads, 1)
    c = {"q": torch.randn((2, heads, dim), generator=g, device=dev).bfloat16(), "k": k, "v": k,
         "cu_q": cc.ints([0, 1, 2], dev), "cu_k": cc.ints([0, 100, keys], dev)}
    last = (keys - 100 - 1) // 64
    lists = torch.tensor([0, 5, last - 7, last], device=dev, dtype=torch.int32).repeat(heads, 2, 1).contiguous()
    out, lse = _run(c, lists, 64, 64, True)
    bc.check_blocks(c, lists, 64, 64, True, out, lse)
