"""GPU: rows quantized into the paged NVFP4 cache, and read back, byte for byte against the oracle's
quantize and the format's definition: every page size and head size, strided rows, sequences of no
rows, rows of no sequence, positions and pages that do not exist, and lists changed between the
replays of a graph."""
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


def _rows(dev, rows, heads, dim, seed, packed=False):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    x = torch.randn((rows, (3 if packed else 1) * heads * dim), generator=g, device=dev) * 2
    x[::3, :16] = 0
    x[1::5, 3] = 1e3
    x = x.bfloat16()
    return (x[:, heads * dim:2 * heads * dim] if packed else x).unflatten(1, (heads, dim))


def _check_write(cache, before, k, v, gs, places):
    for t, x in ((0, k), (1, v)):
        codes, scales = cc.written(before, x, gs[t], t, places)
        assert np.array_equal(cache[2 * t].cpu().numpy(), codes), f"codes of {'kv'[t]}"
        assert np.array_equal(cache[2 * t + 1].cpu().numpy(), scales), f"scales of {'kv'[t]}"


def _check_read(cache, outs, before, gs, places, owned):
    for t in (0, 1):
        values = cc.values32(cache[2 * t].cpu().numpy(), cache[2 * t + 1].cpu().numpy(), gs[t])
        want = before[t].clone().cpu()
        want[owned] = 0
        for r, page, at in places:
            want[r] = torch.from_numpy(values[page, :, at]).bfloat16()
        assert np.array_equal(cc.bits(outs[t]), cc.bits(want)), f"{'kv'[t]} read back"


CASES = [  # (new rows, positions with them) of each sequence, kv heads, dim, page size
    ([(1, 1)], 1, 64, 16),
    ([(1, 17), (1, 16), (1, 1), (1, 33)], 2, 128, 16),
    ([(5, 5), (0, 40), (37, 100), (0, 0), (64, 64)], 3, 128, 32),
    ([(130, 200), (1, 129)], 8, 64, 128),
    ([(9, 70)], 5, 256, 64),
    ([(700, 700), (300, 1001), (2, 65)], 7, 128, 64),
    ([(1, 10 + 7 * i) for i in range(70)], 4, 128, 16),
    ([(2200, 2300)], 20, 128, 64),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("packed", [False, True])
def test_write_and_read(dev, case, packed):
    seqs, heads, dim, page = CASES[case]
    new, length = [a for a, _ in seqs], [b for _, b in seqs]
    rows = sum(new) + 3  # the last three belong to no sequence
    table, pages = cc.paged(dev, length, page, case)
    cu, kv_len = cc.ints(cc.offsets(new).tolist(), dev), cc.ints(length, dev)
    k, v = (_rows(dev, rows, heads, dim, case + s, packed) for s in (0, 50))
    gs = (448.0 / 3, 77.7)
    kg, vg = (torch.tensor([g], device=dev) for g in gs)
    cache = cc.random_cache(dev, pages, heads, page, dim, case)
    before = tuple(t.clone() for t in cache)
    places, owned = cc.row_places(cu, kv_len, table, page, pages, rows)
    assert len(places) == sum(new)
    h3q.h3q_kv_cache_write_nvfp4(k, v, cache, cu, kv_len, table, kg, vg)
    _check_write(cache, before, k, v, gs, places)
    outs = [torch.full((rows, heads, dim), 7.5, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    empty = [t.clone() for t in outs]
    h3q.h3q_kv_cache_read_nvfp4(cache, cu, kv_len, table, kg, vg, outs=outs)
    _check_read(cache, outs, empty, gs, places, owned)


def test_places_that_do_not_exist(dev):
    """Page numbers outside the cache, lengths shorter than the new rows, longer than the table."""
    page, heads, dim, pages = 16, 2, 128, 6
    new, length = [20, 30, 8, 12], [40, 10, 200, 12]
    table = cc.ints([[0, -1, 6, 3], [1, 2, 2, 2], [4, 4, 4, 4], [2 ** 31 - 1, 5, 5, 5]], dev)
    cu, kv_len = cc.ints([2, 22, 52, 60, 72], dev), cc.ints(length, dev)  # rows 0, 1 and 72.. are no sequence's
    rows = 75
    k, v = (_rows(dev, rows, heads, dim, s) for s in (1, 2))
    cache = cc.random_cache(dev, pages, heads, page, dim, 3)
    before = tuple(t.clone() for t in cache)
    places, owned = cc.row_places(cu, kv_len, table, page, pages, rows)
    assert 0 < len(places) < sum(new)
    one = torch.ones(1, device=dev)
    h3q.h3q_kv_cache_write_nvfp4(k, v, cache, cu, kv_len, table, one, one)
    _check_write(cache, before, k, v, (1.0, 1.0), places)
    outs = [torch.full((rows, heads, dim), -3.0, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    empty = [t.clone() for t in outs]
    h3q.h3q_kv_cache_read_nvfp4(cache, cu, kv_len, table, one, one, outs=outs)
    _check_read(cache, outs, empty, (1.0, 1.0), places, owned)


def test_every_code_and_scale_reads_back(dev):
    """All 16 codes under all 128 scale bytes, with scales whose quotients need rounding."""
    page, dim = 128, 64
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).repeat(16, 1)
    kc = codes.flatten()[:128 * 32].view(1, 1, page, dim // 2).to(dev)
    ks = torch.arange(128, dtype=torch.int32).to(torch.uint8)[:, None].repeat(1, 4).view(1, 1, page, 4).to(dev)
    cache = (kc, ks, kc.flip(-1).contiguous(), ks.flip(2).contiguous())
    lists = cc.ints([0, page], dev), cc.ints([page], dev), cc.ints([[0]], dev)
    places, owned = cc.row_places(*lists, page, 1, page)
    for gs in ((3.0, 448.0 * 6 / 7), (1e-30, 1e30), (1.0, 0.7)):
        outs = h3q.h3q_kv_cache_read_nvfp4(cache, *lists, *(torch.tensor([g], device=dev) for g in gs), rows=page)
        _check_read(cache, outs, [torch.zeros_like(o) for o in outs], gs, places, owned)


def test_graph_replay_follows_the_lists(dev):
    page, heads, dim = 32, 2, 128
    table, pages = cc.paged(dev, [100, 100], page, 9)
    cu, kv_len = cc.ints([0, 1, 2], dev), cc.ints([1, 50], dev)
    k, v = (_rows(dev, 2, heads, dim, s) for s in (4, 5))
    one = torch.ones(1, device=dev)
    cache = cc.random_cache(dev, pages, heads, page, dim, 3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h3q.h3q_kv_cache_write_nvfp4(k, v, cache, cu, kv_len, table, one, one)
    for step in range(3):
        before = tuple(t.clone() for t in cache)
        kv_len.copy_(cc.ints([10 + 30 * step, 51 + step], dev))
        k.copy_(_rows(dev, 2, heads, dim, 20 + step))
        graph.replay()
        places, _ = cc.row_places(cu, kv_len, table, page, pages, 2)
        _check_write(cache, before, k, v, (1.0, 1.0), places)


def test_cache_past_2_31_bytes_of_codes(dev):
    """A cache whose last pages lie past 2^32 bytes of codes, one row written at its end."""
    page, heads, dim = 128, 8, 256
    pages = (1 << 32) // (page * heads * dim // 2) + 3
    cache = h3q.kv_cache_nvfp4(pages, heads, page, dim, dev)
    table, cu, kv_len = cc.ints([[pages - 1]], dev), cc.ints([0, 1], dev), cc.ints([page], dev)
    k, v = (_rows(dev, 1, heads, dim, s) for s in (1, 2))
    one = torch.ones(1, device=dev)
    h3q.h3q_kv_cache_write_nvfp4(k, v, cache, cu, kv_len, table, one, one)
    last = tuple(t[-1:].clone() for t in cache)
    zero = tuple(torch.zeros_like(t) for t in last)
    _check_write(last, zero, k, v, (1.0, 1.0), [(0, 0, page - 1)])
    assert all(int(t[:-1].count_nonzero()) == 0 for t in cache[1::2])
    outs = h3q.h3q_kv_cache_read_nvfp4(cache, cu, kv_len, table, one, one, rows=1)
    _check_read(last, outs, [torch.zeros_like(o) for o in outs], (1.0, 1.0), [(0, 0, page - 1)], [0])
    del cache
    torch.cuda.empty_cache()
