"""GPU: attention of new tokens over the paged NVFP4 cache, against the formula in 64 bits on the values that
the cache stands for: head sizes and groups, one token to 64, chains and trees, empty contexts and rows that
see nothing, lengths around tiles and pages, contexts that many CTAs share, strides, pages that do not exist,
graphs, streams, and the same bits every time."""
import numpy as np
import pytest
import torch

import cache_cases as cc
import nvfp4_activation_quantize_gb300 as h3q

pytestmark = pytest.mark.gpu

WEIGHT = 2.0 ** -11  # weights are rounded to fp16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


def _scales(dev, gs):
    return [torch.tensor([g], device=dev) for g in gs]


def _trees(rng, new):
    masks = []
    for n in new:
        mine = []
        for i in range(n):
            parent = int(rng.integers(-1, i)) if i else -1
            mine.append((mine[parent] if parent >= 0 else 0) | 1 << i)
        masks += [m - (1 << 64) if m >= 1 << 63 else m for m in mine]
    return masks


def _case(dev, seqs, heads, kv_heads, dim, page, tree=False, seed=0, packed=False, tail=2, gain=1.0):
    """Inputs for sequences of (new tokens, positions with them)."""
    rng = np.random.default_rng(seed)
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    new, length = [a for a, _ in seqs], [b for _, b in seqs]
    rows = sum(new) + tail
    table, pages = cc.paged(dev, length, page, seed)
    x = torch.randn((rows, (2 if packed else 1) * heads * dim), generator=g, device=dev) * gain
    q = (x.bfloat16()[:, :heads * dim]).unflatten(1, (heads, dim))
    masks = _trees(rng, new) + [0] * tail if tree else None
    return {"q": q, "cache": cc.random_cache(dev, pages, kv_heads, page, dim, seed),
            "cu": cc.ints(cc.offsets(new).tolist(), dev), "len": cc.ints(length, dev), "table": table,
            "gs": (2688.0, 300.0), "scales": _scales(dev, (2688.0, 300.0)), "mask": cc.ints(masks, dev, torch.int64) if tree else None, "page": page,
            "new": new, "most": max(new + [1])}


def _run(c, scale=None, **kw):
    rows, heads, dim = c["q"].shape
    out = torch.full((rows, heads, dim), 5.0, dtype=torch.bfloat16, device=c["q"].device)
    lse = torch.full((heads, rows), 6.0, dtype=torch.float32, device=c["q"].device)
    kg, vg = c["scales"]
    kw.setdefault("max_rows", c["most"])
    got = h3q.h3q_attention_cache_nvfp4(c["q"], c["cache"], c["cu"], c["len"], c["table"], kg, vg, tree_mask=c["mask"],
                                        scale=scale, out=out, lse=lse, **kw)
    assert got is out
    return out, lse


def _check(c, out, lse, scale=None, only=None, what=""):
    dev = c["q"].device
    cu, length = c["cu"].tolist(), c["len"].tolist()
    scale = c["q"].shape[2] ** -0.5 if scale is None else scale
    cap = c["table"].shape[1] * c["page"]
    for b in range(len(length)):
        if only is not None and b not in only:
            continue
        n, keys = cu[b + 1] - cu[b], max(0, min(length[b], cap))
        if n == 0:
            continue
        ctx = length[b] - n
        k, v = cc.cache_values64(c["cache"], c["gs"], c["table"][b], keys, c["page"])
        draft = torch.arange(keys, device=dev)[None] - ctx
        if c["mask"] is None:
            seen = draft <= torch.arange(n, device=dev)[:, None]
        else:
            bits = c["mask"][cu[b]:cu[b + 1], None] >> draft.clamp(0, 63) & 1
            seen = (draft < 0) | ((bits == 1) & (draft < 64))
        ref = cc.attention64(c["q"][cu[b]:cu[b + 1]], k, v, seen, scale)
        cc.check_attention(out[cu[b]:cu[b + 1]], lse[:, cu[b]:cu[b + 1]], ref, keys, WEIGHT, f"{what} sequence {b}")
    assert bool((out[cu[-1]:] == 5.0).all()) and bool((lse[:, cu[-1]:] == 6.0).all()), f"{what}: rows of no sequence"


CASES = [  # sequences, query heads, key heads, dim, page
    ([(1, 1)], 1, 1, 64, 16),
    ([(1, 777)], 8, 2, 64, 16),
    ([(1, n) for n in (1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 500)], 4, 1, 128, 16),
    ([(1, 100), (1, 2000), (1, 3), (1, 640)], 8, 8, 128, 32),
    ([(1, 50 + 61 * i) for i in range(40)], 32, 8, 128, 64),
    ([(1, 300), (1, 70)], 10, 2, 256, 64),
    ([(1, 300), (1, 70)], 64, 2, 256, 16),
    ([(1, 513), (1, 31)], 24, 1, 128, 128),
    ([(1, 513), (1, 31)], 22, 1, 64, 128),
    ([(2, 90), (0, 50), (5, 5), (3, 400), (1, 33)], 14, 2, 128, 64),
    ([(64, 64), (64, 700), (17, 1000)], 8, 2, 128, 64),
    ([(33, 33), (64, 129), (1, 2)], 5, 5, 64, 32),
    ([(7, 200), (16, 16)], 6, 2, 256, 32),
    ([(1, 70000)], 8, 1, 128, 64),
    ([(1, 40000), (1, 1), (3, 30000)], 32, 8, 64, 128),
    ([(9, 9), (16, 800), (12, 129), (1, 5000)], 32, 8, 128, 64),      # 36 to 64 rows a key head
    ([(33, 300), (64, 4000), (2, 2)], 10, 2, 128, 16),                # 320 rows: three row tiles
    ([(40, 20000)], 2, 1, 64, 32),
    ([(1, 700), (1, 128), (1, 129), (1, 255), (1, 257)], 128, 2, 128, 128),   # 64 query heads a key head
    ([(3, 10), (5, 140), (0, 9), (64, 64)], 24, 2, 64, 16),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("tree", [False, True])
def test_against_the_formula(dev, case, tree):
    seqs, heads, kv_heads, dim, page = CASES[case]
    c = _case(dev, seqs, heads, kv_heads, dim, page, tree, seed=case, packed=case % 2 == 1)
    out, lse = _run(c)
    _check(c, out, lse, what=f"case {case}")
    again = _run(c)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1]), "other bits the second time"
    assert h3q.h3q_kernel_error_flag() == 0


def test_written_rows_then_decoded(dev):
    """The calls as they are used: a step's rows written, then attended to, in a growing cache."""
    heads, kv, dim, page, batch = 8, 2, 128, 16, 3
    cache = h3q.kv_cache_nvfp4(40, kv, page, dim, dev)
    table = torch.randperm(40, device=dev)[:36].to(torch.int32).view(batch, 12).contiguous()
    length = cc.ints([0, 0, 0], dev)
    gs = (448.0, 300.0)
    kg, vg = _scales(dev, gs)
    for step, new in enumerate(([100, 1, 40], [1, 1, 1], [5, 0, 2], [1, 1, 1])):
        rows = sum(new)
        g = torch.Generator(device=dev)
        g.manual_seed(step)
        x = torch.randn((rows, (heads + 2 * kv) * dim), generator=g, device=dev).bfloat16().unflatten(1, (-1, dim))
        cu = cc.ints(cc.offsets(new).tolist(), dev)
        length += cu[1:] - cu[:-1]
        h3q.h3q_kv_cache_write_nvfp4(x[:, heads:heads + kv], x[:, heads + kv:], cache, cu, length, table, kg, vg)
        if max(new) > 64:
            continue
        c = {"q": x[:, :heads], "cache": cache, "cu": cu, "len": length, "table": table, "gs": gs, "scales": (kg, vg), "mask": None,
             "page": page, "most": max(new)}
        out, lse = _run(c)
        _check(c, out, lse, what=f"step {step}")


def test_rows_that_see_nothing(dev):
    """No context, and masks that leave out every new token, or all but another one."""
    c = _case(dev, [(4, 4), (2, 50), (3, 0), (2, 1)], 4, 2, 128, 16, tree=True, seed=3)
    c["mask"][:4] = cc.ints([0, 1, 8, 0], dev, torch.int64)
    out, lse = _run(c)
    assert bool((out[0] == 0).all()) and bool((out[3] == 0).all()) and bool((lse[:, 0] == -np.inf).all())
    assert bool((out[6:9] == 0).all()) and bool((lse[:, 6:9] == -np.inf).all())  # a sequence without keys
    _check(c, out, lse, only={0, 1, 3})


def test_query_scales(dev):
    """Rows of very large and very small queries, of zeros, and of values that are no numbers: those rows
    alone have no number to give."""
    c = _case(dev, [(6, 300)], 2, 1, 128, 64, seed=5)
    q = c["q"].clone()
    q[0] *= 1e-30
    q[1] = 0
    q[2, 0] *= 300.0
    q[3, 1, 5] = float("nan")
    q[4, 0, 7] = float("inf")
    q[5, 1, :64] *= 1e-6
    c["q"] = q
    out, lse = _run(c)
    assert bool(torch.isnan(out[3, 1]).all()) and bool(torch.isnan(out[4, 0]).all())
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[3, 1] = bad[4, 0] = True
    c["q"] = q.masked_fill(bad, 0)
    want, want_lse = _run(c)
    assert torch.equal(out[~bad], want[~bad])
    _check(c, want, want_lse)


@pytest.mark.parametrize("scale", [1.0, 0.003, 2.5])
def test_scale(dev, scale):
    c = _case(dev, [(1, 200), (4, 77)], 4, 2, 64, 16, seed=8)
    out, lse = _run(c, scale=scale)
    _check(c, out, lse, scale=scale)


def test_pages_that_do_not_exist(dev):
    """A sequence of bad page numbers, or longer than its table, leaves the others' outputs right."""
    c = _case(dev, [(1, 200), (1, 150), (2, 90), (1, 64)], 8, 2, 128, 16, seed=6)
    pages = c["cache"][0].shape[0]
    c["table"][1, ::2] = cc.ints([pages, -1, 2 ** 31 - 1, -2 ** 31, 1, pages + 5, -3][:c["table"][1, ::2].numel()], dev)
    c["len"][2] = 10 ** 6   # past its table: it has max_pages * page positions
    out, lse = _run(c)
    _check(c, out, lse, only={0, 3})
    assert h3q.h3q_kernel_error_flag() == 0


def test_lists_out_of_order(dev):
    """Lists that decrease or point past the rows: nothing outside the outputs of good sequences is wrong."""
    c = _case(dev, [(1, 60), (1, 70), (1, 80)], 4, 1, 64, 16, seed=7)
    good, _ = _run(c)
    c["cu"] = cc.ints([0, 1, -5, 3], dev)
    out, lse = _run(c)
    assert torch.equal(out[0], good[0])
    c["cu"] = cc.ints([0, 1, 2, 2 ** 31 - 1], dev)
    out, lse = _run(c)
    assert torch.equal(out[:2], good[:2])
    assert h3q.h3q_kernel_error_flag() == 0


def test_graph_replay_follows_the_lists(dev):
    c = _case(dev, [(1, 900), (1, 900)], 8, 2, 128, 64, seed=9, tail=0)
    length = c["len"]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = _run(c)
    for lens in ([900, 900], [1, 650], [64, 65]):
        length.copy_(cc.ints(lens, dev))
        graph.replay()
        _check(c, out, lse, what=str(lens))


def test_two_streams(dev):
    """Two calls that may run at once, each with the workspace that the binding allocates for it."""
    cases = [_case(dev, [(1, 5000 + 1000 * s), (1, 3)], 32, 8, 128, 64, seed=10 + s) for s in range(2)]
    want = [_run(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got = []
        for c, s in zip(cases, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(_run(c))
    given = []
    for c, s in zip(cases, streams):  # and with the stream as an argument
        given.append(_run(c, stream=s))
    torch.cuda.synchronize()
    for w, a, b in zip(want, got, given):
        assert torch.equal(w[0], a[0]) and torch.equal(w[1], a[1])
        assert torch.equal(w[0], b[0]) and torch.equal(w[1], b[1])


def test_more_new_tokens_than_max_rows_are_left(dev):
    c = _case(dev, [(5, 100), (2, 50)], 4, 2, 64, 16, seed=12)
    whole, whole_lse = _run(c)
    out, lse = _run(c, max_rows=3)
    assert bool((out[3:5] == 5.0).all()) and bool((lse[:, 3:5] == 6.0).all())
    out[3:5], lse[:, 3:5] = whole[3:5], whole_lse[:, 3:5]
    _check(c, out, lse)   # (other rows a tile: other roundings, the same formula)


def test_given_workspace_of_any_contents(dev):
    c = _case(dev, [(1, 3000)], 8, 2, 128, 64, seed=13)
    want = _run(c)
    ws = torch.full((h3q.attention_cache_workspace_bytes(1, 8, 2, 128),), 255, dtype=torch.uint8, device=dev)
    got = _run(c, workspace=ws)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    with pytest.raises(ValueError, match="workspace"):
        _run(c, workspace=ws[:-1])


@pytest.mark.parametrize("heads, kv_heads, dim, page, new", [(8, 2, 128, 64, 1), (12, 2, 64, 16, 2), (4, 2, 256, 32, 3), (64, 8, 128, 16, 1),
                                                             (24, 2, 128, 64, 4)])
def test_more_groups_than_ctas(dev, heads, kv_heads, dim, page, new):
    """Many short sequences beside a few long ones: ranges of many groups, of one, and ends of ranges in all places."""
    rng = np.random.default_rng(17)
    length = [int(n) for n in rng.integers(new, 400, 230)]
    for b, n in ((3, 17000), (120, 9000), (229, 4000)):
        length[b] = n
    c = _case(dev, [(new if b % 7 else 0, n) for b, n in enumerate(length)], heads, kv_heads, dim, page, seed=18)
    out, lse = _run(c)
    _check(c, out, lse)
    again = _run(c)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    assert h3q.h3q_kernel_error_flag() == 0


@pytest.mark.parametrize("gain", [0.01, 4.0, 40.0])
@pytest.mark.parametrize("heads, kv_heads, dim", [(8, 2, 128), (16, 1, 128), (32, 1, 64), (8, 1, 256), (40, 1, 128)])
def test_scores_that_grow_along_the_cache(dev, gain, heads, kv_heads, dim):
    """The running maximum moves a little in each tile, or far: keys whose scales grow with their position."""
    c = _case(dev, [(1, 2500), (1, 700)], heads, kv_heads, dim, 16, seed=19, gain=gain)
    scales = c["cache"][1]
    for b in range(2):
        n = c["len"][b].item()
        for i, page in enumerate(c["table"][b, :(n + 15) // 16].tolist()):
            scales[page] = 8 + min(100, 100 * 16 * i // n)
    out, lse = _run(c)
    _check(c, out, lse)


def test_sequences_that_share_pages(dev):
    """A prefix that several sequences have: their tables name the same pages."""
    c = _case(dev, [(1, 200), (1, 200), (2, 130)], 8, 2, 128, 16, seed=21)
    c["table"][1, :12] = c["table"][0, :12]
    c["table"][2, :8] = c["table"][0, :8]
    out, lse = _run(c)
    _check(c, out, lse)


@pytest.mark.parametrize("new, keys", [(1, 9000), (12, 3000)])
def test_graphs_that_share_a_workspace(dev, new, keys):
    """Two captured calls with one workspace, replayed one after the other in any order, and an eager one between."""
    cases = [_case(dev, [(new, keys), (1, keys // 3 + s)], 16, 4, 128, 64, seed=22 + s) for s in range(2)]
    want = [_run(c) for c in cases]
    ws = torch.empty(h3q.attention_cache_workspace_bytes(new, 16, 4, 128), dtype=torch.uint8, device=dev)
    graphs, got = [], []
    for c in cases:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(_run(c, workspace=ws))
    for order in ((0, 1), (1, 0), (0, 0, 1)):
        for i in order:
            for t in got[i]:
                t.fill_(7.0)
            graphs[i].replay()
        _run(cases[0], workspace=ws)
        for a, b in zip(want, got):
            n = cases[0]["cu"][-1]
            assert torch.equal(a[0][:n], b[0][:n]) and torch.equal(a[1][:, :n], b[1][:, :n])


@pytest.mark.parametrize("new, heads", [(1, 8), (3, 32), (8, 64)])
def test_pages_past_2_32_bytes(dev, new, heads):
    """The same pages at the end of a cache of 4.6 GB of codes give the same bits."""
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    c = _case(dev, [(new, 900), (new, 333)], heads, 8, 128, 128, seed=25)
    want = _run(c)
    pages = 70000
    far = [torch.zeros((pages, *t.shape[1:]), dtype=torch.uint8, device=dev) for t in c["cache"]]
    shift = pages - c["cache"][0].shape[0]
    for t, f in zip(c["cache"], far):
        f[shift:] = t
    assert far[0].numel() > 2 ** 32
    got = _run({**c, "cache": tuple(far), "table": c["table"] + shift})
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_more_whole_groups_than_ctas(dev):
    """Tables of one tile a sequence: a CTA takes several groups, and nothing is joined."""
    c = _case(dev, [(b % 3, 2 + b % 254) for b in range(420)], 12, 3, 128, 64, seed=27)
    c["table"] = c["table"][:, :4].contiguous()   # (256 positions)
    out, lse = _run(c)
    _check(c, out, lse)


def test_captured_behind_copies_and_other_streams(dev):
    """The calls as the first of a graph, behind copies from the host, fills, and work of another stream."""
    heads, kv, dim, page, batch = 16, 4, 128, 16, 3
    cache = h3q.kv_cache_nvfp4(64, kv, page, dim, dev)
    table = torch.randperm(64, device=dev)[:60].to(torch.int32).view(batch, 20).contiguous()
    cu, kv_len = cc.ints([0, 1, 2, 3], dev), cc.ints([5, 6, 7], dev)
    new = [torch.tensor(n, dtype=torch.int32).pin_memory() for n in ([300, 17, 1], [20, 301, 64])]
    host = torch.empty_like(new[0]).pin_memory()
    kg, vg = _scales(dev, (448.0, 300.0))
    x = torch.randn((batch, heads + 2 * kv, dim), device=dev).bfloat16()
    for t in cache:
        t.random_(0, 128)
    lse = torch.zeros((heads, batch), device=dev)
    other, y = torch.cuda.Stream(), torch.zeros_like(x)

    def step():
        kv_len.copy_(host, non_blocking=True)
        h3q.h3q_kv_cache_write_nvfp4(y[:, heads:heads + kv], y[:, heads + kv:], cache, cu, kv_len, table, kg, vg)
        lse.zero_()
        out = h3q.h3q_attention_cache_nvfp4(y[:, :heads], cache, cu, kv_len, table, kg, vg, lse=lse)
        return out, h3q.h3q_kv_cache_read_nvfp4(cache, cu, kv_len, table, kg, vg, rows=batch)

    host.copy_(new[0])
    y.copy_(x)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        other.wait_stream(main)
        with torch.cuda.stream(other):
            y.copy_(x)
        kv_len.zero_()
        main.wait_stream(other)
        out, back = step()
    for n in new:
        host.copy_(n)
        x.copy_(torch.randn_like(x))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, lse, *back, *cache)]
        y.copy_(x)
        want, rows = step()
        for a, b in zip(got, (want, lse, *rows, *cache)):
            assert torch.equal(a, b)
        c = {"q": x[:, :heads], "cache": cache, "cu": cu, "len": kv_len, "table": table, "gs": (448.0, 300.0), "mask": None, "page": page}
        _check(c, want, lse)
