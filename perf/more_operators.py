"""What a video transformer's block needs beside the NVFP4 producers: what it is measured on.

* ``axes``    the QKV epilogue with rotary positions of several axes (time, height, width): bias, norm of
              each head, rotation by angles made from the tokens' positions;
* ``norms``   the norm after a block, its gate and scaled residual, the norm before the next block and its
              modulation, NVFP4 out;
* ``select``  the key blocks that each block of queries will attend to, by a score of pooled queries and keys;
* ``sparse``  softmax attention over the listed key blocks (prompts, video, single tokens).

Query block i of sequence b is row cu_q[b] // block_q + b + i of the lists [kv_heads, rows_q // block_q +
batch, top]: ascending block numbers of the sequence's keys, then -1.  Rows of no block hold -1.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # a short prompt of text and image tokens: latency
        {"name": "axes 37 tokens", "op": "axes", "rows": 37, "heads": 8, "kv_heads": 2, "dim": 64,
         "dims": "16,24,24", "pairs": False, "norm": False, "bias": True, "weights": False, "far": 5000},
        # one latent frame of a video, every head's rotation of another axis split
        {"name": "axes 2,040 tokens", "op": "axes", "rows": 2040, "heads": 32, "kv_heads": 8, "dim": 128,
         "dims": "16,24,24", "pairs": False, "norm": True, "bias": True, "weights": False, "far": 1000000},
        # a video clip's 32 latent frames of 34 x 60 tokens
        {"name": "axes 65,280 tokens", "op": "axes", "rows": 65280, "heads": 56, "kv_heads": 56, "dim": 128,
         "dims": "44,42,42", "pairs": True, "norm": True, "bias": True, "weights": True, "far": 0},
        # one decoding step of a language model with norms on both sides
        {"name": "norms 64 rows", "op": "norms", "rows": 64, "cols": 4096, "frames": 0, "bias": False, "mod": False,
         "keep": 1.0},
        # an image of 1,000 tokens, ragged
        {"name": "norms 1,000 rows", "op": "norms", "rows": 1000, "cols": 7168, "frames": 3, "bias": True,
         "mod": True, "keep": 1.0},
        # the clip, 32 frames with a gate and a modulation each
        {"name": "norms 65,280 rows", "op": "norms", "rows": 65280, "cols": 7168, "frames": 32, "bias": True,
         "mod": True, "keep": 0.9375},
        # one new token of 16 conversations
        {"name": "select 16 tokens", "op": "select", "batch": 16, "new_lo": 1, "new_hi": 1, "ctx_lo": 1000,
         "ctx_hi": 9000, "heads": 32, "kv_heads": 8, "dim": 128, "block_q": 64, "block_k": 64, "top": 16,
         "causal": True, "first": 1},
        # chunks of long prompts over their prefixes
        {"name": "select 4 chunks", "op": "select", "batch": 4, "new_lo": 400, "new_hi": 2040, "ctx_lo": 4000,
         "ctx_hi": 30000, "heads": 32, "kv_heads": 8, "dim": 128, "block_q": 64, "block_k": 64, "top": 32,
         "causal": True, "first": 1},
        # the clip: every token may see every other
        {"name": "select 65,280 tokens", "op": "select", "batch": 1, "new_lo": 65280, "new_hi": 65280, "ctx_lo": 0,
         "ctx_hi": 0, "heads": 56, "kv_heads": 56, "dim": 128, "block_q": 128, "block_k": 128, "top": 64,
         "causal": False, "first": 0},
        # one new token of 16 conversations over its blocks
        {"name": "sparse 16 tokens", "op": "sparse", "batch": 16, "new_lo": 1, "new_hi": 1, "ctx_lo": 1000,
         "ctx_hi": 9000, "heads": 32, "kv_heads": 8, "dim": 128, "block_q": 64, "block_k": 64, "top": 16,
         "causal": True},
        # chunks of long prompts
        {"name": "sparse 4 chunks", "op": "sparse", "batch": 4, "new_lo": 400, "new_hi": 2040, "ctx_lo": 4000,
         "ctx_hi": 30000, "heads": 32, "kv_heads": 8, "dim": 128, "block_q": 64, "block_k": 64, "top": 32,
         "causal": True},
        # half of the clip, an eighth of its blocks
        {"name": "sparse 32,640 tokens", "op": "sparse", "batch": 1, "new_lo": 32640, "new_hi": 32640, "ctx_lo": 0,
         "ctx_hi": 0, "heads": 56, "kv_heads": 56, "dim": 128, "block_q": 128, "block_k": 128, "top": 32,
         "causal": False},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _some_heads(rng):
    kv = rng.choice((1, 2, 4, 8, 8, 16, 56))
    return kv, kv * (rng.choice((1, 2, 3, 4, 8)) if kv <= 8 else 1)


def draw(rng):
    op = rng.choice(("axes", "norms", "select", "sparse"))
    if op == "axes":
        dim = rng.choice((64, 128, 128, 256))
        kv, heads = _some_heads(rng)
        cut = rng.choice((1, 2, 3, 4))  # axes
        rot = 16 * rng.randint(1, dim // 16)
        at = sorted(rng.sample(range(1, rot // 2), cut - 1))
        dims = [2 * (b - a) for a, b in zip([0] + at, at + [rot // 2])]
        return {"op": op, "rows": _spread(rng, 1, 65280 * 56 * 128 // (max(heads, 56) * max(dim, 128))), "heads": heads,
                "kv_heads": kv, "dim": dim, "dims": ",".join(map(str, dims)), "pairs": rng.random() < 0.5,
                "norm": rng.random() < 0.7, "bias": rng.random() < 0.5, "weights": rng.random() < 0.5,
                "far": rng.choice((0, 0, 5000, 1000000))}
    if op == "norms":
        frames = rng.choice((0, 1, 3, 32))
        return {"op": op, "rows": _spread(rng, 1, 65280), "cols": rng.choice((64 * rng.randint(1, 112), 2048, 4096, 7168)),
                "frames": frames, "bias": rng.random() < 0.5, "mod": frames > 0 and rng.random() < 0.8,
                "keep": rng.choice((1.0, 1.0, 0.9375, 0.7))}
    kv, heads = _some_heads(rng)
    case = {"op": op, "batch": _spread(rng, 1, 16), "heads": heads, "kv_heads": kv, "dim": rng.choice((64, 128, 128)),
            "block_q": rng.choice((64, 128, 128, 256)), "block_k": rng.choice((64, 64, 128, 256)),
            "causal": rng.random() < 0.5}
    most = 1.5e8 / (case["batch"] * heads * case["dim"])  # rows of a sequence
    case["new_hi"] = _spread(rng, 1, int(min(32640, max(2, most))))
    case["new_lo"] = rng.randint(1, case["new_hi"])
    case["ctx_hi"] = _spread(rng, 1, int(min(100000, max(64, most * heads / kv)))) if rng.random() < 0.7 else 0
    case["ctx_lo"] = rng.randint(0, case["ctx_hi"])
    if op == "select":
        case["first"] = rng.choice((0, 0, 1, 2))
        case["top"] = case["first"] + -(-case["block_q"] // case["block_k"]) + 1 + _spread(rng, 1, 64) - 1
        return case
    case["top"] = _spread(rng, 1, 64)
    blocks = case["batch"] * (1 + case["new_hi"] // case["block_q"])
    # keys and scores that the plain form gathers, against the largest listed case's
    per = blocks * kv * case["block_k"]
    case["top"] = max(1, min(case["top"], int(2.5e7 / per), int(2.5e9 / (per * case["block_q"] * heads // kv))))
    return case


def _lengths(case):
    """New rows and context of each sequence: the same for a case whatever the seed, so that a
    case's work is one number."""
    rng = random.Random(",".join(str(case[k]) for k in sorted(case) if k != "name"))
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]
    return [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])], ctx


# --------------------------------------------------------------------------- inputs

def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEV)


def _offsets(counts):
    total, at = 0, [0]
    for c in counts:
        total += c
        at.append(total)
    return at


def _normal(gen, rows, cols, gain):
    """bf16 rows ~ N(0, 1) times a gain of each column, as a projection's channels have it."""
    out = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
    step = max(1, (1 << 27) // cols)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        out[r:r + n] = torch.randn((n, cols), generator=gen, device=DEV) * gain
    return out


def _gain(gen, cols, spread=0.4):
    return torch.exp(spread * torch.randn(cols, generator=gen, device=DEV))


def _dims(case):
    return [int(x) for x in case["dims"].split(",")]


def _prepare_axes(case, gen):
    s = dict(case)
    rows, dim = case["rows"], case["dim"]
    dims = _dims(case)
    for name, heads in (("q", case["heads"]), ("k", case["kv_heads"]), ("v", case["kv_heads"])):
        s[name] = _normal(gen, rows, heads * dim, _gain(gen, heads * dim))
        s["b" + name] = 0.3 * torch.randn(heads * dim, generator=gen, device=DEV)
        s["b" + name] = s["b" + name].bfloat16()
        s["w" + name] = _gain(gen, dim, 0.1).bfloat16()
    # frames of 34 x 60 tokens, the time counted from some way on (a long video's later clips)
    r = torch.arange(rows, device=DEV)
    place = [r // 2040, r // 60 % 34, r % 60, r % 7][:len(dims)]
    start = torch.randint(-case["far"], case["far"] + 1, (len(dims),), generator=gen, device=DEV)
    s["positions"] = torch.stack([p + a for p, a in zip(place, start)], 1).int().contiguous()
    s["freq"] = torch.tensor([10000.0 ** (-2.0 * i / d) for d in dims for i in range(d // 2)], dtype=torch.float64,
                             device=DEV)
    s["axis"] = _ints([a for a, d in enumerate(dims) for _ in range(d // 2)], torch.int64)
    return s


def _prepare_norms(case, gen):
    s = dict(case)
    rows, cols, frames = case["rows"], case["cols"], case["frames"]
    s["o"] = _normal(gen, rows, cols, _gain(gen, cols))
    s["h"] = torch.randn((rows, cols), generator=gen, device=DEV) * (2.0 * _gain(gen, cols))
    s["gamma_post"] = (0.5 * _gain(gen, cols, 0.2)).bfloat16()
    s["gamma"] = _gain(gen, cols, 0.2).bfloat16()
    s["bias_row"] = (0.2 * torch.randn(cols, generator=gen, device=DEV)).bfloat16() if case["bias"] else None
    s["gate"] = s["table"] = s["frame"] = None
    if frames:
        s["gate"] = (0.5 * torch.randn((frames, cols), generator=gen, device=DEV)).bfloat16()
        if case["mod"]:
            s["table"] = (0.3 * torch.randn((frames, 2, cols), generator=gen, device=DEV)).bfloat16()
        s["frame"] = (torch.arange(rows, device=DEV) * frames // rows).int()
    s["gsf"] = torch.tensor([320.0], device=DEV)  # 2688 over the largest value, near enough
    return s


def _prepare_blocks(case, gen):
    s = dict(case)
    new, ctx = _lengths(case)
    total = [a + b for a, b in zip(new, ctx)]
    rows, keys, heads, kv, dim = sum(new), sum(total), case["heads"], case["kv_heads"], case["dim"]
    s["rows"], s["keys"], s["most"] = rows, keys, max(total)
    s["cu_q"], s["cu_k"] = _ints(_offsets(new)), _ints(_offsets(total))
    s["q"] = _normal(gen, rows, heads * dim, _gain(gen, heads * dim)).view(rows, heads, dim)
    s["k"] = _normal(gen, keys, kv * dim, 1.0).view(keys, kv, dim)
    if case["op"] == "select":
        # what neighbouring tokens share, so that blocks differ as an image's regions do
        for x in (s["q"], s["k"]):
            n = -(-x.shape[0] // 32)
            x += (0.5 * torch.randn((n, *x.shape[1:]), generator=gen, device=DEV).bfloat16()).repeat_interleave(
                32, 0)[:x.shape[0]]
        return s
    s["v"] = _normal(gen, keys, kv * dim, _gain(gen, kv * dim)).view(keys, kv, dim)
    # lists as a selection leaves them: blocks near the queries' own more often, and others
    b, i, there = _block_rows(s)
    length = (s["cu_k"][1:] - s["cu_k"][:-1])[b]
    own_at = (length - (s["cu_q"][1:] - s["cu_q"][:-1])[b] + i * case["block_q"]) // case["block_k"]
    end = length
    if case["causal"]:
        end = torch.minimum(length, length - (s["cu_q"][1:] - s["cu_q"][:-1])[b] + (i + 1) * case["block_q"])
    count = -(-end // case["block_k"])
    j = torch.arange(-(-max(total) // case["block_k"]), device=DEV)
    like = torch.rand((kv, b.shape[0], j.shape[0]), generator=gen, device=DEV)
    like += (-(j - own_at[:, None]).abs() / 8.0).exp()
    like.masked_fill_(~(there[:, None] & (j < count[:, None])), -1.0)
    if case["top"] > j.shape[0]:
        like = torch.nn.functional.pad(like, (0, case["top"] - j.shape[0]), value=-1.0)
    value, at = like.topk(case["top"], -1)
    at = at.masked_fill(value < 0, 1 << 30).sort(-1).values
    s["blocks"] = at.masked_fill(at == 1 << 30, -1).int().contiguous()
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return {"axes": _prepare_axes, "norms": _prepare_norms}.get(case["op"], _prepare_blocks)(case, gen)


# --------------------------------------------------------------------------- plain forms

def _plain_rotated(s, x, bias, weight, heads):
    x = x.float().view(s["rows"], heads, s["dim"])
    if bias is not None:
        x = x + bias.float().view(heads, -1)
    if s["norm"]:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
        if weight is not None:
            x = x * weight.float()
    angle = s["positions"].double()[:, s["axis"]] * s["freq"]  # far positions: in 64 bits
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    rot = 2 * s["axis"].shape[0]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if s["pairs"] else (x[..., :rot // 2], x[..., rot // 2:rot])
    turned = (a * cos - b * sin, a * sin + b * cos)
    turned = torch.stack(turned, -1).flatten(-2) if s["pairs"] else torch.cat(turned, -1)
    return torch.cat((turned, x[..., rot:]), -1).bfloat16()


def _plain_axes(s):
    v = s["v"].float()
    if s["bias"]:
        v = v + s["bv"].float()
    q, k = (_plain_rotated(s, s[n], s["b" + n] if s["bias"] else None, s["w" + n] if s["weights"] else None, h)
            for n, h in (("q", s["heads"]), ("k", s["kv_heads"])))
    return q, k, v.view(s["rows"], s["kv_heads"], s["dim"]).bfloat16()


def _plain_rstd(x):
    """1 / sqrt(mean(x^2) + eps) of fp32 rows, the squares summed in the producers' documented order, on
    which the bits of what is quantised hang: chunk c of 8 columns on lane c % 128, a fused multiply-add for
    each of its 8 partials (here in 64 bits, rounded to 32), then the lanes in a butterfly of 32 and four."""
    rows, cols = x.shape
    wide = torch.nn.functional.pad(x, (0, -cols % 1024)).view(rows, -1, 128, 8)
    p = torch.zeros((rows, 128, 8), device=DEV)
    for j in range(wide.shape[1]):
        p = torch.addcmul(p.double(), wide[:, j].double(), wide[:, j].double()).float()
    p = (p[..., 0] + p[..., 1] + (p[..., 2] + p[..., 3])) + (p[..., 4] + p[..., 5] + (p[..., 6] + p[..., 7]))
    p = p.view(rows, 4, 32)
    for n in (16, 8, 4, 2, 1):
        p = p[..., :n] + p[..., n:]
    p = p[..., 0]
    ss = (p[:, 0] + p[:, 1]) + (p[:, 2] + p[:, 3])
    mean = ss / torch.full((1,), float(cols), device=DEV) + 1e-6
    return (torch.ones_like(mean) / mean.sqrt())[:, None]


def _plain_codes(y, gsf):
    """NVFP4 of bf16 y [rows, cols], each step rounded to 32 bits: packed codes, and the scales in tiles of 128
    rows x 4 groups (row r % 32, then r / 32 % 4, then the group), the rows past the last one zero."""
    blocks = y.float().unflatten(-1, (-1, 16))
    six = torch.full((1,), 6.0, device=DEV)
    scale = (gsf * (blocks.abs().amax(-1) / six)).clamp(max=448.0).to(torch.float8_e4m3fn)
    dec = scale.float() / gsf
    inv = torch.where(dec != 0, torch.ones_like(dec) / dec, torch.zeros_like(dec))
    v = blocks * inv[..., None]
    a = v.abs()
    code = torch.zeros(a.shape, dtype=torch.uint8, device=DEV)
    for edge, even in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= edge) if even else (a > edge)  # a tie goes to the even code
    code = (code + (torch.signbit(v).to(torch.uint8) << 3)).flatten(-2)
    rows, groups = scale.shape
    tiles = torch.nn.functional.pad(scale.view(torch.uint8), (0, 0, 0, -rows % 128))
    tiles = tiles.view(-1, 4, 32, groups // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, groups)
    return code[..., 0::2] | code[..., 1::2] << 4, tiles


def _plain_norms(s):
    u = s["o"] if s["bias_row"] is None else (s["o"].float() + s["bias_row"].float()).bfloat16()
    u = u.float()
    n = u * _plain_rstd(u) * s["gamma_post"].float()
    t = s["frame"].long() if s["frame"] is not None else None
    if s["gate"] is not None:
        n = n * s["gate"].float()[t]
    s["h"].copy_(s["h"] * s["keep"] + n)
    y = s["h"] * _plain_rstd(s["h"]) * s["gamma"].float()
    if s["table"] is not None:
        y = y * (1 + s["table"][:, 1].float())[t] + s["table"][:, 0].float()[t]
    return s["h"], *_plain_codes(y.bfloat16(), s["gsf"])


def _block_rows(s, keys=False):
    """Sequence and number of each block row, and whether it is one: row cu[b] // size + b + i."""
    cu, size, rows = (s["cu_k"], s["block_k"], s["keys"]) if keys else (s["cu_q"], s["block_q"], s["rows"])
    r = torch.arange(rows // size + cu.shape[0] - 1, device=DEV)
    first = cu[:-1].long() // size + torch.arange(cu.shape[0] - 1, device=DEV)
    b = torch.searchsorted(first, r, right=True) - 1
    i = r - first[b]
    return b, i, i * size < (cu[1:] - cu[:-1])[b]


def _row_index(cu, b, i, size):
    """Packed rows [blocks, size] of the blocks, and which are their sequence's."""
    at = i[:, None] * size + torch.arange(size, device=DEV)
    mine = at < (cu[1:] - cu[:-1])[b][:, None]
    return cu[b][:, None].long() + at, mine


def _block_sums(x, cu, b, i, size):
    """Sums in 64 bits [blocks, heads, dim] (what decides next to a border) and counts of the blocks' rows."""
    at, mine = _row_index(cu, b, i, size)
    rows = x[at.clamp(max=x.shape[0] - 1)].double()
    return rows.mul_(mine[..., None, None]).sum(1), mine.sum(1)


def _plain_select(s):
    kv, top = s["kv_heads"], s["top"]
    b, i, there = _block_rows(s)
    kb, kj, _ = _block_rows(s, keys=True)
    q, _ = _block_sums(s["q"], s["cu_q"], b, i, s["block_q"])
    k, n = _block_sums(s["k"], s["cu_k"], kb, kj, s["block_k"])
    q = q.view(q.shape[0], kv, -1, s["dim"]).sum(2)
    score = q.transpose(0, 1) @ k.permute(1, 2, 0) / n.clamp(min=1)  # [kv, query blocks, key blocks]
    rows = (_row_index(s["cu_q"], b, i, s["block_q"])[1].sum(1) * (s["heads"] // kv)).clamp(min=1)[:, None]
    j = torch.arange(max(top, -(-s["most"] // s["block_k"])), device=DEV)
    base = s["cu_k"][:-1].long() // s["block_k"] + torch.arange(s["batch"], device=DEV)
    at = (base[b][:, None] + j).clamp(max=k.shape[0] - 1)
    score = score.gather(2, at[None].expand(kv, -1, -1))
    length, new = (s["cu_k"][1:] - s["cu_k"][:-1])[b], (s["cu_q"][1:] - s["cu_q"][:-1])[b]
    own_from = length - new + i * s["block_q"]  # the position of the block's first query
    end = length
    if s["causal"]:
        end = torch.minimum(length, own_from + s["block_q"])
    allowed = there[:, None] & (j * s["block_k"] < end[:, None])
    always = j.expand_as(allowed) < s["first"]
    if s["causal"]:
        always = always | (torch.minimum((j + 1) * s["block_k"], length[:, None]) > own_from[:, None])
    rank = score.masked_fill(always, math.inf).masked_fill(~allowed, -math.inf)
    value, at = rank.sort(dim=-1, descending=True, stable=True)  # of equal ones the lowest number first
    at = at[..., :top].masked_fill(value[..., :top] == -math.inf, 1 << 30).sort(-1).values
    score = (score / rows).gather(2, at.clamp(max=j.shape[0] - 1)).masked_fill(at == 1 << 30, -math.inf)
    return at.masked_fill(at == 1 << 30, -1).int(), score.float()


def _plain_sparse(s):
    kv, dim, size = s["kv_heads"], s["dim"], s["block_k"]
    group = s["heads"] // kv
    b, i, _ = _block_rows(s)
    at, mine = _row_index(s["cu_q"], b, i, s["block_q"])
    x = s["q"][at.clamp(max=s["rows"] - 1)].float()  # [blocks, rows, heads, dim]
    x = x.view(*at.shape, kv, group, dim).permute(2, 0, 3, 1, 4).reshape(kv, at.shape[0], -1, dim)
    key = (s["blocks"].long()[..., None] * size + torch.arange(size, device=DEV)).flatten(-2)  # [kv, blocks, keys]
    length, rows = (s["cu_k"][1:] - s["cu_k"][:-1])[b], (s["cu_q"][1:] - s["cu_q"][:-1])[b]
    hidden = ((key < 0) | (key >= length[:, None]))[:, :, None]
    if s["causal"]:
        sees = (length - rows)[:, None] + i[:, None] * s["block_q"] + torch.arange(s["block_q"], device=DEV)
        hidden = hidden | (key[:, :, None] > sees[..., None])
    place = (key.clamp(min=0) + s["cu_k"][b][:, None]).clamp(max=s["keys"] - 1)
    head = torch.arange(kv, device=DEV)[:, None, None]
    w = x @ s["k"][place, head].float().transpose(-1, -2)
    w.mul_(dim ** -0.5)
    w = w.view(kv, at.shape[0], group, -1, key.shape[-1]).masked_fill_(hidden[:, :, None], -math.inf)
    top = w.amax(-1, keepdim=True).clamp(min=-3e38)
    w.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    o = (w.flatten(2, 3) @ s["v"][place, head].float()).view(*w.shape[:-1], dim) / total.clamp(min=1e-38)
    lse = (top + total.log()).squeeze(-1)
    o = o.permute(1, 3, 0, 2, 4).reshape(*at.shape, s["heads"], dim)
    lse = lse.permute(1, 3, 0, 2).reshape(*at.shape, s["heads"])
    return o[mine].bfloat16(), lse[mine].t().contiguous()


# --------------------------------------------------------------------------- one pass

def run(s):
    if s["op"] == "axes":
        if own:
            import nvfp4_activation_quantize_gb300 as h3q

            q, k, v = h3q.h3q_qkv_epilogue_axes(
                s["q"], s["k"], s["v"], s["positions"], _dims(s), s["heads"], kv_heads=s["kv_heads"], theta=10000.0,
                biases=(s["bq"], s["bk"], s["bv"]) if s["bias"] else None,
                weights=(s["wq"], s["wk"]) if s["weights"] and s["norm"] else None, norm=s["norm"], eps=1e-6,
                interleaved=s["pairs"])
        else:
            q, k, v = _plain_axes(s)
        return {"q": q, "k": k, "v": v}
    if s["op"] == "norms":
        if own:
            import nvfp4_activation_quantize_gb300 as h3q

            codes, scales = h3q.h3q_postnorm_residual_adaln_nvfp4(
                s["h"], s["o"], s["gamma_post"], s["gamma"], s["gsf"], bias=s["bias_row"], gate_table=s["gate"],
                mod_table=s["table"], residual_scale=s["keep"], row_frame=s["frame"], eps=1e-6)
            h = s["h"]
        else:
            h, codes, scales = _plain_norms(s)
        # codes as they are packed, scales as the E4M3 numbers that they are
        return {"h": h, "codes": codes, "scales": scales.view(torch.float8_e4m3fn)}
    if s["op"] == "select":
        if own:
            import nvfp4_activation_quantize_gb300 as h3q

            blocks = torch.empty((s["kv_heads"], s["rows"] // s["block_q"] + s["batch"], s["top"]), dtype=torch.int32,
                                 device=DEV)
            scores = torch.empty(blocks.shape, dtype=torch.float32, device=DEV)
            h3q.h3q_select_blocks(s["q"], s["k"], s["cu_q"], s["cu_k"], s["top"], block_q=s["block_q"],
                                  block_k=s["block_k"], causal=s["causal"], first=s["first"], blocks=blocks,
                                  scores=scores)
        else:
            blocks, scores = _plain_select(s)
        return {"blocks": blocks, "scores": scores}
    if own:
        import nvfp4_activation_quantize_gb300 as h3q

        lse = torch.empty((s["heads"], s["rows"]), dtype=torch.float32, device=DEV)
        o = h3q.h3q_attention_blocks(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["blocks"], block_q=s["block_q"],
                                     block_k=s["block_k"], causal=s["causal"], lse=lse)
    else:
        o, lse = _plain_sparse(s)
    return {"o": o, "lse": lse}


# --------------------------------------------------------------------------- what it takes

def _listed_pairs(case):
    """(query, key) pairs of one head over full lists, the hidden corner of the last blocks not counted."""
    new, ctx = _lengths(case)
    pairs = 0
    for n, c in zip(new, ctx):
        for first in range(0, n, case["block_q"]):
            rows = min(case["block_q"], n - first)
            keys = min(n + c, c + first + rows) if case["causal"] else n + c
            pairs += rows * min(keys, case["top"] * case["block_k"]) - (rows * (rows - 1) // 2 if case["causal"] else 0)
    return pairs


def work(case):
    if case["op"] == "axes":
        n = case["rows"] * (case["heads"] + 2 * case["kv_heads"]) * case["dim"]
        return {"bytes": 4 * n + 4 * case["rows"] * len(_dims(case)), "flops": 0}
    if case["op"] == "norms":
        rows, cols = case["rows"], case["cols"]
        tables = cols * (4 + 2 * case["bias"] + case["frames"] * (2 + 4 * case["mod"]))
        return {"bytes": rows * cols * 10 + rows * cols // 2 + -(-rows // 128) * 128 * cols // 16 + tables, "flops": 0}
    new, ctx = _lengths(case)
    rows, keys = sum(new), sum(new) + sum(ctx)
    kv, heads, dim = case["kv_heads"], case["heads"], case["dim"]
    lists = kv * (rows // case["block_q"] + case["batch"]) * case["top"] * 4
    if case["op"] == "select":
        lists *= 2  # and scores
        blocks = sum(-(-n // case["block_q"]) * -(-(n + c) // case["block_k"]) for n, c in zip(new, ctx))
        return {"bytes": 2 * dim * (rows * heads + keys * kv) + lists, "flops": 2 * dim * kv * blocks}
    pairs = _listed_pairs(case)
    used = min(keys, sum(-(-n // case["block_q"]) for n in new) * case["top"] * case["block_k"])  # of each key head
    return {"bytes": rows * heads * (4 * dim + 4) + used * kv * dim * 4 + lists, "flops": 4 * dim * heads * pairs}


# --------------------------------------------------------------------------- the definition in 64 bits

def _exact_axes(case, s):
    dims = _dims(case)
    out = {}
    for name, heads in (("q", case["heads"]), ("k", case["kv_heads"]), ("v", case["kv_heads"])):
        x = s[name].double().view(case["rows"], heads, case["dim"])
        if case["bias"]:
            x += s["b" + name].double().view(heads, case["dim"])
        if name != "v":
            if case["norm"]:
                x /= torch.sqrt((x * x).sum(-1, keepdim=True) / case["dim"] + 1e-6)
                if case["weights"]:
                    x *= s["w" + name].double()
            rot, j = sum(dims), 0
            turned = x.clone()
            for axis, d in enumerate(dims):
                for i in range(d // 2):
                    angle = s["positions"][:, axis].double() * math.exp(-math.log(10000.0) * 2 * i / d)
                    c, t = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
                    a, b = (2 * j, 2 * j + 1) if case["pairs"] else (j, j + rot // 2)
                    turned[..., a] = x[..., a] * c - x[..., b] * t
                    turned[..., b] = x[..., b] * c + x[..., a] * t
                    j += 1
            x = turned
        out[name] = x
    return out


def _exact_norms(case, s):
    u = s["o"].double()
    if case["bias"]:
        u = (u + s["bias_row"].double()).bfloat16().double()
    n = u / torch.sqrt((u * u).mean(1, keepdim=True) + 1e-6) * s["gamma_post"].double()
    if case["frames"]:
        n *= s["gate"].double()[s["frame"].long()]
    h = s["h"].double() * case["keep"] + n
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6) * s["gamma"].double()
    if case["frames"] and case["mod"]:
        y = y * (1 + s["table"][:, 1].double()[s["frame"].long()]) + s["table"][:, 0].double()[s["frame"].long()]
    a = (y.bfloat16().double() / 6 * s["gsf"].double()).abs().unflatten(1, (-1, 16)).amax(-1)
    step = torch.pow(2.0, torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)  # E4M3: three bits behind the point
    f = (torch.round(a / step) * step).clamp(max=448.0)
    r, g = torch.arange(f.shape[0], device=DEV)[:, None], torch.arange(f.shape[1], device=DEV)
    place = (r // 128 * (f.shape[1] // 4) + g // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + g % 4
    scales = torch.zeros(-(-f.shape[0] // 128) * 128 * f.shape[1], dtype=torch.float64, device=DEV)
    scales[place.flatten()] = f.flatten()
    return {"h": h, "codes": None, "scales": scales.view(-1, f.shape[1])}


def _exact_select(case, s):
    new, ctx = _lengths(case)
    cu_q, cu_k = _offsets(new), _offsets([a + b for a, b in zip(new, ctx)])
    kv, top, size = case["kv_heads"], case["top"], case["block_k"]
    scores = torch.full((kv, sum(new) // case["block_q"] + case["batch"], top), -math.inf, dtype=torch.float64, device=DEV)
    for b, (n, c) in enumerate(zip(new, ctx)):
        keys = s["k"][cu_k[b]:cu_k[b + 1]].double()
        means = torch.stack([x.mean(0) for x in keys.split(size)])  # [blocks, kv, dim]
        for first in range(0, n, case["block_q"]):
            last = min(n, first + case["block_q"])
            mean = s["q"][cu_q[b] + first:cu_q[b] + last].double().mean(0).view(kv, -1, case["dim"]).mean(1)
            score = torch.einsum("hd,jhd->hj", mean, means)
            end = -(-(c + last if case["causal"] else n + c) // size)
            rank = score[:, :end].clone()
            rank[:, :case["first"]] = math.inf
            if case["causal"]:
                rank[:, (c + first) // size:] = math.inf
            at = rank.topk(min(top, end), -1).indices.sort(-1).values
            scores[:, cu_q[b] // case["block_q"] + b + first // case["block_q"], :at.shape[1]] = score.gather(1, at)
    return {"blocks": None, "scores": scores}


def _exact_sparse(case, s):
    new, ctx = _lengths(case)
    cu_q, cu_k = _offsets(new), _offsets([a + b for a, b in zip(new, ctx)])
    group = case["heads"] // case["kv_heads"]
    o = torch.zeros((sum(new), case["heads"], case["dim"]), dtype=torch.float64, device=DEV)
    lse = torch.zeros((case["heads"], sum(new)), dtype=torch.float64, device=DEV)
    lists = s["blocks"].cpu().tolist()
    for b, (n, c) in enumerate(zip(new, ctx)):
        for first in range(0, n, case["block_q"]):
            last = min(n, first + case["block_q"])
            rows = slice(cu_q[b] + first, cu_q[b] + last)
            for kv in range(case["kv_heads"]):
                blocks = lists[kv][cu_q[b] // case["block_q"] + b + first // case["block_q"]]
                keys = [p for j in blocks if j >= 0 for p in range(j * case["block_k"], min(n + c, (j + 1) * case["block_k"]))]
                at = torch.tensor(keys, device=DEV, dtype=torch.int64)
                k, v = s["k"][cu_k[b] + at, kv].double(), s["v"][cu_k[b] + at, kv].double()
                t = torch.einsum("rgd,kd->grk", s["q"][rows, kv * group:(kv + 1) * group].double(), k) / math.sqrt(case["dim"])
                if case["causal"]:
                    t.masked_fill_(at > c + torch.arange(first, last, device=DEV)[:, None], -math.inf)
                z = torch.logsumexp(t, 2)
                lse[kv * group:(kv + 1) * group, rows] = z
                w = torch.exp(t - z.clamp(min=-1e300)[..., None])
                o[rows, kv * group:(kv + 1) * group] = torch.einsum("grk,kd->rgd", w, v)
    return {"o": o, "lse": lse}


def exact(case, seed):
    if case["op"] in ("select", "sparse"):
        blocks = sum(-(-n // case["block_q"]) for n in _lengths(case)[0])
    if case["op"] == "select" and blocks * case["kv_heads"] > 2500:
        return None
    if case["op"] == "sparse":
        if case["heads"] * case["dim"] * _listed_pairs(case) > 2e11 or blocks * case["kv_heads"] > 2500:
            return None
    if case["op"] == "axes" and case["rows"] * case["heads"] * case["dim"] > 1e8:
        return None
    if case["op"] == "norms" and case["rows"] * case["cols"] > 1e8:
        return None
    s = prepare(case, seed)
    return {"axes": _exact_axes, "norms": _exact_norms, "select": _exact_select, "sparse": _exact_sparse}[case["op"]](
        case, s)
