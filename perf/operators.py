"""Attention beside the NVFP4 producers: what it is measured on.

Four operators stand between the QKV epilogue and the attention-output quantize of a
serving step:

* ``write``   quantise new key and value rows into a paged NVFP4 cache;
* ``read``    the bf16 rows that such a cache holds, packed again;
* ``prompt``  softmax attention over whole packed sequences (causal or not, grouped heads);
* ``cache``   attention of one or a few drafted tokens a sequence (a chain, or a tree given
              by ancestor masks) over the paged cache that holds context and drafts.

The cache's layout: codes uint8 [pages, kv_heads, page, dim/2] (two E2M1 codes a byte, the even
element low), scales uint8 [pages, kv_heads, page, dim/16] (one E4M3 code per 16 elements);
position p of sequence b is row p % page of page table[b, p // page].  The n new rows of a
sequence stand at its last n positions: length[b] counts them.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of 64 conversations: each appends one token
        {"name": "write 64 tokens", "op": "write", "batch": 64, "new_lo": 1, "new_hi": 1, "ctx_lo": 100, "ctx_hi": 2000,
         "kv_heads": 8, "dim": 128, "page": 64},
        # a video clip's 65,280 tokens of 56 heads enter the cache at once
        {"name": "write 65,280 tokens", "op": "write", "batch": 1, "new_lo": 65280, "new_hi": 65280, "ctx_lo": 0,
         "ctx_hi": 0, "kv_heads": 56, "dim": 128, "page": 64},
        # the prefix of one short conversation, for the next chunk of its prompt
        {"name": "read 1,000 rows", "op": "read", "batch": 1, "ctx_lo": 1000, "ctx_hi": 1000, "kv_heads": 8,
         "dim": 64, "page": 16},
        # the shared prefixes of a batch of conversations
        {"name": "read 32 prefixes", "op": "read", "batch": 32, "ctx_lo": 1500, "ctx_hi": 8191, "kv_heads": 8,
         "dim": 128, "page": 64},
        # a single short prompt: latency
        {"name": "prompt 37 tokens", "op": "prompt", "batch": 1, "new_lo": 37, "new_hi": 37, "ctx_lo": 0, "ctx_hi": 0,
         "heads": 8, "kv_heads": 2, "dim": 64, "causal": True},
        # a serving step's prompts of different lengths, packed
        {"name": "prompt 16 packed", "op": "prompt", "batch": 16, "new_lo": 33, "new_hi": 2040, "ctx_lo": 0,
         "ctx_hi": 0, "heads": 32, "kv_heads": 8, "dim": 128, "causal": True},
        # chunks of long prompts over the prefixes read back from the cache
        {"name": "prompt chunks", "op": "prompt", "batch": 4, "new_lo": 400, "new_hi": 1024, "ctx_lo": 2000,
         "ctx_hi": 7000, "heads": 32, "kv_heads": 8, "dim": 128, "causal": True},
        # four latent frames of 2,040 tokens of a video, 56 heads, every token sees every other
        {"name": "prompt 4 frames", "op": "prompt", "batch": 1, "new_lo": 8160, "new_hi": 8160, "ctx_lo": 0,
         "ctx_hi": 0, "heads": 56, "kv_heads": 56, "dim": 128, "causal": False},
        # one token of one conversation: latency
        {"name": "cache 1 token", "op": "cache", "batch": 1, "new_lo": 1, "new_hi": 1, "ctx_lo": 776, "ctx_hi": 776,
         "heads": 8, "kv_heads": 2, "dim": 64, "page": 16, "tree": False},
        # one decoding step of 64 conversations
        {"name": "cache 64 tokens", "op": "cache", "batch": 64, "new_lo": 1, "new_hi": 1, "ctx_lo": 500,
         "ctx_hi": 8191, "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "tree": False},
        # two very long conversations: the work has to be split along the cache
        {"name": "cache 2 long", "op": "cache", "batch": 2, "new_lo": 1, "new_hi": 1, "ctx_lo": 120000,
         "ctx_hi": 131071, "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "tree": False},
        # trees of up to 16 drafted tokens, verified in one pass
        {"name": "cache trees", "op": "cache", "batch": 16, "new_lo": 9, "new_hi": 16, "ctx_lo": 1000,
         "ctx_hi": 8000, "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "tree": True},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(("write", "read", "prompt", "cache"))
    dim = rng.choice((64, 128, 128))
    kv = rng.choice((1, 2, 4, 8, 8, 16))
    case = {"op": op, "batch": _spread(rng, 1, 64), "kv_heads": kv, "dim": dim}
    if op in ("write", "read", "cache"):
        case["page"] = rng.choice((16, 32, 64, 128))
    if op in ("write", "read"):
        most = max(2, 262144 // (case["batch"] * kv))  # rows of a sequence
        hi = _spread(rng, 1, most)
        if op == "write":
            case["new_hi"] = hi
            case["new_lo"] = rng.randint(1, hi)
            case["ctx_hi"] = rng.randint(0, 2000)
            case["ctx_lo"] = rng.randint(0, case["ctx_hi"])
        else:
            case["ctx_hi"] = hi
            case["ctx_lo"] = rng.randint(1, hi)
        return case
    case["heads"] = kv * rng.choice((1, 2, 4, 8) if kv < 16 else (1, 2, 4))
    if op == "prompt":
        case["batch"] = _spread(rng, 1, 16)
        # scores of at most a quarter of the largest listed case's
        case["new_hi"] = _spread(rng, 1, max(2, int(math.sqrt(9e8 / (case["batch"] * case["heads"])) / 2)))
        case["new_lo"] = rng.randint(1, case["new_hi"])
        case["ctx_hi"] = rng.choice((0, 0, rng.randint(1, 2 * case["new_hi"])))
        case["ctx_lo"] = rng.randint(0, case["ctx_hi"])
        case["causal"] = rng.random() < 0.7
        return case
    case["tree"] = rng.random() < 0.5
    case["new_hi"] = _spread(rng, 1, 64) if case["tree"] else rng.choice((1, 1, rng.randint(2, 8)))
    case["new_lo"] = rng.randint(1, case["new_hi"])
    most = min(131072, max(64, 2097152 // (case["batch"] * kv)), max(64, 400_000_000 // (
        case["batch"] * case["heads"] * case["new_hi"])))
    case["ctx_hi"] = _spread(rng, 1, most)
    case["ctx_lo"] = rng.randint(max(1, case["ctx_hi"] // 8), case["ctx_hi"])
    return case


def _lengths(case):
    """New rows and context of each sequence: the same for a case whatever the seed, so that a
    case's work is one number."""
    rng = random.Random(",".join(str(case[k]) for k in sorted(case) if k != "name"))
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]
    if case["op"] == "read":
        return ctx, [0] * case["batch"]
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


def _gain(gen, cols):
    return torch.exp(0.4 * torch.randn(cols, generator=gen, device=DEV))


def _paged(case, gen, total):
    """Pages in a random order for sequences of `total` positions, and a cache of that size that
    holds quantised normal rows."""
    page, heads, dim = case["page"], case["kv_heads"], case["dim"]
    need = [-(-t // page) for t in total]
    spare = 3
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    width = max(need) if need else 1
    at = _ints(_offsets(need)[:-1])[:, None] + torch.arange(width, device=DEV, dtype=torch.int32)
    table = order[at.clamp(max=pages - 1).long()]  # past a sequence's last page: some other page's number
    cache = []
    for scale in (448.0, 437.0):
        pool = torch.randn((8192, dim), generator=gen, device=DEV) * _gain(gen, dim)
        codes, scales = _quantise(pool.bfloat16(), torch.tensor([scale], device=DEV))
        pick = torch.randint(0, 8192, (pages * heads * page,), generator=gen, device=DEV)
        cache += [codes[pick].view(pages, heads, page, dim // 2), scales[pick].view(pages, heads, page, dim // 16)]
    return tuple(cache), table.contiguous()


def _trees(seed, counts):
    """Ancestor masks of random trees: bit j of a token's mask says that it sees token j."""
    rng, masks = random.Random(seed), []
    for n in counts:
        mine = []
        for i in range(n):
            parent = rng.randint(max(-1, i - 5), i - 1)
            mine.append((mine[parent] if parent >= 0 else 0) | 1 << i)
        masks += [m - (1 << 64) if m >= 1 << 63 else m for m in mine]
    return _ints(masks, torch.int64)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = dict(case)
    new, ctx = _lengths(case)
    total = [a + b for a, b in zip(new, ctx)]
    rows, kv, dim = sum(new), case["kv_heads"], case["dim"]
    s["cu"] = _ints(_offsets(new))
    s["length"] = _ints(total)
    s["rows"] = rows
    if case["op"] == "prompt":
        s["cu_k"] = _ints(_offsets(total))
        s["q"] = _normal(gen, rows, case["heads"] * dim, _gain(gen, case["heads"] * dim)).view(rows, -1, dim)
        keys = sum(total)
        s["k"] = _normal(gen, keys, kv * dim, 1.0).view(keys, kv, dim)
        s["v"] = _normal(gen, keys, kv * dim, _gain(gen, kv * dim)).view(keys, kv, dim)
        s["most_q"], s["most_k"] = max(new), max(total)  # the plain form's padding
        return s
    s["cache"], s["table"] = _paged(case, gen, total)
    s["k_scale"], s["v_scale"] = (torch.tensor([x], device=DEV) for x in (448.0, 437.0))
    s["most"] = max(new)
    if case["op"] == "write":
        s["k"] = _normal(gen, rows, kv * dim, 1.0).view(rows, kv, dim)
        s["v"] = _normal(gen, rows, kv * dim, _gain(gen, kv * dim)).view(rows, kv, dim)
    if case["op"] == "cache":
        s["q"] = _normal(gen, rows, case["heads"] * dim, _gain(gen, case["heads"] * dim)).view(rows, -1, dim)
        s["mask"] = _trees(seed, new) if case["tree"] else None
    return s


# --------------------------------------------------------------------------- plain forms

def _quantise(y, gsf):
    """NVFP4 of bf16 y [..., dim]: packed codes and scale codes, each step rounded to 32 bits."""
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
    return code[..., 0::2] | code[..., 1::2] << 4, scale.view(torch.uint8)


def _values(codes, scales, gsf, dtype=torch.float32):
    """The values that codes [..., dim/2] and scales [..., dim/16] stand for."""
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=dtype, device=DEV)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    c = lut[c.int()].unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).to(dtype)[..., None]
    return (c / gsf.to(dtype)).flatten(-2)


def _slots(s):
    """Sequence, page and row inside the page of each new row."""
    r = torch.arange(s["rows"], device=DEV)
    b = torch.searchsorted(s["cu"][1:].contiguous(), r, right=True)
    new = s["cu"][1:] - s["cu"][:-1]
    p = s["length"][b] - new[b] + (r - s["cu"][b])
    return s["table"][b, p // s["page"]].long(), p % s["page"]


def _padded(x, cu, most):
    """Packed x [rows, ...] as [batch, most, ...] (rows past a sequence's end: some row), and which are its own."""
    at = torch.arange(most, device=DEV)
    mine = at < (cu[1:] - cu[:-1])[:, None]
    return x[(cu[:-1, None] + at).clamp(max=x.shape[0] - 1).long()], mine


def _attend(q, k, v, seen, dim):
    """q [B, n, H, D], k and v [B, KH, keys, D], seen [B, n, keys] -> o [B, n, H, D] and the log of the
    sum of exponentials [B, n, H], in 32 bits."""
    b, n, h, d = q.shape
    kh = k.shape[1]
    x = q.float().view(b, n, kh, h // kh, d).permute(0, 2, 3, 1, 4).reshape(b, kh, -1, d)
    s = (x @ k.transpose(-1, -2)).view(b, kh, h // kh, n, -1)
    s.mul_(dim ** -0.5).masked_fill_(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True).clamp(min=-3e38)
    e = s.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    o = (e.view(b, kh, -1, e.shape[-1]) @ v).view(b, kh, h // kh, n, d) / total.clamp(min=1e-38)
    lse = top.squeeze(-1) + total.squeeze(-1).log()
    return o.permute(0, 3, 1, 2, 4).reshape(b, n, h, d), lse.permute(0, 3, 1, 2).reshape(b, n, h)


def _plain_prompt(s):
    q, mine = _padded(s["q"], s["cu"], s["most_q"])
    k, there = _padded(s["k"], s["cu_k"], s["most_k"])
    v = _padded(s["v"], s["cu_k"], s["most_k"])[0]
    seen = there[:, None].expand(-1, q.shape[1], -1)
    if s["causal"]:  # the last query sees the last key
        shift = s["length"] - (s["cu"][1:] - s["cu"][:-1])
        i = torch.arange(q.shape[1], device=DEV)[:, None]
        seen = seen & (torch.arange(k.shape[1], device=DEV) <= i + shift[:, None, None])
    o, lse = _attend(q, k.float().transpose(1, 2), v.float().transpose(1, 2), seen, s["dim"])
    return o[mine].bfloat16(), lse[mine].t().contiguous()


def _plain_cache(s):
    k, v = (_values(c[s["table"].long()], f[s["table"].long()], g).transpose(1, 2).flatten(2, 3)
            for c, f, g in ((*s["cache"][:2], s["k_scale"]), (*s["cache"][2:], s["v_scale"])))
    q, mine = _padded(s["q"], s["cu"], s["most"])
    new = s["cu"][1:] - s["cu"][:-1]
    ctx = (s["length"] - new)[:, None, None]
    i = torch.arange(s["most"], device=DEV)
    at = torch.arange(k.shape[2], device=DEV)
    draft = at - ctx  # [B, 1, keys]: which drafted token a key is
    if s["mask"] is None:
        seen = draft <= i[:, None]
    else:
        bits = _padded(s["mask"], s["cu"], s["most"])[0][..., None] >> draft.clamp(0, 63)
        seen = (draft < 0) | ((bits & 1 == 1) & (draft < new[:, None, None]))
    o, lse = _attend(q, k, v, seen & (at < s["length"][:, None, None]), s["dim"])
    return o[mine].bfloat16(), lse[mine].t().contiguous()


def _plain_write(s):
    page, row = _slots(s)
    for x, g, codes, scales in ((s["k"], s["k_scale"], *s["cache"][:2]), (s["v"], s["v_scale"], *s["cache"][2:])):
        c, f = _quantise(x, g)
        codes[page, :, row] = c
        scales[page, :, row] = f
    return s["cache"]


def _plain_read(s):
    page, row = _slots(s)
    return [_values(codes[page, :, row], scales[page, :, row], g).bfloat16() for codes, scales, g in (
        (*s["cache"][:2], s["k_scale"]), (*s["cache"][2:], s["v_scale"]))]


# --------------------------------------------------------------------------- one pass

def run(s):
    if s["op"] == "write":
        if own:
            import nvfp4_activation_quantize_gb300 as h3q

            cache = h3q.h3q_kv_cache_write_nvfp4(s["k"], s["v"], s["cache"], s["cu"], s["length"], s["table"],
                                                 s["k_scale"], s["v_scale"])
        else:
            cache = _plain_write(s)
        # the whole cache: scales as the E4M3 numbers that they are, codes as they are packed
        return {"k_codes": cache[0], "k_scales": cache[1].view(torch.float8_e4m3fn), "v_codes": cache[2],
                "v_scales": cache[3].view(torch.float8_e4m3fn)}
    if s["op"] == "read":
        if own:
            import nvfp4_activation_quantize_gb300 as h3q

            k, v = h3q.h3q_kv_cache_read_nvfp4(s["cache"], s["cu"], s["length"], s["table"], s["k_scale"],
                                               s["v_scale"], rows=s["rows"])
        else:
            k, v = _plain_read(s)
        return {"k": k, "v": v}
    if not own:
        o, lse = _plain_prompt(s) if s["op"] == "prompt" else _plain_cache(s)
        return {"o": o, "lse": lse}
    import nvfp4_activation_quantize_gb300 as h3q

    lse = torch.empty((s["heads"], s["rows"]), dtype=torch.float32, device=DEV)
    if s["op"] == "prompt":
        o = h3q.h3q_attention_varlen(s["q"], s["k"], s["v"], s["cu"], s["cu_k"], causal=s["causal"], lse=lse)
    else:
        o = h3q.h3q_attention_cache_nvfp4(s["q"], s["cache"], s["cu"], s["length"], s["table"], s["k_scale"],
                                          s["v_scale"], max_rows=s["new_hi"], tree_mask=s["mask"], lse=lse)
    return {"o": o, "lse": lse}


# --------------------------------------------------------------------------- what it takes

def _seen_pairs(case):
    """(query, key) pairs of one head that a softmax runs over (a tree's drafts counted as a chain's)."""
    new, ctx = _lengths(case)
    if case["op"] == "prompt" and not case["causal"]:
        return sum(n * (n + c) for n, c in zip(new, ctx))
    return sum(n * c + n * (n + 1) // 2 for n, c in zip(new, ctx))


def work(case):
    new, ctx = _lengths(case)
    rows, total = sum(new), sum(new) + sum(ctx)
    kv, dim = case["kv_heads"], case["dim"]
    held = kv * (dim // 2 + dim // 16) * 2  # bytes of one position's key and value in the cache
    lists = 4 * (3 * case["batch"] + 1)
    if case["op"] == "write":
        return {"bytes": rows * (kv * dim * 4 + held) + lists, "flops": 0}
    if case["op"] == "read":
        return {"bytes": rows * (kv * dim * 4 + held) + lists, "flops": 0}
    h = case["heads"]
    outs = rows * h * (dim * 4 + 4)
    flops = 4 * dim * h * _seen_pairs(case)
    if case["op"] == "prompt":
        return {"bytes": outs + total * kv * dim * 4 + lists, "flops": flops}
    return {"bytes": outs + total * held + lists + 8 * rows * case["tree"], "flops": flops}


# --------------------------------------------------------------------------- the definition in 64 bits

def _exact_values(codes, scales, gsf):
    """fp64 values of codes and scales, from the formats' bit fields."""
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    e, m = (n >> 1) & 3, (n & 1).double()
    c = torch.where(e == 0, m / 2, (1 + m / 2) * torch.pow(2.0, (e - 1).double()))
    c = torch.where(n >= 8, -c, c)
    f = scales.long()
    e, m = (f >> 3) & 15, (f & 7).double()
    f = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.pow(2.0, (e - 7).double()))
    return c * f.repeat_interleave(16, -1) / gsf.double()


def _exact_scales(x, gsf):
    """E4M3(fl32(gsf * fl32(amax / 6))) of each block of 16, the rounding to E4M3 done on fp64."""
    a = x.double().abs().unflatten(-1, (-1, 16)).amax(-1)
    s = (gsf.double() * (a / 6).float().double()).float().double()
    step = torch.pow(2.0, torch.floor(torch.log2(s.clamp(min=2.0 ** -6))) - 3)
    return (torch.round(s / step) * step).clamp(max=448.0)


def _exact_row_values(s, b, count, first=0):
    at = np.arange(first, first + count)
    pages = s["table"][b].cpu().numpy()[at // s["page"]]
    page, row = torch.from_numpy(pages).long().to(DEV), torch.from_numpy(at % s["page"]).to(DEV)
    return [_exact_values(c[page, :, row], f[page, :, row], g) for c, f, g in (
        (*s["cache"][:2], s["k_scale"]), (*s["cache"][2:], s["v_scale"]))]


def exact(case, seed):
    new, ctx = _lengths(case)
    if case["op"] in ("prompt", "cache") and case["heads"] * case["dim"] * _seen_pairs(case) > 6e11:
        return None
    s = prepare(case, seed)
    cu = _offsets(new)
    if case["op"] == "write":
        page, row = _slots(s)
        out = {"k_codes": None, "v_codes": None}
        for name, x, g, held in (("k_scales", s["k"], s["k_scale"], s["cache"][1]),
                                 ("v_scales", s["v"], s["v_scale"], s["cache"][3])):
            f = held.view(torch.float8_e4m3fn).double()
            f[page, :, row] = _exact_scales(x, g)
            out[name] = f
        return out
    if case["op"] == "read":
        parts = [_exact_row_values(s, b, n) for b, n in enumerate(new)]
        return {"k": torch.cat([p[0] for p in parts]), "v": torch.cat([p[1] for p in parts])}
    outs, sums = [], []
    cu_k = _offsets([a + b for a, b in zip(new, ctx)])
    group = case["heads"] // case["kv_heads"]
    for b, (n, c) in enumerate(zip(new, ctx)):
        keys = n + c
        if case["op"] == "prompt":
            k, v = (s[x][cu_k[b]:cu_k[b + 1]].double() for x in "kv")
        else:
            k, v = _exact_row_values(s, b, keys)
        hidden = torch.zeros((n, keys), dtype=torch.bool, device=DEV)
        if case["op"] == "cache" and s["mask"] is not None:
            mine = s["mask"][cu[b]:cu[b + 1]].cpu().tolist()
            hidden[:, c:] = torch.tensor([[not (m >> j) & 1 for j in range(n)] for m in mine], device=DEV)
        elif case["op"] == "cache" or case["causal"]:
            hidden = torch.ones((n, keys), dtype=torch.bool, device=DEV).triu(c + 1)
        o = torch.empty((n, case["heads"], case["dim"]), dtype=torch.float64, device=DEV)
        total = torch.empty((case["heads"], n), dtype=torch.float64, device=DEV)
        for h in range(case["heads"]):
            t = s["q"][cu[b]:cu[b + 1], h].double() @ k[:, h // group].t() / math.sqrt(case["dim"])
            t.masked_fill_(hidden, -math.inf)
            total[h] = torch.logsumexp(t, 1)
            o[:, h] = torch.exp(t - total[h][:, None]) @ v[:, h // group]
        outs.append(o)
        sums.append(total)
    return {"o": torch.cat(outs), "lse": torch.cat(sums, 1)}
