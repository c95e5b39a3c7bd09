"""Inputs and plain forms that the tests of the paged cache and of attention share."""
from __future__ import annotations

import numpy as np
import torch

import oracle

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float32)


def ints(values, dev, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=dev)


def offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)


def bits(t):
    return t.detach().contiguous().cpu().view(torch.int16).numpy().view(np.uint16)


def paged(dev, lengths, page, seed, spare=2):
    """A block table for sequences of these lengths with their pages in a random order, the
    entries past a sequence's end naming no page; returns (table, pages)."""
    need = [max(0, -(-n // page)) for n in lengths]
    rng = np.random.default_rng(seed)
    pages = sum(need) + spare
    order = rng.permutation(pages)
    table = np.full((len(lengths), max(need + [1])), -7, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return ints(table.tolist(), dev), pages


def random_cache(dev, pages, heads, page, dim, seed):
    """A cache of any bytes: every code, scale bytes up to 448 and also those with all ones."""
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return tuple(torch.randint(0, 256 if per == 2 else 128, (pages, heads, page, dim // per), generator=g, device=dev,
                               dtype=torch.uint8) for per in (2, 16, 2, 16))


def row_places(cu, kv_len, table, page, pages, rows):
    """(row, page, row in page) of the packed rows that have a place, and the rows that a sequence owns."""
    cu, kv_len, table = (np.asarray(t.cpu() if hasattr(t, "cpu") else t) for t in (cu, kv_len, table))
    places, owned = [], []
    for b in range(len(kv_len)):
        for r in range(cu[b], min(cu[b + 1], rows)):
            owned.append(r)
            p = int(kv_len[b]) - int(cu[b + 1]) + r
            if p < 0 or p // page >= table.shape[1]:
                continue
            n = int(table[b, p // page])
            if 0 <= n < pages:
                places.append((r, n, p % page))
    return places, owned


def written(cache, x, gsf, which, places):
    """The codes and scales (numpy) of cache tensors `which` after the rows' write."""
    codes, scales = (cache[2 * which + i].cpu().numpy().copy() for i in (0, 1))
    rows, heads, dim = x.shape
    c, s = oracle.quantize_rows(bits(x).reshape(rows, heads * dim), gsf)
    for r, page, at in places:
        codes[page, :, at] = c[r].reshape(heads, dim // 2)
        scales[page, :, at] = s[r].reshape(heads, dim // 16)
    return codes, scales


def values32(codes, scales, gsf):
    """fl((E2M1 * E4M3) / gsf), from numpy codes [..., dim/2] and scales [..., dim/16]."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = E2M1[c & 7] * np.where(c & 8, np.float32(-1), np.float32(1))
    s = scales.astype(np.int32) & 127
    f = np.where(s >> 3 == 0, (s & 7) * 2.0 ** -9, (1 + (s & 7) / 8) * 2.0 ** ((s >> 3) - 7.0)).astype(np.float32)
    return (v * np.repeat(f, 16, -1)) / np.float32(gsf)


def cache_values64(cache, gs, table_row, length, page):
    """k and v [length, heads, dim] in 64 bits of one sequence's positions (on the cache's device)."""
    at = np.arange(length)
    pages = torch.as_tensor(np.asarray(table_row.cpu())[at // page].astype(np.int64), device=cache[0].device)
    row = torch.as_tensor(at % page, device=cache[0].device)
    lut = torch.tensor(np.concatenate([E2M1, -E2M1]).astype(np.float64), device=cache[0].device)
    out = []
    for t in (0, 1):
        codes, scales = cache[2 * t][pages, :, row], cache[2 * t + 1][pages, :, row].long() & 127
        c = lut[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()]
        e, m = scales >> 3, (scales & 7).double()
        f = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.pow(2.0, (e - 7).double()))
        out.append(c * f.repeat_interleave(16, -1) / gs[t])
    return out


def attention64(q, k, v, seen, scale):
    """Attention of q [n, H, D] over k, v [keys, KH, D] in 64 bits where seen [n, keys]: o [n, H, D], lse [H, n],
    and what the tolerances need: w|v| [n, H, D] and the largest sum of |products| in units of log2."""
    n, heads, dim = q.shape
    group = heads // k.shape[1]
    q, k, v = q.double(), k.double().repeat_interleave(group, 1), v.double().repeat_interleave(group, 1)
    x = torch.einsum("nhd,khd->hnk", q, k) * scale
    if k.shape[0] == 0:
        zero = torch.zeros((n, heads, dim), dtype=torch.float64, device=q.device)
        return zero, torch.full((heads, n), -np.inf, dtype=torch.float64, device=q.device), zero, 0.0
    size = float((torch.einsum("nhd,khd->hnk", q.abs(), k.abs())).max()) * scale * 1.4427
    x = x.masked_fill(~seen[None], -np.inf)
    lse = torch.logsumexp(x, -1)
    w = torch.where(seen[None], torch.exp(x - lse[..., None].clamp(min=-1e300)), torch.zeros_like(x))
    return torch.einsum("hnk,khd->nhd", w, v), lse, torch.einsum("hnk,khd->nhd", w, v.abs()), size


def check_attention(o, lse, ref, keys, weight_step, what=""):
    """o and lse against attention64's answer.  The output is rounded once to bf16 (2^-8 of it).  Each weight
    has a relative error of its own rounding (weight_step, 0 where it is not rounded), and of its exponent:
    fp32 sums of at most 256 products err by 2^-19 of the sum of magnitudes at most (16 steps of four
    roundings of 2^-23 or better), the power of two by 2^-22, and the running sums over `keys` / 16 steps by 2^-22
    each.  An error e of all weights moves the output by at most 2 e sum(w |v|): numerator and denominator."""
    want, want_lse, spread, size = ref
    e = weight_step + 2.0 ** -19 * (size + 8) + 2.0 ** -22 * (keys / 16 + 8)
    tol = want.abs() * 2.0 ** -8 + 2 * e * spread * (1 + 2.0 ** -8) + 1e-38
    err = (o.double() - want).abs()
    assert bool((err <= tol).all()), f"{what}: o off by {float((err / tol).max()):.3g} of what is allowed"
    empty = torch.isinf(want_lse)
    assert bool((lse[empty] == -np.inf).all()), f"{what}: lse of rows that see nothing"
    err = (lse.double() - want_lse)[~empty].abs()
    allowed = 2 * (e - weight_step) + want_lse[~empty].abs() * 2.0 ** -22
    assert bool((err <= allowed).all()), f"{what}: lse off by {float((err / allowed).max()):.3g} of what is allowed"
