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
