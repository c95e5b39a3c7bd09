"""Inputs and plain forms that the tests of block selection and of attention over blocks share."""
from __future__ import annotations

import math

import numpy as np
import torch

import cache_cases as cc


def sequences(dev, seqs, heads, kv_heads, dim, seed=0, packed=False, tail=3):
    """Inputs for sequences of (queries, keys); the last `tail` rows belong to none."""
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def rows(n, h):
        x = torch.randn((n, (2 if packed else 1) * h * dim), generator=g, device=dev).bfloat16()
        return (x[:, h * dim:] if packed else x).unflatten(1, (h, dim))

    nq, nk = [a for a, _ in seqs], [b for _, b in seqs]
    return {"q": rows(sum(nq) + tail, heads), "k": rows(sum(nk) + tail, kv_heads), "v": rows(sum(nk) + tail, kv_heads),
            "cu_q": cc.ints(cc.offsets(nq).tolist(), dev), "cu_k": cc.ints(cc.offsets(nk).tolist(), dev)}


def query_blocks(c, block_q):
    """(list row, sequence, first query, one past its last) of every query block."""
    cu = c["cu_q"].tolist()
    for b in range(len(cu) - 1):
        n = cu[b + 1] - cu[b]
        for i in range(-(-n // block_q)):
            yield cu[b] // block_q + b + i, b, i * block_q, min(n, (i + 1) * block_q)


def counted(entries, blocks):
    """The entries of a list that count: numbers of blocks, above all before them that do."""
    got = []
    for e in entries:
        if 0 <= e < blocks and (not got or e > got[-1]):
            got.append(e)
    return got


def random_lists(c, kv_heads, block_q, block_k, top, seed, junk=False):
    """Lists of random blocks in ascending order, some shorter than others; with `junk` also numbers of no block,
    repeated ones and ones out of order."""
    rng = np.random.default_rng(seed)
    rows = c["q"].shape[0] // block_q + c["cu_q"].shape[0] - 1
    lists = np.full((kv_heads, rows, top), -1, np.int64)
    cu_k = c["cu_k"].tolist()
    for r, b, _, _ in query_blocks(c, block_q):
        blocks = -(-(cu_k[b + 1] - cu_k[b]) // block_k)
        for h in range(kv_heads):
            n = int(rng.integers(0, min(top, blocks) + 1)) if rng.random() < 0.3 else min(top, blocks)
            mine = np.sort(rng.permutation(blocks)[:n])
            if junk:
                mine = np.concatenate([mine, rng.integers(-5, blocks + 5, top)])[:top]
                mine = np.where(rng.random(len(mine)) < 0.2, rng.choice([-1, -2 ** 31, 2 ** 31 - 1, blocks, 0]), mine)
                if rng.random() < 0.3:
                    mine = rng.permutation(mine)
            lists[h, r, :len(mine)] = mine
    return torch.from_numpy(lists.astype(np.int32)).to(c["q"].device)


def check_blocks(c, lists, block_q, block_k, causal, out, lse, scale=None, what="", weight=2.0 ** -8):
    """out and lse of attention over the lists, against the formula in 64 bits."""
    dim = c["q"].shape[2]
    scale = dim ** -0.5 if scale is None else scale
    cu_q, cu_k, kv_heads = c["cu_q"].tolist(), c["cu_k"].tolist(), c["k"].shape[1]
    group = c["q"].shape[1] // kv_heads
    host = lists.cpu().tolist()
    for r, b, first, last in query_blocks(c, block_q):
        n, keys = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        at = slice(cu_q[b] + first, cu_q[b] + last)
        for h in range(kv_heads):
            listed = [p for j in counted(host[h][r], -(-keys // block_k))
                      for p in range(j * block_k, min(keys, (j + 1) * block_k))]
            p = torch.tensor(listed, dtype=torch.int64, device=out.device)
            k, v = (c[x][cu_k[b]:cu_k[b + 1], h:h + 1][p] for x in "kv")
            t = torch.arange(first, last, device=out.device)[:, None]
            seen = p <= t + (keys - n) if causal else torch.ones((last - first, len(listed)), dtype=torch.bool,
                                                                 device=out.device)
            heads = slice(h * group, (h + 1) * group)
            ref = cc.attention64(c["q"][at, heads], k, v, seen, scale)
            cc.check_attention(out[at, heads], lse[heads, at], ref, len(listed), weight,
                               f"{what} sequence {b} queries {first} head {h}")


def selected(c, top, block_q, block_k, causal, first):
    """The lists and scores that the definition gives, in 64 bits: lists [kv_heads, rows, top], scores the same."""
    kv_heads = c["k"].shape[1]
    cu_q, cu_k = c["cu_q"].tolist(), c["cu_k"].tolist()
    rows = c["q"].shape[0] // block_q + len(cu_q) - 1
    lists = np.full((kv_heads, rows, top), -1, np.int64)
    scores = np.full((kv_heads, rows, top), -np.inf)
    sums = {}
    for b in range(len(cu_k) - 1):
        keys = c["k"][cu_k[b]:cu_k[b + 1]].double()
        sums[b] = [(x.sum(0).cpu().numpy(), x.shape[0]) for x in keys.split(block_k)] if len(keys) else []
    for r, b, lo, hi in query_blocks(c, block_q):
        n, keys = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        q = c["q"][cu_q[b] + lo:cu_q[b] + hi].double()
        q = q.unflatten(1, (kv_heads, -1)).sum((0, 2)).cpu().numpy()
        size = (hi - lo) * (c["q"].shape[1] // kv_heads)
        begin = keys - n + lo   # position of the first query
        end = min(keys, begin + hi - lo) if causal else keys
        candidates = -(-end // block_k) if end > 0 else 0
        for h in range(kv_heads):
            ranked = []
            for j in range(candidates):
                s, count = sums[b][j]
                score = float((q[h] * s[h]).sum()) / count
                always = j < first or (causal and min((j + 1) * block_k, keys) > begin)
                rank = math.inf if always else -math.inf if math.isnan(score) else score
                ranked.append((-rank, j, score / size))
            chosen = sorted(sorted(ranked)[:top], key=lambda x: x[1])
            for at, (_, j, score) in enumerate(chosen):
                lists[h, r, at] = j
                scores[h, r, at] = score
    return lists, scores
