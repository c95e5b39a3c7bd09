"""GPU: block selection with more than 16,000 key blocks: of sequences that are short each, and of one that has so many
by itself, whose scores are kept in the workspace."""
import pytest
import torch

import block_cases as bc
import nvfp4_activation_quantize_gb300 as h3q
from test_gpu_select_many_lists import check, dev  # noqa: F401

pytestmark = pytest.mark.gpu

CASES = [  # (queries, keys) of the sequences, query heads, key heads, dim, top
    ([(1, 70_000)] * 16, 8, 2, 64, 16),                              # 1,094 blocks each, 17,504 in all
    ([(300, 1_100_005), (70, 300), (1, 1_060_000)], 2, 1, 64, 50),   # 17,188 and 16,563 by themselves
    ([(130, 1_100_000)], 1, 1, 128, 300),                            # the only one
    ([(200, 1_025_000), (60, 60)], 4, 2, 64, 9),                     # 16,016: a CTA holds them, 16,017 do not fit the rest
    ([(5000, 1_060_000)] + [(64, 64)] * 300, 48, 48, 64, 12),        # more CTAs than the workspace has rows
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("causal, first", [(False, 0), (True, 3)])
def test_against_the_definition(dev, case, causal, first):  # noqa: F811
    seqs, heads, kv_heads, dim, top = CASES[case]
    c = bc.sequences(dev, seqs, heads, kv_heads, dim, seed=80 + case)
    assert c["k"].shape[0] // 64 > 16_000
    check(c, top, 64, 64, causal, first)


def test_ties_and_numbers_that_are_none(dev):  # noqa: F811
    """Equal blocks of a long sequence, among them some of no numbers."""
    c = bc.sequences(dev, [(64, 64 * 17_000)], 1, 1, 64, seed=90, tail=0)
    k = c["k"].view(17_000, 64, 64)
    k[5:] = k[torch.arange(5, 17_000, device=dev) % 5]
    k[2::1000] = float("nan")
    none = set(range(2, 17_000, 1000))
    score = (k[:5].double().sum(1) @ c["q"].double().view(64, 64).sum(0)).nan_to_num(-float("inf"))
    score[2] = k[7].double().sum(0) @ c["q"].double().view(64, 64).sum(0)
    ranked = [j for p in score.sort(descending=True).indices.tolist() for j in range(p, 17_000, 5) if j not in none]
    for top in (40, 4096):
        lists = h3q.h3q_select_blocks(c["q"], c["k"], c["cu_q"], c["cu_k"], top, block_q=64, block_k=64)
        assert lists[0, 0].tolist() == sorted(ranked[:top])


def test_graph_and_workspace_of_any_contents(dev):  # noqa: F811
    c = bc.sequences(dev, [(100, 1_050_000), (100, 30_000)], 2, 2, 64, seed=91)
    nbytes = h3q.select_blocks_workspace_bytes(c["q"].shape[0], c["k"].shape[0], 2, 2, 64, 64, 64)
    guard = 4096
    whole = torch.full((nbytes + guard,), 255, dtype=torch.uint8, device=dev)
    lists = torch.empty((2, h3q.block_rows(c["q"].shape[0], 2, 64), 9), dtype=torch.int32, device=dev)

    def call():
        h3q.h3q_select_blocks(c["q"], c["k"], c["cu_q"], c["cu_k"], 9, block_q=64, block_k=64, causal=True, first=1,
                              blocks=lists, workspace=whole[:nbytes])

    call()
    want = lists.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    whole.fill_(127)
    lists.zero_()
    graph.replay()
    assert torch.equal(lists, want) and bool((whole[nbytes:] == 127).all())
