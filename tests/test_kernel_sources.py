"""Rules that the attention kernels' sources keep, where breaking them shows on a GPU only as a rare hang or
fault."""
import os
import re

import pytest

from nvfp4_activation_quantize_gb300 import build as libbuild


def _source(name):
    text = open(os.path.join(libbuild.CSRC, name)).read()
    return re.sub(r"//.*", "", text)


ATTENTION = ["attention.cu", "attention_cache.cu", "attention_cache_wide.cu"]


@pytest.mark.parametrize("name", ATTENTION)
def test_giving_up_is_one_decision(name):
    """The abort flag may rise between two lanes' reads: it is read through raised (one answer for the warp), or
    raised_here where what follows is one lane's own."""
    text = _source(name)
    assert "raised" in text and not re.search(r"\*abort(?!\s*=[^=])", text)


@pytest.mark.parametrize("name", ["attention.cu", "attention_cache_wide.cu"])
def test_products_are_drained_on_every_way_out(name):
    """The TMEM is freed after the last product whether or not a role gave up: no branch before the drain."""
    text = _source(name)
    at = text.index("commit_elected(bar_drain)")
    assert text[:at].rstrip().endswith("}") and "wait_bounded(bar_drain, 0)" in text[at:at + 120]


def test_outputs_are_read_only_after_their_products():
    """A role that gave up touches no TMEM: another may still write it, or not have been given it yet."""
    text = _source("attention_cache_wide.cu")
    reads = [m.start() for m in re.finditer(r"tc_load32\(taddr_o \+ i, o\)", text)]
    assert len(reads) == 2   # the rescaling, inside a tile whose wait was met, and the join
    assert re.search(r"if \(ok && rows && [^{]*\{\s*$", text[:reads[1]])


@pytest.mark.parametrize("name", ["kv_cache.cu", "attention_cache.cu", "attention_cache_wide.cu", "attention_cache.cuh"])
def test_kernels_launched_early_read_coherently(name):
    """A kernel that is resident while the one before it still writes makes no load that promises constant data."""
    text = _source(name)
    assert "after_stream()" in text
    assert not re.search(r"ld\.global\.nc|load_stream\(|load_reused\(|load16_stream\(|load16_reused\(|__ldg|__restrict__", text)


def test_a_warp_that_gave_up_gives_no_slot_back():
    """A slot whose copy was not waited for may still be written: it is not filled again."""
    text = _source("attention_cache.cu")
    gives = re.findall(r"if \(([^;]*?)\) mbar_arrive\(bar_empty", text)
    assert len(gives) == 1 and "alive" in gives[0]
