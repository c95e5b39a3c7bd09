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
