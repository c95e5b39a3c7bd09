"""Rules that the sources of attention over blocks and of block selection keep, where breaking them shows on a GPU only
as a rare hang or fault."""
import os
import re

from nvfp4_activation_quantize_gb300 import build as libbuild


def _source(name):
    return re.sub(r"//.*", "", open(os.path.join(libbuild.CSRC, name)).read())


def test_giving_up_is_one_decision():
    """The abort flag may rise between two lanes' reads: it is read through raised_here where what follows is one
    lane's own, or after a vote."""
    text = _source("attention_blocks.cu")
    assert "raised_here" in text and not re.search(r"\*abort(?!\s*=[^=])", text)


def test_products_are_drained_on_every_way_out():
    text = _source("attention_blocks.cu")
    at = text.index("commit_elected(bar_drain)")
    assert text[:at].rstrip().endswith("}") and "wait_bounded(bar_drain, 0)" in text[at:at + 120]


def test_every_wait_is_bounded():
    for name in ("attention_blocks.cu", "select_blocks.cu", "qkv_axes.cu", "postnorm.cu"):
        text = _source(name)
        assert not re.search(r"mbarrier\.(try|test)_wait", text)   # (the bounded ones are in a header)
        for loop in re.findall(r"while \(!?mbar_try_wait", text):
            raise AssertionError(f"{name}: {loop}")


def test_sums_are_waited_for():
    """The kernel of scores starts before the sums are there: it reads none of them before it has waited."""
    text = _source("select_blocks.cu")
    kernel = text[text.index("score_kernel(const __grid_constant__"):]
    waits = kernel.index("griddepcontrol.wait")
    assert "sums.hi" not in kernel[:waits] and "sums.size" not in kernel[:waits]
    assert not re.search(r"ld\.global\.nc|load16_stream|load16_reused|__ldg|__restrict__",
                         text[text.index("struct ScoreArgs"):])
