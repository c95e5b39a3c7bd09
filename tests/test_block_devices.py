"""The sources of the calls over blocks take the number of SMs from the device."""
import os
import re

import pytest

from nvfp4_activation_quantize_gb300 import build as libbuild


@pytest.mark.parametrize("name", ["select_blocks.cu", "attention_blocks.cu", "qkv_axes.cu", "postnorm.cu"])
def test_no_number_of_sms_in_the_code(name):
    text = re.sub(r"//.*", "", open(os.path.join(libbuild.CSRC, name)).read())
    assert not re.search(r"\b(76|152|304|456)\b", text)
