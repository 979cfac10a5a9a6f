"""Launches of the layer operators go by the device's number of SMs, not by a number
written into the code (no GPU needed)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w8a8_quantized_matmul_b200", "csrc")


@pytest.mark.parametrize("name", ["adapter.cu", "row_ops.cu", "scaled_matmul.cu"])
def test_no_number_of_sms_in_the_code(name):
    src = open(os.path.join(CSRC, name)).read()
    code = re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", src, flags=re.S))
    assert not re.search(r"(?<![\w.])(?:148|132|144)(?![\w.])", code)
