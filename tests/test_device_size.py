"""The products', quantisers' and rotation's launch shapes, and the models that
choose them, hold no SM count of their own: the device is asked."""
import os
import re

import pytest

from tests.test_abi import ROOT


def code_of(path):
    """A source without its comments."""
    src = open(path).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return re.sub(r"//[^\n]*", "", src)


@pytest.mark.parametrize("name", ["i8_linear.cu", "q8_linear.cu", "quant.cu", "rope_axes.cu", "common.cuh"])
def test_no_sm_count_is_written_into_the_source(name):
    code = code_of(os.path.join(ROOT, "transformer_encoder_forward_gb300", "csrc", name))
    # 148: what sm_count() falls back to without a device
    assert set(re.findall(r"\b1[45][0-9]\b", code)) <= {"148"}
