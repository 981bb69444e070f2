"""Launch shapes follow the device's SM count: no file of the library has that of one chip
in its code but num_sms, which falls back to it where the driver gives none."""
import os
import re

import pytest

import structured_sparse_gemm_compress_b200 as nm

CSRC = os.path.join(os.path.dirname(os.path.abspath(nm.__file__)), "csrc")


@pytest.mark.parametrize("name", sorted(os.listdir(CSRC)))
def test_no_sm_count_of_one_chip(name):
    text = re.sub(r"/\*.*?\*/|//[^\n]*", "", open(os.path.join(CSRC, name)).read(), flags=re.S)
    text = re.sub(r"int num_sms\(int dev\) \{.*?\n\}", "", text, flags=re.S)
    assert not re.search(r"\b(148|74)\b", text)
