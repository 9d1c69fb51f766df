"""What the sources of the verification-step kernels hold to and no run can show."""
import os
import re

from conftest import ROOT


def source(name):
    with open(os.path.join(ROOT, "bit_weight_only_packed_gb300", "csrc", name)) as f:
        return f.read()


def test_what_the_ctas_of_a_cluster_store_to_each_other_is_aligned():
    # a 16-byte store needs a 16-byte address wherever the array comes to lie
    text = source("qmv_sample.cu")
    assert re.search(r"struct alignas\(16\) Part \{", text)
    assert "static_assert(sizeof(Part) == 16 && alignof(Part) == 16" in text
    # the other exchange is 8 bytes of an array of 8-byte numbers
    assert re.search(r"long long [^;]*parts\[2\]\[MAX_C\]", text)
