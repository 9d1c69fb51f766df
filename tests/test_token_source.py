"""What the sources of the decode-step kernels hold to and no run can show."""
import os
import re

from conftest import ROOT

KERNELS = {"qmv_rope.cu": 1, "qmv_route.cu": 1, "qmv_draw.cu": 1, "qmv_experts.cu": 2, "qmv_experts.cuh": 1}


def source(name):
    with open(os.path.join(ROOT, "bit_weight_only_packed_gb300", "csrc", name)) as f:
        return f.read()


def kernels_of(text):
    return re.findall(r"\n__global__ .*?\n\}\n", text, re.S)


def test_every_kernel_waits_for_the_one_before_and_then_lets_the_next_one_start():
    for name, n in KERNELS.items():
        text = source(name)
        assert "griddepcontrol" not in text, name
        kernels = kernels_of(text)
        assert len(kernels) == n, name
        for k in kernels:
            assert "pdl_begin();" in k, name
    # the products wait at one of two places, by one condition
    k = kernels_of(source("qmv_experts.cuh"))[0]
    assert k.count("pdl_begin();") == 2
    assert "if (!ahead) pdl_begin();" in k and re.search(r"if \(ahead\) \{\n\s*pdl_begin\(\);", k)
    # where x comes from the kernel before, it is fetched behind the wait
    assert "if (!ahead && warp == 0 && segs > 0) issue_x(0);" in k
    late = k[k.index("if (ahead) {"):]
    assert late.index("pdl_begin();") < late.index("issue_x(0);")


def test_no_thread_leaves_before_that_wait():
    # one that did would count as having waited, and the next kernel might start too early
    for name in KERNELS:
        for k in kernels_of(source(name)):
            assert not re.search(r"\n\s*(if \([^\n]*\) )?return;", k[:k.index("pdl_begin();")]), name


def test_waits_of_the_products_are_bounded():
    k = kernels_of(source("qmv_experts.cuh"))[0]
    assert not re.search(r"while \(!?pipe::", k)
    assert len(re.findall(r"mbar_wait_fast\(", k)) == 2 and len(re.findall(r"mbar_drain\(", k)) == 2


def test_a_cta_of_a_cluster_stays_until_nobody_reaches_into_it():
    # stores to other CTAs end with a meeting of all before anyone may return
    k = kernels_of(source("qmv_draw.cu"))[0]
    tell = re.search(r"const auto tell = .*?\n  \};", k, re.S).group(0)
    assert tell.index("st_cluster64") < tell.index("meet();")
    few = k[k.index("gather(told);\n        in_order(n);\n        u64 w[4], sum"):]
    assert few.index("if (C > 1) meet();") < few.index("return;")
