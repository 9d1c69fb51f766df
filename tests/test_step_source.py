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


def test_dependents_start_after_the_wait():
    # A matvec with early weights reads them ahead of its own wait. It may do so because the
    # kernel before it let it start only after all kernels before that one had ended; one that
    # lets its dependents start first would let them read weights that are still being written.
    texts = {n: source(n) for n in ("qmv_step.cuh", "qmv_norm.cu", "qmv_sample.cu", "qmv_w4_gemv.cuh", "qmv_w4.cu")}
    assert texts["qmv_step.cuh"].index("griddepcontrol.wait;\"") < texts["qmv_step.cuh"].index("griddepcontrol.launch_dependents;\"")
    assert sum(t.count("griddepcontrol.launch_dependents;") for t in texts.values()) == 1
    # every kernel goes through it: the softmaxes, the verification, the norms, the matvec
    for name, kernels in (("qmv_norm.cu", 3), ("qmv_sample.cu", 3), ("qmv_w4_gemv.cuh", 1)):
        assert texts[name].count("pdl_begin();") == kernels, name


def test_a_cta_whose_wait_ran_out_stays_until_nobody_stores_to_it():
    # The CTAs of a cluster store to each other's shared memory; one that ended after a wait that
    # ran out, while another has yet to store, would be stored to after its end.
    text = source("qmv_sample.cu")
    leave = re.search(r"void exchange_leave\(.*?\n\}", text, re.S).group(0)
    assert leave.index("cluster_arrive();") < leave.index("cluster_wait();") < leave.index("mbar_drain(")
    kernels = re.findall(r"\n__global__ .*?\n\}\n", text, re.S)
    waits = 0
    for k in kernels:
        if "exchange_begin(" not in k:
            continue
        # between the wait for the others' values and the next use of them
        for m in re.finditer(r"mbar_wait_fast\(&all_here", k):
            after = k[m.start():m.start() + 600]
            assert re.search(r"return exchange_leave\(", after), after
            waits += 1
        # no other way out once the exchange has begun
        body = k[k.index("exchange_begin("):]
        assert not re.search(r"\breturn;", body)
    assert waits == 2
