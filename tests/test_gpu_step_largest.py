"""The largest counts of rows and ids that the calls take: host sums of them stay in range."""
import math

import pytest
import torch

from gpu_util import qmv
from test_gpu_step import BF16, F16

pytestmark = pytest.mark.gpu

MOST = 2 ** 31 - 1


def test_softmax_over_as_many_ids_as_an_int_holds():
    V = MOST
    x = torch.zeros(1, V, dtype=F16, device="cuda")
    at = torch.tensor([0, 1, 134217727, 134217728, 2013265919, 2013265920, V - 2, V - 1], device="cuda")
    x[0, at[1::2]] = 1.0
    x[0, 77:1077] = -math.inf
    out = torch.full((1, V), -1.0, device="cuda")
    qmv().qmv_softmax(x, out=out)
    total = V - 1000 - 4 + 4 * math.e
    # A thread adds 2^18 terms relative to its warp's maximum (16 CTAs of 512 threads). Where that
    # is 0 the terms are ones, added exactly. In the at most four of 256 warps where it is 1 they are
    # exp(-1), each added with a rounding of at most 2^-24 of the sum so far: 2^18 * 2^-24 = 2^-6 of
    # that warp's sum, and its places are 2^-8 of all, so at most 4 * 2^-8 * 2^-6 of the total.
    # What joins the threads, warps and CTAs has ten roundings, exp2 and its argument six units
    # more, the quotient one
    rel = 2.0 ** -12 + 20 * 2.0 ** -24
    got = out[0, at].double().cpu()
    for i, v in enumerate(got):
        ref = (math.e if i % 2 else 1.0) / total
        assert abs(float(v) - ref) <= ref * rel, i
    assert not bool(out[0, 77:1077].any())
    for lo in range(0, V, 2 ** 28):            # every place is written
        assert bool((out[0, lo:lo + 2 ** 28] >= 0).all())


def test_norms_of_as_many_rows_as_an_int_holds():
    M = MOST
    y = torch.full((M, 1), 0.5, dtype=BF16, device="cuda")
    r = torch.full((M, 1), 1.5, dtype=BF16, device="cuda")
    at = torch.tensor([0, 7, 8, 2 ** 30, M - 8, M - 2, M - 1], device="cuda")
    r[at] = -4.5
    one = torch.ones(1, dtype=BF16, device="cuda")
    h, z = torch.zeros(M, 1, dtype=BF16, device="cuda"), torch.zeros(M, 1, dtype=BF16, device="cuda")
    qmv().qmv_block_norm(y, r, one, h_out=h, out=z)
    # h = 2 or -4, z = h / |h| but for eps, which a rounding to bf16 takes away
    assert bool((h[at] == -4).all()) and bool((z[at] == -1).all())
    for lo in range(0, M, 2 ** 28):
        n = int(((at >= lo) & (at < lo + 2 ** 28)).sum())
        assert int((h[lo:lo + 2 ** 28] == 2).sum()) == min(2 ** 28, M - lo) - n
        assert int((z[lo:lo + 2 ** 28] == 1).sum()) == min(2 ** 28, M - lo) - n
