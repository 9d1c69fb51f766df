"""Values at the ends of their types: infinities, NaN and overflow in the 4-bit matvec for
both types of x, with a cluster along k and with x at any element; the smallest numbers of
bf16; NaN in the draft's probabilities."""
import numpy as np
import pytest
import torch

from gpu_util import qmv
from test_gpu_step import BF16, F16, F32, Padded, gen, make_w4, probs, ref_verify, run_verify

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("xdt", [F16, BF16])
# the second: two strips of 128 blocks, which eight CTAs along k share (16 blocks a CTA)
@pytest.mark.parametrize("N,K,group", [(64, 512, 128), (60, 16384, 64), (3000, 1056, 32)])
def test_w4_infinities_and_nan(N, K, group, xdt, shift):
    M = 9
    p, _, w = make_w4(N, K, group, True, F16, 13)
    x = Padded(M, K, xdt, ld=K + shift, shift=shift)
    x.t.copy_(torch.randn(M, K, generator=gen(2), device="cuda"))
    clean = qmv().qmv_w4_gemv(p, x.t)
    x.t[1, K - 5] = NAN
    x.t[3, 17], x.t[3, K // 2] = INF, INF
    x.t[4, 40] = -INF
    x.t[6, 3], x.t[6, K - 3] = INF, -INF           # in the shares of two CTAs
    x.t[8, K - 1] = NAN
    y = qmv().qmv_w4_gemv(p, x.t)
    bad = [1, 3, 4, 6, 8]
    # the definition: a product with a weight of 0 is NaN, and so is a sum of both infinities
    ref = torch.stack([(x.t[m].double() * w).sum(1) for m in bad])
    got = y[bad].double()
    assert torch.equal(got.isnan(), ref.isnan())
    assert torch.equal(got.nan_to_num(7.0, 8.0, 9.0), ref.nan_to_num(7.0, 8.0, 9.0))
    keep = [m for m in range(M) if m not in bad]
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("N,K", [(64, 512), (60, 16384)])
def test_w4_sums_at_the_end_of_fp32(N, K):
    # weights of 0 .. 15 (zero points of 0): one column whose sums pass fp32's largest, one of
    # -3e38 whose single weight keeps it there, ordinary ones beside them
    g = gen(5)
    codes = torch.randint(1, 16, (N, K), generator=g, device="cuda", dtype=torch.uint8)
    codes[:, 7] = 1
    z = torch.zeros(N, K // 128, device="cuda", dtype=torch.uint8)
    p = qmv().W4Pack(N, K, 128, BF16, True).pack_weights(codes, torch.ones(N, K // 128, device="cuda", dtype=BF16), z)
    x = torch.randint(-2, 3, (4, K), generator=g, device="cuda").to(BF16)
    x[1] = 1e37
    x[2] = 0
    x[2, 7] = -3e38
    y = qmv().qmv_w4_gemv(p, x)
    ref = x.double() @ codes.double().t()
    assert bool((y[1] == INF).all())
    assert torch.equal(y[2].double(), ref[2]) and torch.equal(y[[0, 3]].double(), ref[[0, 3]])


@pytest.mark.parametrize("e", [-133, -128, -120, -112])
def test_w4_smallest_bf16_columns_are_exact(e):
    # Whole numbers up to 255 times 2^e: bf16 has nothing between the multiples of 2^-133, so
    # a column's scaling, by 2^126 at most, leaves multiples of 2^-7 or more, of which fp16 holds
    # the first 255 exactly. Sums stay below
    # 255 * 15 * 2048 < 2^23 units: exact in fp32 in any order, subnormal ones too.
    N, K = 130, 2048
    codes = torch.randint(0, 16, (N, K), generator=gen(6), device="cuda", dtype=torch.uint8)
    z = torch.randint(0, 16, (N, K // 64), generator=gen(7), device="cuda", dtype=torch.uint8)
    p = qmv().W4Pack(N, K, 64, BF16, True).pack_weights(codes, torch.ones(N, K // 64, device="cuda", dtype=BF16), z)
    whole = torch.randint(-255, 256, (3, K), generator=gen(8), device="cuda").double()
    whole[1] = whole[1].clamp(-1, 1)
    x = (whole * 2.0 ** e).to(BF16)
    assert torch.equal(x.double(), whole * 2.0 ** e)
    w = codes.double() - z.double().repeat_interleave(64, 1)
    y = qmv().qmv_w4_gemv(p, x)
    assert torch.equal(y.double(), (whole @ w.t()) * 2.0 ** e)


@pytest.mark.parametrize("V", [600, 4099])
def test_verify_nan_in_the_drafts_probabilities(V):
    rng = np.random.default_rng(V)
    B, S = 6, 2
    p, q = probs(rng, B, S + 1, V), probs(rng, B, S, V)
    d = rng.integers(0, V, (B, S)).astype(np.int32)
    ua, us = np.full((B, S), 0.9, np.float32), rng.random(B, dtype=np.float32)
    ua[3:] = 0.0
    for b in range(B):
        q[b, 0, rng.integers(0, V, V // 2)] = np.nan        # ids that have no weight
        q[b, 1, d[b, 1]] = np.nan                            # refuses its token
    q[1, 0] = np.nan                                         # no weight at all: drawn from p
    q[4, 0, d[4, 0]] = 0.5                                   # stands, then NaN refuses the next
    tok, acc = run_verify(p, q, d, None, ua, us)
    rt, ra = ref_verify(p, q, d, None, ua, us)
    assert np.array_equal(acc, ra) and np.array_equal(tok, rt)
    assert acc.max() <= 1 and acc[4] == 1
    for b in range(B):
        j = acc[b]
        if not np.isnan(q[b, j]).all():
            assert not np.isnan(q[b, j, tok[b, j]])
