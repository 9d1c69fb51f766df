"""The decode-step operators on the GPU against plain 64-bit definitions: norms and
rotation of heads, routing to experts, the experts' products, and the next token;
then a run of them together with the matvecs, captured and replayed."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from gpu_util import qmv
from test_gpu_step import BF16, EPS, F16, F32, TINY, Padded, code, gen, make_w4

pytestmark = pytest.mark.gpu


def randn(seed, *shape):
    return torch.randn(*shape, generator=gen(seed), device="cuda")


# ------------------------------------------------------------------ rope --

def rope_ref(x, n, D, positions, freq, amp, layout, gamma, goff, eps):
    """(values in 64 bits, the magnitudes that their errors go by) of [M, n, D] heads."""
    v = x.double().reshape(x.shape[0], n, D)
    if gamma is not None:
        v = v / torch.sqrt(v.pow(2).mean(2, keepdim=True) + eps) * (gamma.double() + goff)
    out, mag = v.clone(), v.abs()
    rot = 2 * len(freq)
    if rot:
        t = positions.double()[:, None, None] * torch.tensor(freq, dtype=torch.float64, device="cuda")
        i, j = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == 0 else (slice(0, rot, 2), slice(1, rot, 2))
        a, b = v[..., i], v[..., j]
        out[..., i] = amp * (a * t.cos() - b * t.sin())
        out[..., j] = amp * (b * t.cos() + a * t.sin())
        mag = mag.clone()
        mag[..., i] = mag[..., j] = amp * (a.abs() + b.abs())
    return out, mag


def check_rope(got, ref, mag, dt, what):
    # the sum of squares: at most 32 serial steps a lane and 5 exchanges, half of it in the
    # root, then root, quotient and two products: (18.5 + 4) 2^-24; cosines and sines 2^-21;
    # two products and a sum: below 2^-18 in all, then one rounding
    tol = mag * 2.0 ** -18
    tol = tol + (ref.abs() + tol) * EPS[dt] + TINY[dt]
    err = (got.double().reshape(ref.shape) - ref).abs()
    assert bool((err <= tol).all()), (what, float((err / tol).max()))


ROPE_SHAPES = [
    # M, n_q, n_k, D, rot
    (1, 1, 1, 2, 2), (1, 8, 1, 256, 256), (3, 2, 1, 7, 4), (5, 3, 3, 64, 32), (2, 7, 1, 72, 40), (9, 4, 2, 128, 128),
    (4, 5, 0, 80, 16), (6, 0, 3, 96, 96), (3, 12, 4, 100, 50), (2, 32, 8, 256, 64), (33, 1, 1, 512, 512), (2, 3, 1, 1024, 1024),
    (2, 2, 2, 1023, 510), (300, 9, 3, 48, 48), (1000, 4, 1, 32, 30), (7, 1, 2, 1, 0), (5, 6, 2, 200, 0), (2500, 2, 1, 256, 256),
    (17, 40, 8, 16, 16), (3, 4, 4, 520, 8),
    (2600, 20, 5, 72, 40), (2600, 20, 5, 128, 128), (2500, 11, 2, 256, 96),
]


@pytest.mark.parametrize("xdt,dt", [(F32, F16), (F16, F16), (BF16, BF16), (F32, BF16), (BF16, F16), (F16, BF16)])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("M,nq,nk,D,rot", ROPE_SHAPES)
def test_rope(M, nq, nk, D, rot, layout, xdt, dt):
    q = qmv()
    C = (nq + nk) * D
    pad = 0 if M % 2 else 24
    x, oq, ok = Padded(M, C, xdt, ld=C + pad), Padded(M, max(nq * D, 1), dt, ld=nq * D + pad), Padded(M, max(nk * D, 1), dt, ld=nk * D + 8)
    x.t.copy_(randn(M + D, M, C) * 3)
    norm = D % 3 != 0
    gq, gk = ((randn(5 + i, D) * 0.3).to(dt) if norm else None for i in range(2))
    pos = torch.randint(-50, 1_000_000, (M,), generator=gen(D), device="cuda", dtype=torch.int32)
    r = q.Rope(rot, base=1e5, layout=layout, amplitude=1.25) if rot else None
    q.qmv_qk_norm_rope(x.t, nq, nk, D, r, pos if rot else None, gq, gk, gamma_offset=1.0, eps=1e-5,
                       y_dtype=code(dt), q=oq.t[:, :nq * D] if nq else None, k=ok.t[:, :nk * D] if nk else None)
    torch.cuda.synchronize()
    oq.check("q")
    ok.check("k")
    freq = [1e5 ** (-2 * i / rot) for i in range(rot // 2)]
    for o, at, n, g in ((oq, 0, nq, gq), (ok, nq, nk, gk)):
        if n:
            ref, mag = rope_ref(x.t[:, at * D:(at + n) * D], n, D, pos, freq, 1.25, layout, g, 1.0, 1e-5)
            check_rope(o.t[:, :n * D], ref, mag, dt, (at, n))


@pytest.mark.parametrize("shift", [1, 2, 4])
def test_rope_at_any_element(shift):
    q = qmv()
    M, nq, nk, D = 3, 2, 1, 64
    x, oq = Padded(M, 3 * D, F16, ld=3 * D + 5, shift=shift), Padded(M, nq * D, F16, ld=nq * D + 3, shift=shift)
    x.t.copy_(randn(1, M, 3 * D))
    pos = torch.tensor([0, 5, 77], device="cuda", dtype=torch.int32)
    a = q.qmv_qk_norm_rope(x.t, nq, nk, D, q.Rope(D), pos, q=oq.t)
    b = q.qmv_qk_norm_rope(x.t.contiguous(), nq, nk, D, q.Rope(D), pos)
    oq.check("q")
    assert torch.equal(a[0].reshape(M, nq, D), b[0]) and torch.equal(a[1], b[1])


def test_rope_in_place_and_values_stay():
    q = qmv()
    M, nq, nk, D = 40, 6, 2, 128
    g = (1 + 0.1 * randn(2, D)).to(BF16)
    pos = torch.arange(M, device="cuda", dtype=torch.int32) * 1000
    r = q.Rope(D, scaling=q.QMV_SCALE_YARN, factor=4.0, original_length=4096)
    x = randn(3, M, (nq + 2 * nk) * D).to(BF16)
    fq, fk = q.qmv_qk_norm_rope(x, nq, nk, D, r, pos, g, g)
    y = x.clone()
    hq, hk = y[:, :nq * D], y[:, nq * D:(nq + nk) * D]
    q.qmv_qk_norm_rope(y, nq, nk, D, r, pos, g, g, q=hq, k=hk)
    assert torch.equal(hq.reshape(M, nq, D), fq) and torch.equal(hk.reshape(M, nk, D), fk)
    assert torch.equal(y[:, (nq + nk) * D:], x[:, (nq + nk) * D:])
    # heads alone, and rows one by one, give the same bits
    for m in (0, 17):
        a = q.qmv_qk_norm_rope(x[m], nq, nk, D, r, pos[m:m + 1], g, g)
        assert torch.equal(a[0][0], fq[m]) and torch.equal(a[1][0], fk[m])


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("D,rot", [(128, 64), (72, 40), (70, 20), (300, 100)])
@pytest.mark.parametrize("M", [3, 3000])
def test_rope_leaves_what_it_does_not_turn(M, D, rot, layout):
    # an infinity there shows in its own place alone; one that is turned, in its pair's
    q = qmv()
    nq, nk = 9, 2
    x = randn(D, M, (nq + nk) * D).to(F16)
    h = x.view(M, nq + nk, D)
    h[:, 1, rot + 3] = math.inf
    h[:, 4, D - 1] = -math.inf
    h[:, 10, rot] = math.nan
    h[:, 2, 6] = math.inf
    pos = torch.full((M,), 12345, device="cuda", dtype=torch.int32)
    fq, fk = q.qmv_qk_norm_rope(x, nq, nk, D, q.Rope(rot, layout=layout), pos)
    y = torch.cat((fq.reshape(M, nq, D), fk.reshape(M, nk, D)), 1)
    assert torch.equal(torch.nan_to_num(y[:, :, rot:], 7.0), torch.nan_to_num(h[:, :, rot:], 7.0))
    odd = torch.zeros(nq + nk, rot, dtype=torch.bool, device="cuda")
    odd[2, 6] = odd[2, 7 if layout else (6 + rot // 2) % rot] = True
    assert torch.equal(~torch.isfinite(y[:, :, :rot]), odd.expand(M, -1, -1))


@pytest.mark.parametrize("scaling", ["NONE", "LINEAR", "NTK", "YARN"])
@pytest.mark.parametrize("far", [1, 100_000, 2 ** 31 - 1])
def test_rope_far_positions(scaling, far):
    # a single pair of ones a frequency shows the angle itself
    q = qmv()
    rot = 64
    r = q.Rope(rot, scaling=getattr(q, "QMV_SCALE_" + scaling), factor=8.0, original_length=4096, layout=1)
    x = torch.zeros(3, rot, device="cuda")
    x[:, 0::2] = 1.0
    pos = torch.tensor([far, far - 1, -far], device="cuda", dtype=torch.int32)
    y = q.qmv_qk_norm_rope(x, 1, 0, rot, r, pos, y_dtype=q.QMV_F16)[0][:, 0].double() / r.amplitude
    ref = torch.empty(3, rot, dtype=torch.float64)
    for m, p in enumerate(pos.tolist()):
        for i, w in enumerate(r.inv_freq):
            # the frequency's own 53 bits set how well its angle is known: compare against
            # the same double, reduced exactly
            t = float(Fraction(w) * p / Fraction(6.283185307179586) % 1)
            ref[m, 2 * i], ref[m, 2 * i + 1] = math.cos(2 * math.pi * t), math.sin(2 * math.pi * t)
    # turns = frequency / (2 pi) is rounded once and the divisor is 2 pi in 53 bits (as here):
    # far * w / 2 pi * 2^-53 turns, times 2 pi; then 2^-21, and the rounding to fp16 (of up to amplitude)
    tol = abs(far) * 2.0 ** -53 * 8 + 2.0 ** -21 + EPS[F16] * 1.01 + TINY[F16]
    assert float((y.cpu() - ref).abs().max()) <= tol


# ----------------------------------------------------------------- route --

def route_ref(x, T, score, bias, groups, group_k, group_top, renorm, scale):
    x = x.double()
    b = torch.zeros(x.shape[1], dtype=torch.float64, device="cuda") if bias is None else bias.double()
    out = torch.isnan(x) | (x == -math.inf) | torch.isnan(b) | (b == -math.inf)
    x = torch.where(out, -math.inf, x)
    if score:
        s = torch.where(x >= 0, 1 / (1 + torch.exp(-x)), torch.exp(x) / (1 + torch.exp(x)))
        s = torch.where(out, 0.0, s)
    else:
        top = x.amax(1, keepdim=True)
        e = torch.where(x == top, 1.0, torch.exp(x - top))
        e = torch.where(out, 0.0, e)
        s = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    rank = torch.where(out, -math.inf, s + b)
    key = torch.where(out, -math.inf, x) if bias is None else rank          # s rises with x
    if groups > 1:
        M, E = x.shape
        worth = rank.view(M, groups, -1).sort(dim=2, descending=True).values[..., :group_top].sum(2)
        best = worth.sort(dim=1, descending=True, stable=True).indices[:, :group_k]
        keep = torch.zeros(M, groups, dtype=torch.bool, device="cuda").scatter_(1, best, True)
        key = torch.where(keep[:, :, None], key.view(M, groups, -1), -math.inf).view(M, E)
    k = key.sort(dim=1, descending=True, stable=True)
    ids, left = k.indices[:, :T], k.values[:, :T] > -math.inf
    w = torch.where(left, s.gather(1, ids), 0.0)
    if renorm:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total.clamp(min=1e-300), 0.0)
    return torch.where(left, ids, -1).int(), w * scale


def check_route(x, T, score, bias=None, groups=1, group_k=1, group_top=1, renorm=True, scale=1.0):
    q = qmv()
    ids, w = q.qmv_route(x, T, score=score, bias=bias, groups=groups, group_k=group_k, group_top=group_top,
                         renormalise=renorm, scale=scale)
    ri, rw = route_ref(x, T, score, bias, groups, group_k, group_top, renorm, scale)
    assert torch.equal(ids, ri), ((ids != ri).any(1).nonzero()[:4], ids[(ids != ri).any(1)][:2], ri[(ids != ri).any(1)][:2])
    assert bool(((w.double() - rw).abs() <= rw.abs() * 2.0 ** -20 + 2.0 ** -126 * abs(scale)).all())
    return ids, w


ROUTES = [
    # M, E, T, groups, group_k, group_top
    (1, 1, 1, 1, 1, 1), (1, 64, 8, 1, 1, 1), (7, 5, 5, 1, 1, 1), (33, 100, 64, 1, 1, 1), (129, 156, 6, 12, 3, 2),
    (50, 256, 8, 8, 4, 2), (20, 512, 16, 4, 2, 1), (11, 1024, 33, 32, 7, 2), (9, 31, 2, 31, 5, 1), (300, 128, 1, 16, 16, 2),
    (5, 6, 3, 2, 1, 2), (64, 60, 10, 3, 2, 1), (3, 999, 40, 9, 4, 2),
    (400, 384, 16, 1, 1, 1), (200, 512, 31, 1, 1, 1), (200, 1024, 24, 8, 2, 2), (100, 1024, 32, 1, 1, 1), (100, 300, 20, 2, 1, 1),
]


@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("M,E,T,groups,group_k,group_top", ROUTES)
def test_route(M, E, T, groups, group_k, group_top, biased, score, dt):
    x = (randn(M + E, M, E) * 2).to(dt)
    bias = 0.2 * randn(E, E) if biased else None
    check_route(x, T, score, bias, groups, group_k, group_top, E % 2 == 0, 1.0 if T % 2 else 2.5)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("groups,group_k,group_top", [(1, 1, 1), (8, 3, 2), (8, 3, 1)])
def test_route_ranks_that_fp32_cannot_tell_apart(score, groups, group_k, group_top):
    # biases that take every rank to the same number, up to their own rounding
    M, E = 40, 128
    x = randn(4, 1, E).expand(M, E).contiguous()
    s = torch.sigmoid(x[0].double()) if score else torch.softmax(x[0].double(), 0)
    bias = (1.0 - s).float()
    check_route(x, 8, score, bias, groups, group_k, group_top)
    # and a few such among others
    y = randn(5, M, E)
    y[:, ::9] = x[:, ::9]
    check_route(y, 8, score, bias, groups, group_k, group_top)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups,group_k,group_top", [(1, 1, 1), (4, 2, 2)])
def test_route_ties_masks_and_extremes(score, biased, groups, group_k, group_top):
    E, T = 64, 8
    inf, nan, low = math.inf, math.nan, torch.finfo(F32).min
    x = randn(8, 12, E)
    x[0] = 0.0                                  # all alike
    x[1] = torch.randint(0, 3, (E,), generator=gen(1), device="cuda").float()
    x[2] = -inf                                 # nothing left
    x[3] = -inf
    x[3, [5, 60, 17]] = torch.tensor([1.0, 2.0, 2.0], device="cuda")       # less than T left
    x[4, ::2] = low
    x[5] = low
    x[6, 7] = nan
    x[7] = nan
    x[8, 40] = inf
    x[9, [3, 4, 40]] = inf
    x[10, 1:] = -90.0
    x[11] = -0.0
    x[11, ::3] = 0.0
    bias = torch.zeros(E, device="cuda") if biased else None
    if biased:
        bias[10], bias[11], bias[12] = nan, -inf, 0.5
    check_route(x, T, score, bias, groups, group_k, group_top)
    for dt in (F16, BF16):
        y = x.clone()
        y[y == low] = torch.finfo(dt).min
        check_route(y.to(dt), T, score, bias, groups, group_k, group_top)


def test_route_strides_and_own_outputs():
    q = qmv()
    x = Padded(9, 70, F16, ld=77, shift=1)
    x.t.copy_(randn(2, 9, 70))
    ids, w = Padded(9, 5, torch.int32), Padded(9, 5, F32)
    q.qmv_route(x.t, 5, ids=ids.t, weights=w.t)
    ids.check("ids")
    w.check("weights")
    a, b = q.qmv_route(x.t.contiguous(), 5)
    assert torch.equal(a, ids.t) and torch.equal(b, w.t)
    one = q.qmv_route(x.t[4], 5)
    assert torch.equal(one[0], a[4:5]) and torch.equal(one[1], b[4:5])


# --------------------------------------------------------------- experts --

def act_ref(x, act):
    a, b = x.double().chunk(2, -1)
    if act == 1:
        return a / (1 + torch.exp(-a)) * b
    return 0.5 * a * (1 + torch.tanh(math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3))) * b


EXPERTS = [
    # M, T, E, R, K, group
    (1, 1, 1, 32, 32, 32), (1, 8, 16, 64, 256, 128), (2, 3, 5, 96, 160, 64), (5, 2, 4, 32, 416, 32), (7, 4, 9, 160, 1056, 128),
    (16, 8, 8, 64, 512, 64), (40, 2, 3, 96, 288, 32), (64, 6, 40, 128, 640, 128), (3, 1, 200, 32, 96, 32), (100, 8, 24, 64, 128, 64),
    (1, 2, 2, 2048, 2048, 128), (9, 3, 4, 64, 8192, 128), (2, 2, 3, 32, 16384, 64), (300, 1, 2, 32, 64, 64), (600, 3, 5, 96, 192, 32),
]


def distinct(M, T, E, seed):
    if T > E:
        return torch.randint(0, E, (M, T), generator=gen(seed), device="cuda", dtype=torch.int32)
    return torch.rand(M, E, generator=gen(seed), device="cuda").argsort(1)[:, :T].to(torch.int32).contiguous()


@pytest.mark.parametrize("xdt", [F16, BF16])
@pytest.mark.parametrize("per_pair", [False, True])
@pytest.mark.parametrize("M,T,E,R,K,group", EXPERTS)
def test_experts_exact_on_whole_numbers(M, T, E, R, K, group, per_pair, xdt):
    # as the 4-bit matvec's: every partial sum is a multiple of 2^-3 below 2 * 15 * 16384 < 2^19
    q = qmv()
    p, _, w = make_w4(E * R, K, group, M % 2 == 0, xdt, 50 + M + K, exact=True)
    ids = distinct(M, T, E, 3)
    ids[M // 2, T - 1] = -1
    shape = (M, T, K) if per_pair else (M, K)
    x = torch.randint(-2, 3, shape, generator=gen(K), device="cuda").to(xdt)
    y = Padded(M * T, R, F32)
    q.qmv_w4_experts(p, R, ids, x, y=y.t.view(M, T, R))
    torch.cuda.synchronize()
    y.check("y")
    xs = (x if per_pair else x[:, None, :].expand(M, T, K)).reshape(M * T, K).double()
    ref = torch.zeros(M * T, R, dtype=torch.float64, device="cuda")
    flat = ids.view(-1)
    for e in flat.unique().tolist():
        if e >= 0:
            at = (flat == e).nonzero()[:, 0]
            ref[at] = xs[at] @ w[e * R:(e + 1) * R].t()
    assert torch.equal(y.t.double(), ref)
    # weights that are powers of two keep the sum exact
    ws = torch.pow(2.0, torch.randint(-2, 1, (M, T), generator=gen(9), device="cuda").float())
    z = q.qmv_w4_experts(p, R, ids, x, weights=ws)
    assert torch.equal(z.double(), (ref.view(M, T, R) * ws[:, :, None]).sum(1))
    assert q.qmv_device_error(clear=True) == 0


@pytest.mark.parametrize("ydt", [F32, F16, BF16])
@pytest.mark.parametrize("xdt,sdt", [(F16, F16), (BF16, BF16), (F16, BF16), (BF16, F16)])
@pytest.mark.parametrize("act", [0, 1, 2])
@pytest.mark.parametrize("M,T,E,R,K,group", [(1, 8, 12, 64, 1024, 128), (12, 4, 6, 96, 672, 32), (50, 2, 3, 32, 320, 64)])
def test_experts_general(M, T, E, R, K, group, act, xdt, sdt, ydt):
    q = qmv()
    p, _, w = make_w4(E * R, K, group, True, sdt, 7 + M)
    ids = distinct(M, T, E, 5)
    width = K * (2 if act else 1)
    x = Padded(M * T, width, xdt, ld=width + 40)
    x.t.copy_(randn(3, M * T, width))
    x3 = x.t.as_strided((M, T, width), (T * x.ld, x.ld, 1))
    ws = torch.rand(M, T, generator=gen(8), device="cuda")
    y = Padded(M, R, ydt, ld=R + 3)
    q.qmv_w4_experts(p, R, ids, x3, weights=ws, act=act, y=y.t, y_dtype=code(ydt))
    torch.cuda.synchronize()
    y.check("y")
    u = x.t.double()
    flip = torch.zeros_like(u)
    if act:
        u = act_ref(x.t, act)
        # fp32 steps of the activation: below 2^-20 of itself and of what a difference
        # 1 + tanh takes away (2^-22 of |gate * up|); where that crosses a border the rounding goes the other way
        near = u.abs() * 2.0 ** -20 + (x.t[:, :K].double() * x.t[:, K:].double()).abs() * 2.0 ** -22 + 2.0 ** -140
        flip = ((u + near).to(xdt).double() - (u - near).to(xdt).double()).abs()
        u = u.to(xdt).double()
    flat = ids.view(-1).long()
    wr = w.view(E, R, K)
    ref, A, F = (torch.zeros(M * T, R, dtype=torch.float64, device="cuda") for _ in range(3))
    for e in range(E):
        at = (flat == e).nonzero()[:, 0]
        ref[at], A[at], F[at] = u[at] @ wr[e].t(), u[at].abs() @ wr[e].abs().t(), flip[at] @ wr[e].abs().t()
    # the products' fp32 sums as in the 4-bit matvec (17 terms a step of 16 k, up to 8 steps a group), x * q
    # and z * sum(x) apart, then T terms
    B = u.abs().sum(1, keepdim=True) * 30 * 0.02
    tol = (A + B) * (17 * 8 + -(-K // group) + 32) * 2.0 ** -23 + F
    g = ws.double()[:, :, None]
    ref = (ref.view(M, T, R) * g).sum(1)
    tol = (tol.view(M, T, R) * g).sum(1) + (A.view(M, T, R) * g).sum(1) * (T + 1) * 2.0 ** -24
    tol = tol + (ref.abs() + tol) * EPS[ydt] * (ydt != F32) + TINY[ydt]
    err = (y.t.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


def test_experts_rows_are_their_own():
    # a token's result does not depend on what else is in the batch, and repeats
    q = qmv()
    M, T, E, R, K = 37, 4, 6, 64, 512
    p, _, _ = make_w4(E * R, K, 64, True, BF16, 3)
    ids = distinct(M, T, E, 1)
    x = randn(2, M, K).to(BF16)
    x[5, 17], x[9, 3], x[11] = math.inf, math.nan, 0.0
    y = q.qmv_w4_experts(p, R, ids, x)
    assert torch.equal(y.view(torch.int32), q.qmv_w4_experts(p, R, ids, x).view(torch.int32))
    clean = [m for m in range(M) if m not in (5, 9)]
    assert bool(torch.isfinite(y[clean]).all()) and not bool(y[11].any())
    assert bool(torch.isnan(y[9]).all()) and not bool(torch.isfinite(y[5]).any())
    for m in (0, 5, 20):
        one = q.qmv_w4_experts(p, R, ids[m:m + 1], x[m:m + 1])
        a, b = one[0], y[m]
        assert torch.equal(torch.isnan(a), torch.isnan(b))
        fin = torch.isfinite(b)
        tol = b[fin].abs() * 2.0 ** -10 + 1e-2
        assert bool(((a[fin] - b[fin]).abs() <= tol).all())


@pytest.mark.parametrize("M,T", [(3, 8), (16, 8), (17, 8), (64, 5)])
def test_experts_that_a_token_has_twice(M, T):
    # an id may stand more than once in a row, or none at all
    q = qmv()
    p, _, w = make_w4(6 * 64, 256, 64, True, F16, 8, exact=True)
    x = torch.randint(-2, 3, (M, 256), generator=gen(M), device="cuda").to(F16)
    ids = torch.randint(-1, 6, (M, T), generator=gen(T), device="cuda", dtype=torch.int32)
    ids[0], ids[M - 1] = 4, -1
    y = q.qmv_w4_experts(p, 64, ids, x)
    # whole numbers: every partial sum is exact
    all_of = torch.cat(((x.double() @ w.t()).view(M, 6, 64), torch.zeros(M, 1, 64, dtype=torch.float64, device="cuda")), 1)
    ref = all_of.gather(1, torch.where(ids < 0, 6, ids).long()[:, :, None].expand(-1, -1, 64))
    assert torch.equal(y.double(), ref)
    none = q.qmv_w4_experts(p, 64, torch.full_like(ids, -1), x, weights=torch.ones(M, T, device="cuda"))
    assert not bool(none.any()) and q.qmv_device_error(clear=True) == 0


def test_experts_ids_out_of_range():
    q = qmv()
    p, _, w = make_w4(4 * 32, 128, 128, True, F16, 3)
    x = randn(2, 3, 128).to(F16)
    assert q.qmv_device_error(clear=True) == 0
    full = q.qmv_w4_experts(p, 32, torch.tensor([[0, 1], [2, 3], [3, 0]], device="cuda", dtype=torch.int32), x)
    ids = torch.tensor([[0, 4], [-7, 3], [-1, -1]], device="cuda", dtype=torch.int32)
    y = q.qmv_w4_experts(p, 32, ids, x)
    assert q.qmv_device_error(clear=True) == 8
    assert torch.equal(y[0, 0], full[0, 0]) and torch.equal(y[1, 1], full[1, 1])
    assert not bool(y[0, 1].any()) and not bool(y[1, 0].any()) and not bool(y[2].any())
    ids[0, 1] = ids[1, 0] = -1
    z = q.qmv_w4_experts(p, 32, ids, x, weights=torch.ones(3, 2, device="cuda"))
    assert q.qmv_device_error(clear=True) == 0
    assert torch.equal(z[0], y[0, 0]) and torch.equal(z[1], y[1, 1]) and not bool(z[2].any())


# ---------------------------------------------------------------- sample --

COEFF = [np.float32(c) for c in (1.0, 0.6931471824645996, 0.2402234971523285, 0.055503811687231064, 0.00966636836528778,
                                 0.0013381302123889327)]


def draw_ref(x, u, t, k, p, m):
    """The token of one row by the definition, with whole numbers of any length."""
    f32 = np.float32
    x = np.where(np.isnan(x), f32(-np.inf), x.astype(f32))
    V = len(x)
    top = x.max()
    if top == -np.inf:
        return -1
    if not t > 0:
        return int(np.argmax(x))
    with np.errstate(all="ignore"):
        c = f32(1.4426950408889634) / np.maximum(f32(t), f32(2.0 ** -100))
        z = np.where(x == top, f32(0), np.minimum((top - x).astype(f32) * c, f32(64))).astype(f32)
        z = np.where(x == -np.inf, f32(64), z)
        n = np.rint(z)
        f = (n - z).astype(np.float64)
        g = np.full(V, COEFF[-1], f32)
        for a in COEFF[-2::-1]:
            g = (g.astype(np.float64) * f + np.float64(a)).astype(f32)
        w = np.floor(g.astype(np.float64) * np.exp2(42.0 - n.astype(np.float64))).astype(np.int64)
    w[x == -np.inf] = 0
    order = np.lexsort((np.arange(V), -x))
    if 0 < k < V:
        order = order[:k]
    run = np.cumsum(w[order])
    if p < 1:
        need = int(run[-1]) * int(max(float(f32(p)), 0.0) * 2 ** 31) >> 31
        before = run - w[order]
        order = order[(before < need) | (np.arange(len(order)) == 0)]
    order = order[w[order] >= int(min(max(float(f32(m)), 0.0), 1.0) * 2 ** 42)]
    ids = np.sort(order)
    run = np.cumsum(w[ids])
    at = int(run[-1]) * int(min(max(float(u), 0.0) * 2 ** 31, 2 ** 31 - 128)) >> 31
    return int(ids[np.searchsorted(run, at, side="right")])


def logits_like(seed, rows, V):
    x = randn(seed, rows, V) * 2
    g = gen(seed + 1)
    x.scatter_add_(1, torch.randint(0, V, (rows, 8), generator=g, device="cuda"), 6 + 5 * torch.rand(rows, 8, generator=g, device="cuda"))
    return x


def check_sample(x, u, t=1.0, k=0, p=1.0, m=0.0):
    got = qmv().qmv_sample(x, u, temperature=t, top_k=k, top_p=p, min_p=m)
    xs, us = x.float().cpu().numpy(), u.cpu().numpy()
    row = lambda v, r: v[r].item() if torch.is_tensor(v) else v
    ref = [draw_ref(xs[r], us[r], row(t, r), row(k, r), row(p, r), row(m, r)) for r in range(len(xs))]
    assert got.tolist() == ref, [(i, a, b) for i, (a, b) in enumerate(zip(got.tolist(), ref)) if a != b][:5]
    return got


@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("k,p,m", [(0, 1.0, 0.0), (1, 1.0, 0.0), (50, 1.0, 0.0), (0, 0.9, 0.0), (0, 1.0, 0.05), (64, 0.95, 0.01),
                                   (1000, 0.5, 0.0), (0, 0.0, 0.0), (7, 1.0, 1.0), (0, 0.9999, 0.0)])
@pytest.mark.parametrize("rows,V", [(1, 1), (3, 2), (17, 100), (9, 1000), (5, 4096), (8, 5003), (4, 32768), (3, 50257), (2, 262144)])
def test_sample(rows, V, k, p, m, dt):
    x = logits_like(V, rows, V).to(dt)
    check_sample(x, torch.rand(rows, generator=gen(V + k), device="cuda"), 0.8, k, p, m)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("k,p,m", [(50, 0.9, 0.0), (0, 0.9, 0.0), (0, 0.999, 0.001), (3000, 0.8, 0.0), (0, 1.0, 0.0), (2000, 1.0, 0.02), (200, 0.95, 0.0), (256, 1.0, 0.0)])
@pytest.mark.parametrize("rows,V", [(320, 5001), (160, 20000), (40, 100_000), (1, 300_001), (2, 1 << 20), (6, 25601), (5, 8200), (6, 7000)])
def test_sample_many_and_long_rows(rows, V, k, p, m, dt):
    x = logits_like(V, rows, V).to(dt)
    check_sample(x, torch.rand(rows, generator=gen(V + k), device="cuda"), 0.8, k, p, m)


@pytest.mark.parametrize("V", [300, 20000, 131073])
def test_sample_settings_a_row(V):
    rows = 24
    x = logits_like(3, rows, V)
    r = lambda s: torch.rand(rows, generator=gen(s), device="cuda")
    t = 0.3 + 1.5 * r(1)
    t[0], t[1], t[2], t[3], t[4] = 0.0, -1.0, math.nan, math.inf, 1e-30
    k = torch.randint(-3, 400, (rows,), generator=gen(2), device="cuda", dtype=torch.int32)
    p = 0.5 + 0.7 * r(3)
    p[5], p[6], p[7] = math.nan, -1.0, 2.0
    m = 0.1 * r(4) - 0.02
    m[8], m[9] = math.nan, 5.0
    u = r(5)
    u[10], u[11], u[12] = 0.0, 1.0 - 2.0 ** -24, 1.0
    xs, us = x.cpu().numpy(), u.cpu().numpy()
    got = qmv().qmv_sample(x, u, t, k, p, m).tolist()
    for i in range(rows):
        pi, mi = p[i].item(), m[i].item()
        ref = draw_ref(xs[i], us[i], t[i].item(), max(k[i].item(), 0), 1.0 if math.isnan(pi) else pi, 0.0 if math.isnan(mi) else mi)
        assert got[i] == ref, (i, got[i], ref)


@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("V", [33, 4097, 70000])
@pytest.mark.parametrize("k,p,m", [(0, 1.0, 0.0), (5, 1.0, 0.0), (40, 0.7, 0.0), (0, 0.6, 0.0), (0, 1.0, 0.5)])
def test_sample_ties_masks_and_extremes(V, k, p, m, dt):
    x = randn(7, 12, V)
    inf, low = math.inf, torch.finfo(dt).min
    x[0] = 0.25                                              # all alike
    x[1] = torch.randint(0, 3, (V,), generator=gen(1), device="cuda").float()
    x[2] = -inf
    x[3] = -inf
    x[3, V // 2] = -3.0
    x[4] = low
    x[5, 1::2] = low
    x[6, V - 1] = inf
    x[7, [1, V // 3, V - 2]] = inf
    x[8, 5] = math.nan
    x[9] = math.nan
    x[10] = torch.where(torch.arange(V, device="cuda") % 3 == 0, 0.0, -0.0)
    x[11] = -40.0
    x[11, 3:9] = 30.0
    x = x.to(dt)
    for s in range(4):
        check_sample(x, torch.rand(12, generator=gen(s), device="cuda"), (0.05, 0.7, 1.0, 9.0)[s], k, p, m)


def test_sample_follows_the_probabilities():
    # 40000 draws of one row: each id's count is within 6 standard deviations of its mean
    V, n = 50, 40000
    x = randn(3, 1, V)
    u = (torch.arange(n, device="cuda") + 0.5) / n
    got = qmv().qmv_sample(x.expand(n, V).contiguous(), u[torch.randperm(n, generator=gen(2), device="cuda")], 0.7)
    count = torch.bincount(got.long(), minlength=V).double()
    p = torch.softmax(x[0].double() / 0.7, 0)
    # the numbers are evenly spaced, so a count is off by less than 1, and by 2^-18 of itself
    assert bool(((count - n * p).abs() <= 1 + n * p * 2.0 ** -18).all())


def test_sample_strides_and_own_tokens():
    q = qmv()
    for dt in (F32, F16):
        x = Padded(5, 1001, dt, ld=1013, shift=1)
        x.t.copy_(logits_like(3, 5, 1001))
        u = torch.rand(5, generator=gen(2), device="cuda")
        tok = Padded(1, 5, torch.int32)
        q.qmv_sample(x.t, u, 0.9, 30, 0.9, tokens=tok.t[0])
        tok.check("tokens")
        assert tok.t[0].tolist() == q.qmv_sample(x.t.contiguous(), u, 0.9, 30, 0.9).tolist()
        assert q.qmv_sample(x.t[2], u[2:3], 0.9, 30, 0.9).item() == tok.t[0, 2].item()


# -------------------------------------------------------------- together --

def test_a_decode_step_together_captured_and_replayed():
    """One block and the lm_head of a small mixture-of-experts decoder, with the library's own
    matvecs and norms between: eager, on another stream, and as a replayed graph."""
    q = qmv()
    M, Dm, nq, nk, D, E, T, F, V = 4, 512, 4, 2, 64, 16, 4, 256, 5000
    wqkv, _, _ = make_w4((nq + 2 * nk) * D, Dm, 128, True, BF16, 1)
    router, _, _ = make_w4(E, Dm, 128, True, BF16, 2)
    up, _, _ = make_w4(E * 2 * F, Dm, 64, True, BF16, 3)
    down, _, _ = make_w4(E * Dm, F, 64, True, BF16, 4)
    head, _, _ = make_w4(V, Dm, 128, True, BF16, 5)
    g = (1 + 0.1 * randn(6, Dm)).to(BF16)
    gh = (1 + 0.1 * randn(7, D)).to(BF16)
    bias = 0.05 * randn(8, E)
    rope = q.Rope(D)
    pos = torch.zeros(M, device="cuda", dtype=torch.int32)
    h0, a0 = torch.zeros(M, Dm, device="cuda", dtype=BF16), torch.zeros(M, Dm, device="cuda", dtype=BF16)
    u = torch.zeros(M, device="cuda")
    ws1, ws2 = q.qmv_w4_experts_workspace(up, 2 * F, M, T), q.qmv_w4_experts_workspace(down, Dm, M, T)

    def step():
        h, z = q.qmv_block_norm(a0, h0, g)
        qkv = q.qmv_w4_gemv(wqkv, z)
        qh, kh = q.qmv_qk_norm_rope(qkv, nq, nk, D, rope, pos, gh, gh, y_dtype=q.QMV_BF16)
        ids, w = q.qmv_route(q.qmv_w4_gemv(router, z), T, score=q.QMV_SCORE_SIGMOID, bias=bias, groups=4, group_k=2, group_top=2)
        y = q.qmv_w4_experts(up, 2 * F, ids, z, y_dtype=q.QMV_BF16, workspace=ws1)
        y = q.qmv_w4_experts(down, Dm, ids, y, weights=w, act=q.QMV_ACT_SILU, y_dtype=q.QMV_BF16, workspace=ws2)
        h, z = q.qmv_block_norm(y, h, g)
        logits = q.qmv_w4_gemv(head, z)
        return qh, kh, ids, w, y, logits, q.qmv_sample(logits, u, 0.8, 40, 0.95)

    def fill(seed):
        h0.copy_(randn(seed, M, Dm))
        a0.copy_(randn(seed + 1, M, Dm))
        pos.copy_(torch.randint(0, 100000, (M,), generator=gen(seed), device="cuda"))
        u.copy_(torch.rand(M, generator=gen(seed), device="cuda"))

    fill(1)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    tokens = set()
    for seed in (11, 12, 13):
        fill(seed)
        eager = step()
        graph.replay()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            aside = step()
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        for a, b, c in zip(eager, captured, aside):
            assert torch.equal(a, b) and torch.equal(a, c)
        # each against its definition, on the inputs that it had
        qh, kh, ids, w, y, logits, tok = eager
        z = q.qmv_block_norm(a0, h0, g)[1]
        qkv = q.qmv_w4_gemv(wqkv, z)
        freq = [10000.0 ** (-2 * i / D) for i in range(D // 2)]
        for o, at, n in ((qh, 0, nq), (kh, nq, nk)):
            ref, mag = rope_ref(qkv[:, at * D:(at + n) * D], n, D, pos, freq, 1.0, 0, gh, 0.0, 1e-6)
            check_rope(o, ref, mag, BF16, at)
        ri, rw = route_ref(q.qmv_w4_gemv(router, z), T, 1, bias, 4, 2, 2, True, 1.0)
        assert torch.equal(ids, ri) and bool(((w.double() - rw).abs() <= rw * 2.0 ** -20).all())
        for r in range(M):
            assert tok[r].item() == draw_ref(logits[r].cpu().numpy(), u[r].item(), 0.8, 40, 0.95, 0.0)
        tokens.add(tuple(tok.tolist()))
    assert len(tokens) == 3
    assert q.qmv_device_error(clear=True) == 0
