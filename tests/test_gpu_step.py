"""The verification-step operators on the GPU against plain 64-bit definitions:
the 4-bit matvec with group scales and zero points, the norms between two
blocks, row softmax, and the verification of drafted tokens; then a run of them
together, captured and replayed."""
import math

import numpy as np
import pytest
import torch

from gpu_util import GuardBuf, qmv

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
EPS = {F16: torch.finfo(F16).eps / 2, BF16: torch.finfo(BF16).eps / 2, F32: torch.finfo(F32).eps / 2}
TINY = {F16: 2.0 ** -25, BF16: 2.0 ** -134, F32: 2.0 ** -150}     # half of the smallest step
U24 = 2.0 ** -24


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def code(dt):
    q = qmv()
    return {F32: q.QMV_F32, F16: q.QMV_F16, BF16: q.QMV_BF16}[dt]


class Padded:
    """A [rows, cols] view with row stride ld inside guard bands; the columns
    behind a row's end hold a canary too."""

    def __init__(self, rows, cols, dtype, ld=None, shift=0):
        self.ld = ld or cols
        esize = torch.empty(0, dtype=dtype).element_size()
        n = ((rows - 1) * self.ld + cols + shift) * esize
        self.g = GuardBuf(n)
        self.raw = self.g.view(dtype, (n // esize,))
        self.shift, self.rows, self.cols = shift, rows, cols
        self.t = self.raw[shift:].as_strided((rows, cols), (self.ld, 1))

    def check(self, what):
        self.g.check(what)
        keep = torch.ones_like(self.raw, dtype=torch.bool)
        keep[self.shift:].as_strided((self.rows, self.cols), (self.ld, 1)).fill_(False)
        b = self.raw.view(torch.uint8).view(self.raw.numel(), -1)[keep]
        assert bool((b == 0xA5).all()), f"{what}: written between the rows"


# -------------------------------------------------------------------- w4 --

def make_w4(N, K, group, zeros, sdt, seed, exact=False):
    g = gen(seed)
    G = -(-K // group)
    codes = torch.randint(0, 16, (N, K), generator=g, device="cuda", dtype=torch.uint8)
    if exact:
        scales = torch.pow(2.0, torch.randint(-3, 1, (N, G), generator=g, device="cuda").float()).to(sdt)
    else:
        scales = (0.005 + 0.015 * torch.rand(N, G, generator=g, device="cuda")).to(sdt)
    z = torch.randint(0, 16, (N, G), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    p = qmv().W4Pack(N, K, group, sdt, zeros).pack_weights(codes, scales, z)
    at = torch.arange(K, device="cuda") // group
    w = (codes.double() - (z.double()[:, at] if zeros else 8.0)) * scales.double()[:, at]
    return p, codes, w


W4_SHAPES = [
    # M, N, K, group
    (1, 32, 128, 128), (1, 1, 32, 32), (1, 33, 160, 128), (2, 31, 96, 64), (3, 65, 416, 32), (5, 130, 2048, 128),
    (7, 77, 1056, 64), (8, 256, 512, 32), (9, 100, 4128, 128), (16, 515, 1024, 64), (17, 64, 640, 128),
    (31, 40, 2080, 32), (33, 96, 320, 64), (64, 129, 768, 128), (130, 67, 288, 32), (1, 2048, 2048, 128),
    (4, 8, 21504, 64), (1, 5000, 32, 32), (12, 160, 8192, 128), (1, 16, 70016, 128), (24, 96, 16384, 64),
]


@pytest.mark.parametrize("xdt", [F16, BF16])
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("M,N,K,group", W4_SHAPES)
def test_w4_exact_on_whole_numbers(M, N, K, group, zeros, xdt):
    # x in -2..2, scales 2^-3..1: every partial sum is a multiple of 2^-3 below
    # 2 * 15 * 70016 < 2^21, so it has at most 24 bits: fp32 sums in any order are exact
    p, codes, w = make_w4(N, K, group, zeros, xdt, 100 + M + N + K, exact=True)
    assert torch.equal(p.unpack_codes(), codes)
    x = torch.randint(-2, 3, (M, K), generator=gen(K), device="cuda").to(xdt)
    y = Padded(M, N, F32)
    qmv().qmv_w4_gemv(p, x, y=y.t)
    torch.cuda.synchronize()
    y.check("y")
    assert torch.equal(y.t.double(), x.double() @ w.t())


@pytest.mark.parametrize("ydt", [F32, F16, BF16])
@pytest.mark.parametrize("xdt,sdt", [(F16, F16), (BF16, BF16), (F16, BF16), (BF16, F16)])
@pytest.mark.parametrize("M,N,K,group", [(1, 515, 4096, 128), (6, 130, 5376, 64), (19, 99, 4128, 32), (40, 70, 2048, 128)])
def test_w4_general(M, N, K, group, xdt, sdt, ydt):
    p, _, w = make_w4(N, K, group, True, sdt, 7 + M, exact=False)
    x = torch.randn(M, K, generator=gen(3), device="cuda").to(xdt)
    xp, y = Padded(M, K, xdt, ld=K + 40), Padded(M, N, ydt, ld=N + 3)
    xp.t.copy_(x)
    qmv().qmv_w4_gemv(p, xp.t, y=y.t, y_dtype=code(ydt))
    torch.cuda.synchronize()
    y.check("y")
    ref = x.double() @ w.t()
    # fp32 sums: a product step of 16 k aligns and cuts 17 terms (2^-23 each of
    # the magnitudes' sum), a group has up to 8 steps; scales and the joined
    # parts add one rounding each
    A = x.double().abs() @ w.abs().t()
    tol = A * (17 * 8 + -(-K // group) + 32) * 2.0 ** -23
    tol = tol + (ref.abs() + tol) * EPS[ydt] * (ydt != F32) + TINY[ydt]
    err = (y.t.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


def test_w4_bf16_magnitudes():
    # columns of very different scales, one with a single large value among small
    # ones, one of zeros, one of the smallest normal numbers
    N, K = 130, 2048
    p, _, w = make_w4(N, K, 64, True, BF16, 23)
    x = torch.randn(7, K, generator=gen(4), device="cuda")
    x = x * torch.tensor([2.0 ** -100, 2.0 ** -20, 1.0, 2.0 ** 60, 1e-3, 0.0, 2.0 ** -125], device="cuda")[:, None]
    x[4, 77] = 1e4
    x = x.to(BF16)
    y = qmv().qmv_w4_gemv(p, x)
    ref = x.double() @ w.t()
    A, top = x.double().abs() @ w.abs().t(), x.double().abs().amax(1, keepdim=True)
    # x * q and z * sum(x) apart: (q + z) / |q - z| larger than the sum of magnitudes;
    # q + z is at most 30 and s is A's; and each value off by 2^-39 of its column's largest
    # (2^-21 in the last column, where the scaling stops at 2^126)
    B = x.double().abs().sum(1, keepdim=True) * 30 * 0.02
    off = top * w.abs().sum(1) * torch.tensor([2.0 ** -39] * 6 + [2.0 ** -21], device="cuda")[:, None]
    tol = (A + B) * (17 * 4 + K / 64 + 32) * 2.0 ** -23 + off + 2.0 ** -149
    assert bool(((y.double() - ref).abs() <= tol).all())
    rel = (y.double() - ref).norm(dim=1) / ref.norm(dim=1).clamp(min=1e-300)
    assert float(rel[[0, 1, 2, 3]].max()) < 1e-6 and not bool(y[5].any())


@pytest.mark.parametrize("shift", [1, 2, 4])
def test_w4_x_at_any_element(shift):
    # x and y not aligned to 16 bytes, odd strides
    M, N, K = 5, 67, 416
    p, _, w = make_w4(N, K, 64, True, F16, 11, exact=True)
    xp, y = Padded(M, K, F16, ld=K + 7, shift=shift), Padded(M, N, F16, ld=N + 5, shift=shift)
    xp.t.copy_(torch.randint(-2, 3, (M, K), generator=gen(5), device="cuda"))
    qmv().qmv_w4_gemv(p, xp.t, y=y.t, y_dtype=code(F16))
    torch.cuda.synchronize()
    y.check("y")
    # sums below 2 * 15 * 416 = 12480, in steps of 2^-3: rounded once to fp16
    assert torch.equal(y.t, (xp.t.double() @ w.t()).to(F16))


def test_w4_infinities_and_nan_stay_in_their_column():
    M, N, K = 9, 64, 512
    p, _, w = make_w4(N, K, 128, True, F16, 13)
    x = torch.randn(M, K, generator=gen(2), device="cuda").to(F16)
    clean = qmv().qmv_w4_gemv(p, x)
    x[3, 17] = float("nan")
    x[8, 500] = float("inf")
    y = qmv().qmv_w4_gemv(p, x)
    assert bool(torch.isnan(y[3]).all())
    z = w[:, 500] == 0
    assert bool(torch.isnan(y[8][z]).all()) and torch.equal(y[8][~z], torch.where(w[:, 500][~z] > 0, 1, -1) * torch.inf)
    keep = [i for i in range(M) if i not in (3, 8)]
    assert torch.equal(y[keep], clean[keep])


def test_w4_bound_bytes_other_stream_and_repeat():
    q = qmv()
    p, codes, w = make_w4(300, 640, 64, True, BF16, 17)
    x = torch.randn(3, 640, generator=gen(2), device="cuda").to(BF16)
    y = q.qmv_w4_gemv(p, x)
    p2 = q.W4Pack(300, 640, 64, BF16, True).bind_packed(p.packed.clone())
    assert p2.info() == (300, 640, 64, BF16, True)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y2 = q.qmv_w4_gemv(p2, x, stream=st)
    with torch.cuda.stream(st):
        y3 = q.qmv_w4_gemv(p2, x)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(y, y3)
    assert torch.equal(q.qmv_w4_gemv(p, x[0]), q.qmv_w4_gemv(p, x[:1]))


# ------------------------------------------------------------------ norm --

def ref_h(y, r, gpo, gate, rs, bs, off, eps):
    u = y.double()
    if gpo is not None:
        u = u / torch.sqrt(u.pow(2).mean(1, keepdim=True) + eps) * (gpo.double() + off)
    if gate is not None:
        u = u * gate.double()
    return rs * r.double() + bs * u, (rs * r.double()).abs() + (bs * u).abs()


@pytest.mark.parametrize("ydt,dt", [(F32, F16), (F16, F16), (BF16, BF16), (F32, BF16), (F16, BF16)])
@pytest.mark.parametrize("post,gate", [(True, "none"), (False, "channel"), (True, "token"), (False, "none")])
@pytest.mark.parametrize("M,D,pad", [(1, 1, 0), (3, 7, 2), (1, 2048, 0), (5, 64, 8), (4, 1000, 0), (2, 4099, 5), (7, 5376, 0),
                                     (2, 16384, 16), (300, 256, 0), (1, 65536, 0), (2, 40000, 0), (33, 8192, 8),
                                     (320, 1024, 0), (310, 4096, 8), (305, 5384, 0), (400, 8192, 8), (340, 1001, 0),
                                     (400, 64, 0), (999, 99, 0), (310, 515, 3), (320, 512, 8), (330, 1009, 16), (305, 5381, 0), (306, 4099, 1),
                                     (304, 12001, 0), (311, 8191, 0), (3, 12001, 0), (2, 16383, 0), (5, 5381, 0)])
def test_block_norm(M, D, pad, post, gate, ydt, dt):
    g = gen(M * 7 + D)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    eps, rs, bs, off = 1e-5, 0.75, -1.5, (1.0 if post else 0.0)
    y = Padded(M, D, ydt, ld=D + pad)
    r = Padded(M, D, dt, ld=D + pad)
    h, out = Padded(M, D, dt, ld=D + pad), Padded(M, D, dt, ld=D + pad)
    y.t.copy_(rn(M, D) * 0.7)
    r.t.copy_(rn(M, D) * 2)
    gpr = (1 + 0.1 * rn(D)).to(dt)
    gpo = (0.1 * rn(D)).to(dt) if post else None
    gt = {"none": None, "channel": torch.sigmoid(rn(D)).to(dt), "token": torch.sigmoid(rn(M, D)).to(dt)}[gate]
    a, b = qmv().qmv_block_norm(y.t, r.t, gpr, gamma_post=gpo, gate=gt, residual_scale=rs, branch_scale=bs,
                                gamma_offset=off, eps=eps, h_out=h.t, out=out.t)
    torch.cuda.synchronize()
    assert a is h.t and b is out.t
    h.check("h"), out.check("out")
    hr, mag = ref_h(y.t, r.t, gpo, gt, rs, bs, off, eps)
    # a row's squares are summed by at least 32 threads: D / 32 + 64 roundings, half
    # of them after the root; a dozen more roundings on the way
    rel = (D / 64 + 48) * U24
    tol = mag * rel + (hr.abs() + mag * rel) * EPS[dt] + TINY[dt]
    assert bool(((h.t.double() - hr).abs() <= tol).all())
    hs = h.t.double()
    zr = hs / torch.sqrt(hs.pow(2).mean(1, keepdim=True) + eps) * (gpr.double() + off)
    tol = zr.abs() * (rel + EPS[dt] * (1 + rel)) + TINY[dt]
    assert bool(((out.t.double() - zr).abs() <= tol).all())


def test_block_norm_in_place_and_zero_rows():
    q = qmv()
    M, D = 6, 1537
    g = gen(4)
    y, r = torch.randn(M, D, generator=g, device="cuda"), torch.randn(M, D, generator=g, device="cuda").to(BF16)
    gam = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(BF16)
    y[2], r[2] = 0, 0
    h, z = q.qmv_block_norm(y, r, gam, gamma_post=gam)
    r2 = r.clone()
    h2, z2 = q.qmv_block_norm(y, r2, gam, gamma_post=gam, h_out=r2)
    assert h2 is r2 and torch.equal(h, h2) and torch.equal(z, z2)
    assert not bool(h[2].any()) and not bool(z[2].any())     # a row of zeros stays one: eps keeps the root
    # values whose squares pass fp16's range, and one NaN row that stays alone
    big = torch.full((M, D), 3e4, device="cuda").to(F16)
    one = torch.ones(D, device="cuda", dtype=F16)
    big[1, 5] = float("nan")
    h, z = q.qmv_block_norm(torch.zeros(M, D, device="cuda"), big, one)
    assert bool(torch.isnan(z[1]).all()) and bool((z[[0, 2, 3, 4, 5]] == 1).all())


# --------------------------------------------------------------- softmax --

SOFT = [(1, 1), (3, 2), (2, 31), (5, 1000), (4, 4099), (1, 32768), (2, 50257), (3, 65536), (1, 151937), (2, 262144),
        (1, 262147), (1, 600001), (200, 515)]


@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("rows,V", SOFT)
@pytest.mark.parametrize("pad", [0, 3])
def test_softmax(rows, V, dt, pad):
    g = gen(V)
    x = Padded(rows, V, dt, ld=V + pad)
    x.t.copy_(torch.randn(rows, V, generator=g, device="cuda") * 4)
    if V > 30:
        x.t[:, 5:12] = -torch.inf
    t = 0.25 + torch.rand(rows, generator=g, device="cuda")
    o = Padded(rows, V, F32, ld=V + pad)
    qmv().qmv_softmax(x.t, t, out=o.t)
    torch.cuda.synchronize()
    o.check("out")
    arg = (x.t.double() - x.t.double().amax(1, keepdim=True)) / t.double()[:, None]
    ref = torch.softmax(arg, 1)
    # the exponent is rounded three times (difference, log2(e) / T, product) and fp32's
    # log2(e) is off by 1.34e-8 = 0.23 units of 2^-24; exp2f is good to 2 units, the sum
    # of positive terms has at most V / 128 + 64 roundings
    rel = 3.25 * U24 * arg.abs().clamp(max=200) + (4 + 2 + V / 128 + 64) * U24
    err = (o.t.double() - ref).abs()
    assert bool((err <= ref * rel + 2.0 ** -126).all())
    if V > 30:
        assert not bool(o.t[:, 5:12].any())


def test_softmax_masks_and_special_rows():
    q = qmv()
    inf, nan = float("inf"), float("nan")
    for V in (7, 3000, 70001):
        x = torch.randn(8, V, generator=gen(V), device="cuda")
        x[0] = -inf                                  # nothing is left
        x[1] = torch.finfo(F32).min                  # the type's lowest value everywhere
        x[2, 3] = nan
        x[3, 4] = inf
        x[4, :] = -inf
        x[4, V - 1] = -5.0                           # one token is left
        x[5] = 3.0e38
        y = q.qmv_softmax(x, 0.7)
        assert not bool(y[0].any())
        assert bool((y[1] == y[1, 0]).all()) and abs(float(y[1, 0]) * V - 1) < 1e-4
        assert bool(torch.isnan(y[2]).all()) and bool(torch.isnan(y[3]).all())
        assert float(y[4, V - 1]) == 1.0 and not bool(y[4, :V - 1].any())
        assert bool((y[5] == y[5, 0]).all())
        # temperatures: 0, negative and NaN give the first maximum; huge ones a flat row
        x = torch.randn(6, V, generator=gen(V + 1), device="cuda")
        x[:, 2] = 9.0
        x[:, 6] = 9.0
        x[4] = -inf
        x[5, 1] = nan
        t = torch.tensor([0.0, -1.0, nan, inf, 0.0, 0.0], device="cuda")
        y = q.qmv_softmax(x, t)
        for i in range(3):
            assert float(y[i, 2]) == 1.0 and float(y[i].sum()) == 1.0
        assert bool((y[3] == y[3, 0]).all())
        assert not bool(y[4].any()) and bool(torch.isnan(y[5]).all())
        # a subnormal temperature
        y = q.qmv_softmax(x[:1], torch.tensor([1e-42], device="cuda"))
        assert float(y[0, 2]) == 0.5 and float(y[0, 6]) == 0.5
        assert torch.equal(q.qmv_softmax(x[:3], 0.0), q.qmv_softmax(x[:3], t[:3]))
        # in place
        z = x[:4].clone()
        ref = q.qmv_softmax(z, 0.9)
        assert q.qmv_softmax(z, 0.9, out=z) is z and torch.equal(z, ref)


# ---------------------------------------------------------------- verify --

def units(w):
    w = np.nan_to_num(np.asarray(w, np.float64), nan=0.0)
    return np.floor(np.clip(w, 0, 1) * 2.0 ** 42).astype(np.int64)


def ref_verify(p, q, d, n, ua, us):
    B, S1, V = p.shape
    S = S1 - 1
    tok, acc = np.full((B, S1), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        nb = S if n is None else max(0, min(S, int(n[b])))
        j = 0
        while j < nb:
            t = int(d[b, j])
            if not 0 <= t < V:
                break
            qq = 1.0 if q is None else float(q[b, j, t])
            if not float(ua[b, j]) * qq < float(p[b, j, t]):
                break
            j += 1
        w = p[b, j].astype(np.float32)
        if j < nb:
            one = np.zeros(V, np.float32)
            if q is not None:
                one = q[b, j]
            elif 0 <= int(d[b, j]) < V:
                one[int(d[b, j])] = 1
            rest = units(w - one)
            wi = rest if rest.sum() > 0 else units(w)
        else:
            wi = units(w)
        total = int(wi.sum())
        t = (int(math.floor(float(us[b]) * 2 ** 31)) * total) >> 31
        tok[b, :j] = d[b, :j]
        if total > 0:
            tok[b, j] = int(np.searchsorted(np.cumsum(wi), t, side="right"))
        acc[b] = j
    return tok, acc


def run_verify(p, q, d, n, ua, us):
    dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()
    B, S1, _ = p.shape
    gt, ga = GuardBuf(B * S1 * 4), GuardBuf(B * 4)
    tok, acc = gt.view(torch.int32, (B, S1)), ga.view(torch.int32, (B,))
    qmv().qmv_verify_draft(dev(p), dev(q), dev(d), dev(ua), dev(us), n_draft=dev(n), tokens=tok, n_accepted=acc)
    torch.cuda.synchronize()
    gt.check("tokens"), ga.check("n_accepted")
    return tok.cpu().numpy(), acc.cpu().numpy()


def probs(rng, *shape, sharp=3.0):
    x = rng.normal(size=shape).astype(np.float32) * sharp
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


@pytest.mark.parametrize("with_q", [True, False])
@pytest.mark.parametrize("ragged", [True, False])
@pytest.mark.parametrize("B,S,V", [(1, 1, 1), (3, 2, 2), (4, 3, 33), (16, 4, 1000), (2, 8, 4099), (5, 5, 32003), (1, 4, 262144),
                                   (3, 1, 70001), (2, 0, 515), (70, 2, 129), (1, 600, 40), (1, 1, 1 << 20)])
def test_verify(B, S, V, ragged, with_q):
    rng = np.random.default_rng(B * 100 + S + V)
    p = probs(rng, B, S + 1, V)
    q = probs(rng, B, S, V) * 0.5 + p[:, :S] * 0.5 if with_q else None
    d = rng.integers(0, V, (B, S)).astype(np.int32)
    for b in range(B):                                # likely tokens, so that some stand
        for i in range(S):
            if rng.random() < 0.8:
                d[b, i] = int(p[b, i].argmax())
    n = rng.integers(-1, S + 2, B).astype(np.int32) if ragged else None
    for k in range(3):
        ua, us = rng.random((B, S), dtype=np.float32) * 0.7, rng.random(B, dtype=np.float32)
        if k == 1:
            us[:] = 0.0
        if k == 2:
            us[:] = np.float32(1 - 2.0 ** -24)
            ua[:] = 0.0
        tok, acc = run_verify(p, q, d, n, ua, us)
        rt, ra = ref_verify(p, q, d, n, ua, us)
        assert np.array_equal(acc, ra) and np.array_equal(tok, rt), (k, tok, rt)


def test_verify_borders():
    V = 600
    p = np.zeros((9, 2, V), np.float32)
    q = np.zeros((9, 1, V), np.float32)
    d = np.full((9, 1), 7, np.int32)
    ua, us = np.full((9, 1), 0.5, np.float32), np.full(9, 0.999, np.float32)
    p[:, 0, 7], p[:, 0, 300], q[:, 0, 7] = 0.5, 0.5, 1.0
    p[:, 1, 11] = 1.0
    # 0: u q == p refuses.  1: one step less stands.  2: q = 0 and p > 0 stands
    ua[1] = np.nextafter(np.float32(0.5), np.float32(0))
    q[2, 0, 7] = 0
    # 3: an id below 0, 4: one past the end (the kernel must not read there)
    d[3], d[4] = -1, V
    # 5: refused with p == q everywhere: no rest, so p itself is drawn from
    p[5, 0] = q[5, 0] = 0
    p[5, 0, 40] = q[5, 0, 40] = 1.0
    # 6: p has no mass at all;  7: NaN in p;  8: the last id only
    p[6] = 0
    p[7, 0, 7] = np.nan
    p[8, 0] = 0
    p[8, 0, V - 1] = 1.0
    tok, acc = run_verify(p, q, d, None, ua, us)
    rt, ra = ref_verify(p, q, d, None, ua, us)
    assert np.array_equal(acc, ra) and np.array_equal(tok, rt)
    assert list(acc) == [0, 1, 1, 0, 0, 0, 0, 0, 0]
    assert tok[0].tolist() == [300, -1] and tok[1].tolist() == [7, 11] and tok[2].tolist() == [7, 11]
    assert tok[5].tolist() == [40, -1] and tok[6].tolist() == [-1, -1] and tok[8].tolist() == [V - 1, -1]
    # without draft probabilities an id outside is refused and p drawn from as it is
    tok, acc = run_verify(p, None, d, None, ua, us)
    rt, ra = ref_verify(p, None, d, None, ua, us)
    assert np.array_equal(acc, ra) and np.array_equal(tok, rt)


def test_verify_draws_the_target_distribution():
    # With the drafted token drawn from q, the first emitted token is distributed as
    # p: over a grid of u (accept x sample x draft), counts meet p exactly up to the grid.
    V, n = 8, 24
    rng = np.random.default_rng(1)
    p1, q1 = probs(rng, V, sharp=1.0), probs(rng, V, sharp=1.0)
    ua = ((np.arange(n) + 0.5) / n).astype(np.float32)
    tot = np.zeros(V)
    for d in range(V):
        B = n * n
        p = np.broadcast_to(p1, (B, 2, V))
        q = np.broadcast_to(q1, (B, 1, V))
        tok, _ = run_verify(p, q, np.full((B, 1), d, np.int32), None, np.repeat(ua, n)[:, None], np.tile(ua, n))
        tot += q1[d] * np.bincount(tok[:, 0], minlength=V) / B
    # each of the two grids is off by at most one cell in each of its borders
    assert np.abs(tot - p1).max() <= 2.0 / n


# -------------------------------------------------------------- together --

def test_a_verification_step_together():
    """Block output -> norms -> gate/up and down -> norms -> logits -> probabilities ->
    accepted tokens for 5 columns: each stage against its own 64-bit form on the
    stage's actual inputs, then the same step captured into a graph and replayed."""
    q = qmv()
    B, S, D, FF, V = 1, 4, 512, 1536, 4099
    M = S + 1
    g = gen(21)
    up, _, wup = make_w4(FF, D, 128, True, BF16, 1)
    down, _, wdown = make_w4(D, FF, 64, True, BF16, 2)
    head, _, whead = make_w4(V, D, 32, False, BF16, 3)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    y0, r0 = rn(M, D), rn(M, D).to(BF16)
    g1, g2, g3 = ((1 + 0.1 * rn(D)).to(BF16) for _ in range(3))
    draft = torch.randint(0, V, (B, S), generator=g, device="cuda", dtype=torch.int32)
    ua, us = torch.rand(B, S, generator=g, device="cuda") * 1e-3, torch.rand(B, generator=g, device="cuda")

    def step(stream=None):
        h, z = q.qmv_block_norm(y0, r0, g1, gamma_post=g2, stream=stream)
        a = q.qmv_w4_gemv(up, z, y_dtype=q.QMV_BF16, stream=stream)
        d = q.qmv_w4_gemv(down, a, stream=stream)
        h2, z2 = q.qmv_block_norm(d, h, g3, gamma_post=g2, stream=stream)
        lo = q.qmv_w4_gemv(head, z2, stream=stream)
        pr = q.qmv_softmax(lo, 0.8, stream=stream)
        t, n = q.qmv_verify_draft(pr.view(B, M, V), None, draft, ua, us, stream=stream)
        return h, z, a, d, h2, z2, lo, pr, t, n

    out = step()
    torch.cuda.synchronize()
    h, z, a, d, h2, z2, lo, pr, t, n = out
    near = lambda v, ref, rel: float((v.double() - ref).norm() / ref.norm()) <= rel
    # one rounding to bf16 is at most 2^-8 of each value; fp32 stages stay below 2^-16
    assert near(a, z.double() @ wup.t(), 2.0 ** -8)
    assert near(d, a.double() @ wdown.t(), 2.0 ** -16)
    assert near(h2, ref_h(d, h, g2, None, 1.0, 1.0, 0.0, 1e-6)[0], 2.0 ** -8)
    assert near(lo, z2.double() @ whead.t(), 2.0 ** -16)
    assert near(pr, torch.softmax(lo.double() / 0.8, 1), 2.0 ** -16)
    rt, ra = ref_verify(pr.view(B, M, V).cpu().numpy(), None, draft.cpu().numpy(), None, ua.cpu().numpy(),
                        us.cpu().numpy())
    assert np.array_equal(t.cpu().numpy(), rt) and np.array_equal(n.cpu().numpy(), ra)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        step()
        st.synchronize()
        with torch.cuda.graph(graph, stream=st):
            cap = step()
    for _ in range(3):
        for o in cap:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(out, cap))
