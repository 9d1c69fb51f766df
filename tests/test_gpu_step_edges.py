"""The verification-step operators where they are used together with other work:
captured first, forked and joined, on several streams, under programmatic launch
with early weights, through both forms of the binding, at offsets past 32 bits and
at the ends of their sizes."""
import subprocess
import sys

import numpy as np
import pytest
import torch

from conftest import ROOT
from gpu_util import qmv
from test_gpu_step import BF16, F16, F32, gen, make_w4, ref_h, ref_verify

pytestmark = pytest.mark.gpu


def case(seed=5, M=5, D=512, V=4099):
    """Inputs of a small step, and a function that runs it: (outputs, ...)."""
    q = qmv()
    g = gen(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    up, _, _ = make_w4(1536, D, 128, True, BF16, seed + 1)
    down, _, _ = make_w4(D, 1536, 64, True, BF16, seed + 2)
    head, _, _ = make_w4(V, D, 32, False, BF16, seed + 3)
    y, r = rn(M, D), rn(M, D).to(BF16)
    g1, g2 = ((1 + 0.1 * rn(D)).to(BF16) for _ in range(2))
    draft = torch.randint(0, V, (1, M - 1), generator=g, device="cuda", dtype=torch.int32)
    ua, us = torch.rand(1, M - 1, generator=g, device="cuda") * 1e-3, torch.rand(1, generator=g, device="cuda")

    def run():
        h, z = q.qmv_block_norm(y, r, g1, gamma_post=g2)
        a = q.qmv_w4_gemv(up, z, y_dtype=q.QMV_BF16)
        d = q.qmv_w4_gemv(down, a)
        h2, z2 = q.qmv_block_norm(d, h, g2, gamma_post=g1)
        p = q.qmv_softmax(q.qmv_w4_gemv(head, z2), 0.8)
        return (h2, p, *q.qmv_verify_draft(p.view(1, M, V), None, draft, ua, us))

    return run


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


FIRST = """
import sys; sys.path[:0] = [{root!r}, {root!r} + '/tests']
import torch
from test_gpu_step_edges import case, same
run = case(V=70001)                      # packing and inputs; no operator of the step has run yet
s = torch.cuda.Stream()
s.wait_stream(torch.cuda.current_stream())
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=s):
    cap = run()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in cap]
assert same(got, run())
graph.replay()
torch.cuda.synchronize()
assert same(got, cap)
print('captured first')
"""


def test_first_call_of_a_process_may_be_captured():
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=ROOT)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


def test_fork_and_join_in_a_capture():
    q = qmv()
    g = gen(9)
    x = torch.randn(3, 1024, generator=g, device="cuda").to(F16)
    one = torch.ones(1024, device="cuda", dtype=F16)
    pa, _, _ = make_w4(2048, 1024, 64, True, F16, 31)
    pb, _, _ = make_w4(1024, 2048, 128, True, F16, 32)
    side = torch.cuda.Stream()

    def run(main):
        h, z = q.qmv_block_norm(x, x, one)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            b = q.qmv_w4_gemv(pa, z, y_dtype=q.QMV_F16)
        a = q.qmv_softmax(z, 0.5)
        main.wait_stream(side)
        c = q.qmv_w4_gemv(pb, b)
        return h, a, b, c

    ref = run(torch.cuda.current_stream())
    torch.cuda.synchronize()
    main = torch.cuda.Stream()
    main.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        cap = run(main)
    for _ in range(3):
        for t in cap:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(cap, ref)


def test_two_steps_at_once_on_two_streams():
    runs = [case(seed=5), case(seed=50)]
    ref = [r() for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(10):
        outs = []
        for r, s in zip(runs, streams):
            with torch.cuda.stream(s):
                outs.append(r())
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(outs, ref))


def test_early_weights_under_programmatic_launch():
    q = qmv()
    run = case(seed=7)
    ref = run()
    torch.cuda.synchronize()
    q.qmv_set_pdl(True)
    try:
        for _ in range(20):
            out = run()
        torch.cuda.synchronize()
    finally:
        q.qmv_set_pdl(False)
    assert same(out, ref) and q.qmv_device_error(clear=True) == 0


def test_both_forms_of_the_binding_agree():
    # fresh outputs on the current stream go through the host module; outputs that are
    # given go through the checks in full
    q = qmv()
    g = gen(3)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    p, _, _ = make_w4(515, 640, 64, True, BF16, 3)
    x = rn(3, 640).to(BF16)
    for dt, c in ((F32, q.QMV_F32), (F16, q.QMV_F16), (BF16, q.QMV_BF16)):
        y = q.qmv_w4_gemv(p, x, y_dtype=c)
        assert y.dtype == dt and torch.equal(y, q.qmv_w4_gemv(p, x, y=torch.empty_like(y), y_dtype=c))
    gam, gate1, gate2 = rn(640).to(BF16), rn(640).to(BF16), rn(3, 640).to(BF16)
    for gate in (None, gate1, gate2):
        for post in (None, gam):
            a = q.qmv_block_norm(x.float(), x, gam, post, gate, 0.5, 2.0, 1.0, 1e-5)
            b = q.qmv_block_norm(x.float(), x, gam, post, gate, 0.5, 2.0, 1.0, 1e-5, h_out=torch.empty_like(x))
            assert same(a, b)
    for t in (0.7, torch.rand(3, device="cuda")):
        a = q.qmv_softmax(x, t)
        assert torch.equal(a, q.qmv_softmax(x, t, out=torch.empty_like(a)))
    tg = torch.softmax(rn(2, 4, 77), 2)
    dq, d = torch.softmax(rn(2, 3, 77), 2), torch.randint(0, 77, (2, 3), device="cuda", dtype=torch.int32)
    ua, us = torch.rand(2, 3, device="cuda"), torch.rand(2, device="cuda")
    n = torch.tensor([3, 1], device="cuda", dtype=torch.int32)
    for qq in (None, dq):
        for nn in (None, n):
            a = q.qmv_verify_draft(tg, qq, d, ua, us, n_draft=nn)
            b = q.qmv_verify_draft(tg, qq, d, ua, us, n_draft=nn, tokens=torch.empty_like(a[0]))
            assert same(a, b)
    # what the host module leaves to the checks
    for call in (lambda: q.qmv_w4_gemv(p, x[:, :639]), lambda: q.qmv_block_norm(x, x.float(), gam),
                 lambda: q.qmv_softmax(x, torch.rand(2, device="cuda")), lambda: q.qmv_softmax(x.cpu()),
                 lambda: q.qmv_verify_draft(tg, dq[:1], d, ua, us), lambda: q.qmv_block_norm(x, x, gam.cpu())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(q.QmvError):
        q.qmv_softmax(x, -1.0)
    with pytest.raises(q.QmvError):
        q.qmv_w4_gemv(p, x[:0])
    p.close()
    with pytest.raises((q.QmvError, ValueError)):
        q.qmv_w4_gemv(p, x)


def test_w4_many_columns_and_the_longest_rows():
    q = qmv()
    # the last two: clusters along k that meet several times over many strips
    for M, N, K, group in ((4096, 40, 256, 128), (40, 64, 131072, 32), (1, 33, 131072, 128),
                           (32, 8192, 16384, 128), (13, 12000, 24576, 64)):
        g = gen(M)
        codes = torch.randint(0, 16, (N, K), generator=g, device="cuda", dtype=torch.uint8)
        z = torch.randint(0, 16, (N, K // group), generator=g, device="cuda", dtype=torch.uint8)
        p = q.W4Pack(N, K, group, F16, True).pack_weights(codes, torch.ones(N, K // group, device="cuda", dtype=F16), z)
        x = torch.randint(-2, 3, (M, K), generator=g, device="cuda").to(F16)
        # whole numbers below 2 * 15 * 131072 < 2^24: exact in fp32 in any order
        w = codes.double() - z.double().repeat_interleave(group, 1)
        assert torch.equal(q.qmv_w4_gemv(p, x).double(), x.double() @ w.t())


@pytest.mark.parametrize("V", [33, 1000, 4099, 70001])
@pytest.mark.parametrize("dt", [F32, F16])
def test_softmax_rows_and_results_shifted_differently(V, dt):
    q = qmv()
    x = torch.randn(7, V + 3, generator=gen(V), device="cuda").to(dt)
    x[2, 1:] = -torch.inf
    t = torch.tensor([0.5, 0.0, 1.0, 2.0, 0.1, 1.0, 0.0], device="cuda")
    ref = q.qmv_softmax(x[:, 1:V + 1].contiguous(), t)
    for lead, ld in ((0, V), (1, V + 2), (3, V + 5)):
        out = torch.full((7, ld + lead), -7.0, device="cuda")
        v = out[:, lead:lead + V]
        assert q.qmv_softmax(x[:, 1:V + 1], t, out=v) is v
        # other paths sum in other orders: V / 128 + 70 roundings each, as elsewhere
        assert bool(((v - ref).abs() <= ref * 2 * (V / 128 + 70) * 2.0 ** -24 + 2.0 ** -126).all())
        rest = torch.cat([out[:, :lead], out[:, lead + V:]], 1)
        assert bool((rest == -7.0).all())


@pytest.mark.parametrize("M", [3, 320])
@pytest.mark.parametrize("D", [96, 1003, 4100])
def test_norm_tensors_shifted_differently(M, D):
    # y, residual, gate and the results begin at elements and have strides of their own;
    # every placement gives what contiguous tensors give, up to the order of the sums
    q = qmv()
    g = gen(D)

    def view(t, lead, pad):
        out = torch.full((M * (D + pad) + lead + 8,), 9.0, device="cuda", dtype=t.dtype)
        v = out[lead:].as_strided((M, D), (D + pad, 1))
        v.copy_(t)
        return v

    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    y, r, gate = rn(M, D), rn(M, D).to(BF16), torch.sigmoid(rn(M, D)).to(BF16)
    g1, g2 = ((1 + 0.1 * rn(D)).to(BF16) for _ in range(2))
    ref = q.qmv_block_norm(y, r, g1, g2, gate)
    # Two orders of the sums. Each form's fp32 h is off by at most (D / 64 + 48) 2^-24 of the
    # magnitudes added in it, then rounded to bf16 by 2^-8 of itself: off_h. With z = h gamma / rms,
    # |dz| <= |dh| gamma / rms + |z| d(rms) / rms, where d(rms) <= rms(dh), to which come the
    # norm's own sum, twice, and a rounding of z on each side. 1.02 covers the second-order terms,
    # each below (2^-7)^2 times a few
    sums = 2 * (D / 64 + 48) * 2.0 ** -24
    mag = ref_h(y, r, g2, gate, 1.0, 1.0, 0.0, 1e-6)[1].float()
    h0, z0 = ref[0].float(), ref[1].float().abs()
    off_h = mag * sums + h0.abs() * 2.0 ** -7
    rms = torch.sqrt(h0.pow(2).mean(1, keepdim=True) + 1e-6)
    drms = off_h.pow(2).mean(1, keepdim=True).sqrt() / rms
    off = (off_h, 1.02 * (off_h * g1.float().abs() / rms + z0 * (drms + sums + 2.0 ** -7)))
    for lead, pad in ((0, 8), (3, 8), (4, 0), (1, 5)):
        for same_too in (True, False):
            l2, p2 = (lead, pad) if same_too else (lead + 1, pad + 3)
            h, z = view(r, l2, p2), view(r, lead, pad)
            vec = view(g1.expand(M, D).contiguous(), lead, pad)[0] if same_too else g1
            out = q.qmv_block_norm(view(y, lead, pad), view(r, lead, pad), vec, g2, view(gate, lead, pad), h_out=h, out=z)
            for a, b, o in zip(out, ref, off):
                assert bool(((a.float() - b.float()).abs() <= o).all())


def test_offsets_past_32_bits():
    q = qmv()
    # packed bytes past 2^32, codes past 2^33
    N, K = 409600, 21504
    codes = torch.empty(N, K, dtype=torch.uint8, device="cuda").random_(0, 16)
    scales = torch.ones(N, K // 128, device="cuda", dtype=F16)
    p = q.W4Pack(N, K, 128, F16, False).pack_weights(codes, scales)
    assert p.packed_bytes > 2 ** 32
    x = torch.randint(-2, 3, (2, K), device="cuda").to(F16)
    y = q.qmv_w4_gemv(p, x)
    rows = torch.tensor([0, 1, 199999, N - 33, N - 1], device="cuda")
    assert torch.equal(y[:, rows].double(), x.double() @ (codes[rows].double() - 8).t())
    del codes, scales, p, y
    # rows past 2^31 elements
    rows, V = 8300, 262144
    x = torch.empty(rows, V, dtype=F16, device="cuda").normal_()
    pr = q.qmv_softmax(x)
    for i in (0, 8191, rows - 1):
        ref = torch.softmax(x[i].double(), 0)
        assert float((pr[i].double() - ref).abs().max() / ref.max()) < 1e-5
    # the same rows as B = 1660 sequences of five positions
    B = rows // 5
    d = torch.zeros(B, 4, dtype=torch.int32, device="cuda")
    ua, us = torch.ones(B, 4, device="cuda") * 0.999, torch.rand(B, device="cuda")
    n = torch.full((B,), 4, dtype=torch.int32, device="cuda")
    n[-1] = 0
    ua[-2] = 0.0
    tok, acc = q.qmv_verify_draft(pr.view(B, 5, V), None, d, ua, us, n_draft=n)
    for b in (0, B - 2, B - 1):
        rt, ra = ref_verify(pr.view(B, 5, V)[b:b + 1].cpu().numpy(), None, d[b:b + 1].cpu().numpy(),
                            n[b:b + 1].cpu().numpy(), ua[b:b + 1].cpu().numpy(), us[b:b + 1].cpu().numpy())
        assert np.array_equal(tok[b:b + 1].cpu().numpy(), rt) and int(acc[b]) == ra[0]
    del x, pr
    M, D = 540000, 4096
    y = torch.empty(M, D, dtype=BF16, device="cuda").normal_()
    one = torch.ones(D, dtype=BF16, device="cuda")
    h, z = q.qmv_block_norm(y, y, one)
    for i in (0, 524288, M - 1):
        assert torch.equal(h[i], (2 * y[i].float()).to(BF16))
        hs = h[i].double()
        ref = hs / torch.sqrt(hs.pow(2).mean() + 1e-6)
        # one rounding to bf16, and less than a hundredth of it for the fp32 steps before
        assert bool(((z[i].double() - ref).abs() <= ref.abs() * 2.0 ** -8 * 1.01).all())


@pytest.mark.parametrize("M", [1, 2, 5])
def test_halves_of_one_tensor(M):
    # rows that lie between each other's share no memory
    q = qmv()
    D, g = 192, gen(M)
    y, r = torch.randn(M, D, generator=g, device="cuda"), torch.randn(M, D, generator=g, device="cuda").to(F16)
    g1 = torch.ones(D, device="cuda", dtype=F16)
    both = torch.zeros(M, 2 * D, device="cuda", dtype=F16)
    h, z = q.qmv_block_norm(y, r, g1)
    q.qmv_block_norm(y, r, g1, h_out=both[:, :D], out=both[:, D:])
    assert torch.equal(both[:, :D], h) and torch.equal(both[:, D:], z)
    wide = torch.zeros(M, 2 * D, device="cuda")
    wide[:, D:] = y
    q.qmv_softmax(wide[:, D:], out=wide[:, :D])
    assert torch.equal(wide[:, :D], q.qmv_softmax(y)) and torch.equal(wide[:, D:], y)
    with pytest.raises(q.QmvError):
        q.qmv_softmax(wide[:, 1:D + 1], out=wide[:, :D])


@pytest.mark.parametrize("dt", [F32, F16, BF16])
@pytest.mark.parametrize("rows,V", [(304, 4097), (311, 5003), (400, 20003), (700, 9001), (305, 27001), (333, 50257), (304, 56001)])
def test_softmax_many_rows(rows, V, dt):
    # rows enough that a streaming multiprocessor takes several; special ones among them, and
    # rows that begin at any element
    q = qmv()
    inf, nan = float("inf"), float("nan")
    lead, pad = V % 3, V % 5
    buf = torch.full((rows * (V + pad) + 16,), 5.0, device="cuda", dtype=dt)
    x = buf[lead:].as_strided((rows, V), (V + pad, 1))
    x.copy_(torch.randn(rows, V, generator=gen(V), device="cuda") * 4)
    t = 0.25 + torch.rand(rows, generator=gen(rows), device="cuda")
    x[:, 3:9] = -inf
    x[1] = -inf
    x[160, V - 1] = nan
    x[161, 0] = inf
    x[162, :V - 1] = -inf
    x[163, 9:] = -inf
    t[[164, 165, 166, 167]] = torch.tensor([0.0, -1.0, nan, inf], device="cuda")
    x[164:167, V - 2:] = 60.0
    x[165, 0] = 60.0
    x[303] = torch.finfo(dt).min
    out = torch.full((rows * (V + pad) + 16,), -7.0, device="cuda")
    o = out[lead:].as_strided((rows, V), (V + pad, 1))
    q.qmv_softmax(x, t, out=o)
    plain = torch.ones(rows, dtype=torch.bool, device="cuda")
    plain[[1, 160, 161, 162, 164, 165, 166, 167, 303]] = False
    arg = (x[plain].double() - x[plain].double().amax(1, keepdim=True)) / t[plain].double()[:, None]
    ref = torch.softmax(arg, 1)
    # as for few rows: the exponent's roundings, exp2 and the sum's
    rel = 3.25 * 2.0 ** -24 * arg.abs().clamp(max=200) + (4 + 2 + V / 128 + 64) * 2.0 ** -24
    assert bool(((o[plain].double() - ref).abs() <= ref * rel + 2.0 ** -126).all())
    assert not bool(o[1].any())
    assert bool(torch.isnan(o[160]).all()) and bool(torch.isnan(o[161]).all())
    assert float(o[162, V - 1]) == 1.0 and float(o[162].sum()) == 1.0
    for row, at in ((164, V - 2), (165, 0), (166, V - 2)):
        assert float(o[row, at]) == 1.0 and float(o[row].sum()) == 1.0
    assert not bool(o[167, 3:9].any()) and bool((o[167, 9:] == o[167, 0]).all())
    assert bool((o[303] == o[303, 0]).all()) and abs(float(o[303, 0]) * V - 1) < 1e-4
    gaps = torch.ones_like(out, dtype=torch.bool)
    gaps[lead:].as_strided((rows, V), (V + pad, 1)).fill_(False)
    assert bool((out[gaps] == -7.0).all())
    again = torch.empty_like(o.contiguous())
    q.qmv_softmax(x.contiguous(), t, out=again)
    if dt == F32:
        assert torch.equal(q.qmv_softmax(x, t, out=x).nan_to_num(9.0), o.nan_to_num(9.0))      # in place
    assert torch.equal(again.isnan(), o.isnan())
    assert bool(((again[plain].double() - ref).abs() <= ref * rel + 2.0 ** -126).all())
