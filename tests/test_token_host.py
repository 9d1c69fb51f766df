"""The decode-step calls check their arguments on the host: status codes of the C ABI and
ValueErrors of the binding, before any device is touched; and what they compute on the host."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

F32, F16, BF16 = 0, 1, 2


@pytest.fixture(scope="module")
def q():
    from bit_weight_only_packed_gb300 import build
    build.build()
    from bit_weight_only_packed_gb300 import qmv
    return qmv


def freqs(q, rot, base=10000.0, scaling=0, factor=1.0, length=4096.0, fast=32.0, slow=1.0):
    w, a = (ctypes.c_double * max(rot // 2, 1))(), ctypes.c_float(-1)
    rc = q.lib().qmv_rope_inv_freq(rot, base, scaling, factor, length, fast, slow, w, ctypes.byref(a))
    return rc, list(w), a.value


def test_rope_inv_freq(q):
    for rot in (2, 4, 64, 100, 256, 1024):
        for scaling in (0, 1, 2, 3):
            rc, w, a = freqs(q, rot, scaling=scaling, factor=8.0)
            if rot == 2 and scaling == 2:
                assert rc == -4
                continue
            assert rc == 0
            b = 10000.0 * (8.0 ** (rot / (rot - 2)) if scaling == 2 else 1.0)
            plain = [b ** (-2 * i / rot) for i in range(rot // 2)]
            if scaling == 1:
                plain = [v / 8 for v in plain]
            if scaling == 3:
                def pair(turns):
                    return rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0))
                lo, hi = max(math.floor(pair(32)), 0), min(math.ceil(pair(1)), rot - 1)
                ramp = [min(max((i - lo) / max(hi - lo, 1e-3), 0), 1) for i in range(rot // 2)]
                plain = [v / 8 * r + v * (1 - r) for v, r in zip(plain, ramp)]
                assert w[0] == plain[0] if lo > 0 else True
            assert all(abs(x - y) <= 1e-14 * y for x, y in zip(w, plain))
            assert abs(a - (0.1 * math.log(8) + 1 if scaling == 3 else 1)) < 1e-7
    # the slowest turns are stretched whole, the fastest stay
    rc, w, _ = freqs(q, 128, scaling=3, factor=16.0)
    assert w[0] == 1.0 and abs(w[63] * 16 / 10000.0 ** (-126 / 128) - 1) < 1e-14
    for kw in (dict(base=1.0), dict(base=math.nan), dict(base=math.inf), dict(scaling=4), dict(scaling=-1),
               dict(scaling=1, factor=0.0), dict(scaling=2, factor=math.nan), dict(scaling=3, factor=math.inf),
               dict(scaling=3, length=0.0), dict(scaling=3, fast=-1.0), dict(scaling=3, slow=math.nan)):
        assert freqs(q, 64, **kw)[0] == -1, kw
    for rot in (0, 1, 3, 1026, -2):
        assert freqs(q, rot)[0] == -4, rot
    assert q.lib().qmv_rope_inv_freq(64, 1e4, 0, 1.0, 1.0, 1.0, 1.0, None, None) == -1


def test_rope_turns(q):
    w = [0.0, 1.0, 2 * math.pi, 1e-9, 0.1, 1234.5678, -0.25, 1e300, -1e-300, math.pi]
    n = len(w)
    a, t = (ctypes.c_double * n)(*w), (ctypes.c_int64 * n)()
    assert q.lib().qmv_rope_turns(n, a, t) == 0
    for v, got in zip(w, t):
        # w / 2 pi in doubles, its whole turns taken off, exactly
        whole = Fraction(v / (2 * math.pi)) % 1
        gap = abs(Fraction(got % 2 ** 64, 2 ** 64) - whole)
        assert min(gap, 1 - gap) <= Fraction(1, 2 ** 53), v
    assert t[0] == 0 and t[2] == 0 and t[9] == -2 ** 63
    for bad in (math.nan, math.inf, -math.inf):
        a[3] = bad
        assert q.lib().qmv_rope_turns(n, a, t) == -1
    assert q.lib().qmv_rope_turns(0, a, t) == q.lib().qmv_rope_turns(2, None, t) == q.lib().qmv_rope_turns(2, a, None) == -1


def test_qk_norm_rope_calls(q):
    def call(M=2, nq=2, nk=1, D=64, x=4096, ld=256, xd=F16, pos=64, turns=64, rot=64, layout=0, gq=None, gk=None, eps=1e-6,
             qo=65536, ldq=128, ko=131072, ldk=64, dt=F16):
        return q.lib().qmv_qk_norm_rope(M, nq, nk, D, x, ld, xd, pos, turns, rot, layout, 1.0, gq, gk, 0.0, eps, qo, ldq, ko,
                                        ldk, dt, None)

    for kw in (dict(M=0), dict(nq=-1), dict(nk=-1), dict(nq=0, nk=0, qo=None, ko=None), dict(D=0), dict(x=None), dict(qo=None),
               dict(ko=None), dict(nq=0), dict(nk=0), dict(xd=3), dict(dt=F32), dict(dt=3), dict(layout=2), dict(eps=-1.0),
               dict(eps=math.nan), dict(pos=None), dict(turns=None), dict(rot=0)):
        assert call(**kw) == -1, kw
    # an output on top of an input or of the other one; in place of another type or stride
    for kw in (dict(qo=131072), dict(ko=4096), dict(qo=4096, xd=F32, ldq=256), dict(qo=4096, ldq=128), dict(qo=4096 + 128, ldq=256),
               dict(pos=65536), dict(turns=65536), dict(gq=65536), dict(gk=131072 + 2), dict(ko=4096 + 2 * 128, ldk=64)):
        assert call(**kw) == -1, kw
    for kw in (dict(nq=4097, ld=10 ** 6, ldq=10 ** 6), dict(nk=4097, ld=10 ** 6, ldk=10 ** 6),
               dict(D=1025, ld=10 ** 5, ldq=10 ** 5, ldk=10 ** 5)):
        assert call(**kw) == -2, kw
    for kw in (dict(rot=-2), dict(rot=66), dict(rot=3), dict(ld=191), dict(ldq=127), dict(ldk=63)):
        assert call(**kw) == -4, kw
    for kw in (dict(x=4097), dict(x=4098, xd=F32), dict(qo=65537), dict(ko=131073), dict(gq=9), dict(gk=9), dict(pos=66),
               dict(turns=68)):
        assert call(**kw) == -3, kw


def test_route_calls(q):
    def call(M=2, E=64, T=8, x=4096, ldl=64, dt=F32, score=0, bias=None, groups=1, gk=1, gt=1, ids=65536, w=131072):
        return q.lib().qmv_route(M, E, T, x, ldl, dt, score, bias, groups, gk, gt, 1, 1.0, ids, w, None)

    for kw in (dict(M=0), dict(E=0), dict(T=0), dict(x=None), dict(ids=None), dict(w=None), dict(dt=3), dict(score=2), dict(score=-1),
               dict(groups=0), dict(gk=0), dict(gt=0), dict(gt=3), dict(ids=131072), dict(w=4096), dict(ids=4100), dict(bias=65540)):
        assert call(**kw) == -1, kw
    for kw in (dict(E=1025, ldl=2000), dict(T=65), dict(groups=33, E=66, ldl=66)):
        assert call(**kw) == -2, kw
    for kw in (dict(groups=5), dict(groups=4, gk=5), dict(T=64, E=32, ldl=32), dict(groups=8, gk=1, T=9), dict(ldl=63),
               dict(groups=32, E=32, ldl=32, gt=2, gk=32)):
        assert call(**kw) == -4, kw
    for kw in (dict(x=4098), dict(x=4097, dt=F16), dict(ids=65538), dict(w=131074), dict(bias=18)):
        assert call(**kw) == -3, kw


def test_experts_calls(q):
    p = q.W4Pack(256, 256, 128)
    args = dict(R=64, M=2, T=2, ids=64, w=None, x=4096, ldx=256, pp=0, xd=F16, act=0, y=65536, ldy=64, yd=F32, ws=1 << 20, wb=1 << 30)

    def call(pack=p.handle, **kw):
        a = {**args, **kw}
        return q.lib().qmv_w4_experts(pack, a["R"], a["M"], a["T"], a["ids"], a["w"], a["x"], a["ldx"], a["pp"], a["xd"], a["act"],
                                      a["y"], a["ldy"], a["yd"], a["ws"], a["wb"], None)

    assert call() == -1                                           # no weights yet
    assert q.lib().qmv_w4_bind(p.handle, 1 << 40) == 0            # an address that nothing reads
    for kw in (dict(pack=None), dict(M=0), dict(T=0), dict(ids=None), dict(x=None), dict(y=None), dict(xd=F32), dict(xd=3),
               dict(yd=3), dict(act=3), dict(act=-1)):
        assert call(**kw) == -1, kw
    for kw in (dict(y=4096), dict(ids=65536), dict(w=65536), dict(y=1 << 40)):
        assert call(**kw) == -1, kw
    for kw in (dict(R=0), dict(R=-32), dict(R=16), dict(R=96), dict(R=512), dict(ldx=255), dict(act=1, ldx=511), dict(ldy=63)):
        assert call(**kw) == -4, kw
    for kw in (dict(M=4097), dict(T=65), dict(M=4096, T=9)):
        assert call(**kw) == -2, kw
    for kw in (dict(ids=66), dict(w=66), dict(x=4097), dict(y=65538), dict(y=65537, yd=F16), dict(ws=(1 << 20) + 128)):
        assert call(**kw) == -3, kw
    need = q.qmv_w4_experts_workspace_bytes(p, 64, 2, 2)
    if need:
        assert call(ws=None) == -7 and call(wb=need - 1) == -7
        assert call(x=1 << 20, ldx=256) == -1 and call(y=(1 << 20) + 256) == -1
    big = q.W4Pack(64, 16416, 32)
    assert q.lib().qmv_w4_bind(big.handle, 1 << 40) == 0
    assert call(pack=big.handle, ldx=20000) == -2
    ws = q.lib().qmv_w4_experts_workspace_bytes
    assert ws(None, 64, 1, 1) == ws(p.handle, 96, 1, 1) == ws(p.handle, 64, 0, 1) == ws(p.handle, 64, 4097, 1) == ws(big.handle, 32, 1, 1) == 0
    sizes = [q.qmv_w4_experts_workspace_bytes(p, 64, m, 4) for m in (1, 2, 8, 64, 512)]
    assert sizes == sorted(sizes) and all(s % 256 == 0 for s in sizes)


def test_sample_calls(q):
    def call(rows=2, V=64, x=4096, ldl=64, dt=F32, t=None, t0=1.0, k=None, k0=0, p=None, p0=1.0, m=None, m0=0.0, u=64, tok=128):
        return q.lib().qmv_sample(rows, V, x, ldl, dt, t, t0, k, k0, p, p0, m, m0, u, tok, None)

    for kw in (dict(rows=0), dict(V=0), dict(x=None), dict(u=None), dict(tok=None), dict(dt=3), dict(t0=-1.0), dict(t0=math.nan),
               dict(k0=-1), dict(p0=-0.1), dict(p0=1.5), dict(p0=math.nan), dict(m0=-0.1), dict(m0=1.5), dict(m0=math.nan)):
        assert call(**kw) == -1, kw
    for kw in (dict(tok=4096), dict(tok=68), dict(t=128), dict(k=132), dict(p=128), dict(m=128)):
        assert call(**kw) == -1, kw
    assert call(V=(1 << 20) + 1, ldl=1 << 21) == -2
    assert call(ldl=63) == -4
    for kw in (dict(x=4098), dict(x=4097, dt=F16), dict(t=18), dict(k=18), dict(p=18), dict(m=18), dict(u=66), dict(tok=130)):
        assert call(**kw) == -3, kw


def test_binding_refuses_before_any_call(q):
    T = torch.zeros
    f16 = lambda *s: T(*s, dtype=torch.float16)
    i32 = lambda *s: T(*s, dtype=torch.int32)
    rope = q.Rope(64, device="cpu")
    p = q.W4Pack(128, 256, 128)
    cases = [
        (lambda: q.Rope(63, device="cpu"), "rot: expected"),
        (lambda: q.Rope(64, layout=2, device="cpu"), "layout: unknown"),
        (lambda: q.Rope(64, inv_freq=[1.0] * 31, device="cpu"), "inv_freq: needs 32"),
        (lambda: q.qmv_qk_norm_rope(f16(2, 128), 2, 1, 64), "does not hold"),
        (lambda: q.qmv_qk_norm_rope(f16(2, 2, 128), 2, 1, 64), "qkv: expected a"),
        (lambda: q.qmv_qk_norm_rope(T(2, 192, dtype=torch.int32), 2, 1, 64), "qkv: expected"),
        (lambda: q.qmv_qk_norm_rope(f16(2, 192), 2, 1, 64, rope), "positions: given"),
        (lambda: q.qmv_qk_norm_rope(f16(2, 192), 2, 1, 64, None, i32(2)), "positions: given"),
        (lambda: q.qmv_qk_norm_rope(f16(2, 192), 2, 1, 64, rope, T(2, dtype=torch.int64)), "positions: expected"),
        (lambda: q.qmv_qk_norm_rope(f16(2, 192), 2, 1, 64, rope, i32(3)), "positions: needs"),
        (lambda: q.qmv_qk_norm_rope(f16(2, 96), 2, 1, 32, rope, i32(2)), "rope: turns"),
        (lambda: q.qmv_qk_norm_rope(f16(2, 192), 2, 1, 64, rope, i32(2), gamma_q=T(64)), "gamma_q: expected"),
        (lambda: q.qmv_qk_norm_rope(f16(2, 192), 2, 1, 64, rope, i32(2), gamma_k=f16(63)), "gamma_k: needs"),
        (lambda: q.qmv_qk_norm_rope(f16(2, 192), 2, 1, 64, rope, i32(2), y_dtype=q.QMV_F32), "y_dtype: expected"),
        (lambda: q.qmv_qk_norm_rope(f16(2, 192), 2, 1, 64, rope, i32(2), q=f16(2, 64)), "q: expected"),
        (lambda: q.qmv_qk_norm_rope(f16(2, 192), 2, 1, 64, rope, i32(2), k=f16(2, 2, 64)), "k: expected"),
        (lambda: q.qmv_qk_norm_rope(f16(2, 192), 3, 0, 64, rope, i32(2), k=f16(2, 64)), "k: there are no"),
        (lambda: q.qmv_qk_norm_rope(f16(2, 192), 2, 1, 64, rope, i32(2), q=f16(2, 64, 2).transpose(1, 2)), "heads of a row"),
        (lambda: q.qmv_qk_norm_rope(f16(2, 192), 2, 1, 64, rope, i32(2)), "CUDA"),
        (lambda: q.qmv_route(T(2, 64, dtype=torch.int32), 2), "logits: expected"),
        (lambda: q.qmv_route(T(2, 64), 2, bias=f16(64)), "bias: expected"),
        (lambda: q.qmv_route(T(2, 64), 2, bias=T(63)), "bias: needs"),
        (lambda: q.qmv_route(T(2, 64), 2, ids=i32(3)), "ids: needs"),
        (lambda: q.qmv_route(T(2, 64), 2, weights=f16(4)), "weights: expected"),
        (lambda: q.qmv_route(T(2, 64), 2), "CUDA"),
        (lambda: q.qmv_w4_experts(p, 64, i32(4), f16(2, 256)), "ids: expected"),
        (lambda: q.qmv_w4_experts(p, 64, T(2, 2, dtype=torch.int64), f16(2, 256)), "ids: expected"),
        (lambda: q.qmv_w4_experts(p, 64, i32(2, 2), f16(2, 256)), "holds no weights"),
        (lambda: q.qmv_sample(T(2, 64), T(3)), "u: needs"),
        (lambda: q.qmv_sample(T(2, 64), f16(2)), "u: expected"),
        (lambda: q.qmv_sample(T(2, 64), T(2), temperature=T(3)), "temperature: needs"),
        (lambda: q.qmv_sample(T(2, 64), T(2), top_k=T(2)), "top_k: expected"),
        (lambda: q.qmv_sample(T(2, 64), T(2), top_p=f16(2)), "top_p: expected"),
        (lambda: q.qmv_sample(T(2, 64), T(2), min_p=T(1)), "min_p: needs"),
        (lambda: q.qmv_sample(T(2, 64), T(2), tokens=T(2, dtype=torch.int64)), "tokens: expected"),
        (lambda: q.qmv_sample(T(2, 64), T(2)), "CUDA"),
    ]
    for i, (f, text) in enumerate(cases):
        with pytest.raises(ValueError, match=text):
            f()
            raise AssertionError(f"case {i} ({text}) was not refused")


def test_binding_refuses_the_same_without_its_cpp_form(q, monkeypatch):
    monkeypatch.setattr(q, "_host", q._NoHost())
    test_binding_refuses_before_any_call(q)
