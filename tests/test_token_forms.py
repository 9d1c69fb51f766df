"""Scratch of the experts' products by the form of the call, and numbers past 32 bits: host checks."""
import pytest
import torch

F32, F16, BF16 = 0, 1, 2


@pytest.fixture(scope="module")
def q():
    from bit_weight_only_packed_gb300 import build
    build.build()
    from bit_weight_only_packed_gb300 import qmv
    return qmv


def up(n):
    return -(-n // 256) * 256


def test_experts_scratch_of_a_form(q):
    R, K = 64, 256
    p = q.W4Pack(16 * R, K, 128)

    def form(M, T, weighted=0, x=4096, ldx=K, per_pair=0, dt=F16, act=0, rows=R):
        return q.lib().qmv_w4_experts_form_bytes(p.handle, rows, M, T, weighted, x, ldx, per_pair, dt, act)

    for M, T in ((1, 1), (1, 8), (16, 8), (17, 8), (129, 1), (512, 4), (4096, 8)):
        P = M * T
        order = 256 + up(4 * P) + up(16 * P) if P > 128 else 0
        made = lambda rows: up(4 * rows) + up(2 * rows * K)
        parts = up(4 * P * R)
        assert form(M, T) == form(M, T, per_pair=1) == order                # fp16 as it is
        assert form(M, T, weighted=1) == order + parts
        for kw in (dict(dt=BF16), dict(act=1, ldx=2 * K), dict(x=4098), dict(ldx=K + 4), dict(dt=BF16, act=2, ldx=2 * K)):
            assert form(M, T, **kw) == order + made(M), kw
            assert form(M, T, per_pair=1, **kw) == order + made(P), kw
            assert form(M, T, per_pair=1, weighted=1, **kw) == order + made(P) + parts, kw
        # one workspace holds every form, of fewer tokens too
        every = q.qmv_w4_experts_workspace_bytes(p, R, M, T)
        assert form(M, T, per_pair=1, weighted=1, dt=BF16) <= every
        assert q.qmv_w4_experts_workspace_bytes(p, R, max(M // 2, 1), T) <= every
    for kw in (dict(rows=48), dict(rows=0), dict(M=0), dict(T=0), dict(M=4097), dict(T=65)):
        assert form(**{**dict(M=1, T=1, weighted=1), **kw}) == 0, kw
    assert q.lib().qmv_w4_experts_form_bytes(None, R, 1, 1, 1, 4096, K, 0, F16, 0) == 0


def test_experts_form_calls(q):
    R, K = 64, 256
    p = q.W4Pack(4 * R, K, 128)
    assert q.lib().qmv_w4_bind(p.handle, 1 << 40) == 0                      # an address that nothing reads

    def call(M=2, T=2, ids=64, w=None, x=4096, ldx=K, pp=0, xd=BF16, act=0, y=65536, ldy=R, yd=F32, ws=1 << 20, wb=1 << 30):
        return q.lib().qmv_w4_experts_form(p.handle, R, M, T, ids, w, x, ldx, pp, xd, act, y, ldy, yd, ws, wb, None)

    need = q.lib().qmv_w4_experts_form_bytes(p.handle, R, 2, 2, 0, 4096, K, 0, BF16, 0)
    assert 0 < need < q.qmv_w4_experts_workspace_bytes(p, R, 2, 2)
    assert call(ws=None) == call(wb=need - 1) == -7
    assert call(w=256, wb=need) == -7                                       # the sums need more
    assert call(wb=need, ws=(1 << 20) + 128) == -3
    for kw in (dict(ids=None), dict(x=None), dict(y=None), dict(xd=F32), dict(act=3), dict(y=4096), dict(x=1 << 20), dict(y=(1 << 20) + 256)):
        assert call(**kw) == -1, kw
    for kw in (dict(ldx=K - 1), dict(ldy=R - 1)):
        assert call(**kw) == -4, kw
    assert call(M=4097) == call(T=65) == -2


def test_numbers_past_32_bits_are_refused_not_cut_off(q):
    far = 1 << 32
    f16 = lambda *s: torch.zeros(*s, dtype=torch.float16)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    p = q.W4Pack(128, 256, 128)
    rows = torch.empty(far + 1, 1, device="meta")
    cases = [
        (lambda: q.qmv_sample(torch.zeros(2, 64), torch.zeros(2), top_k=far + 5), "top_k"),
        (lambda: q.qmv_sample(torch.zeros(2, 64), torch.zeros(2), top_k=2.5), "top_k"),
        (lambda: q.qmv_sample(rows, torch.empty(far + 1, device="meta")), "logits's rows"),
        (lambda: q.qmv_route(rows, 1), "logits's rows"),
        (lambda: q.qmv_route(torch.zeros(2, 64), far + 2), "top_k"),
        (lambda: q.qmv_route(torch.zeros(2, 64), 2, groups=far + 1), "groups"),
        (lambda: q.qmv_route(torch.zeros(2, 64), 2, score=far), "score"),
        (lambda: q.qmv_qk_norm_rope(rows, 1, 0, 1), "qkv's rows"),
        (lambda: q.qmv_qk_norm_rope(f16(2, 192), far + 2, 1, 64), "n_q"),
        (lambda: q.qmv_w4_experts(p, far + 64, i32(2, 2), f16(2, 256)), "rows_per_expert"),
        (lambda: q.qmv_w4_experts(p, 64, i32(2, 2), f16(2, 256), act=far), "act"),
        (lambda: q.qmv_w4_experts_workspace_bytes(p, 64, far + 1, 1), "M"),
        (lambda: q.Rope(64, scaling=far, device="cpu"), "scaling"),
    ]
    for i, (f, text) in enumerate(cases):
        with pytest.raises(ValueError, match=text):
            f()
            raise AssertionError(f"case {i} ({text}) was not refused")
