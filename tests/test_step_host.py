"""The verification-step calls check their arguments on the host: status codes of
the C ABI and ValueErrors of the binding, before any device is touched."""
import ctypes

import pytest
import torch

F32, F16, BF16 = 0, 1, 2


@pytest.fixture(scope="module")
def q():
    from bit_weight_only_packed_gb300 import build
    build.build()
    from bit_weight_only_packed_gb300 import qmv
    return qmv


@pytest.mark.parametrize("N,K,group,dt,zeros,status", [
    (64, 256, 128, F16, 1, 0), (1, 32, 32, BF16, 0, 0), (33, 160, 128, F16, 1, 0), (64, 256, 64, F16, 0, 0),
    (64, 256, 16, F16, 1, -1), (64, 256, 256, F16, 1, -1), (64, 256, 0, F16, 1, -1),
    (64, 256, 128, F32, 1, -1), (64, 256, 128, 3, 1, -1),
    (0, 256, 128, F16, 1, -4), (64, 0, 128, F16, 1, -4), (64, 48, 32, F16, 1, -4), (-5, 64, 32, F16, 1, -4),
    (2**31 - 1, 64, 32, F16, 1, -4), (64, 131072, 32, F16, 1, 0), (64, 131104, 32, F16, 1, -2),
])
def test_w4_create(q, N, K, group, dt, zeros, status):
    h, nb = ctypes.c_void_p(), ctypes.c_size_t()
    assert q.lib().qmv_w4_create(ctypes.byref(h), N, K, group, dt, zeros, ctypes.byref(nb)) == status
    if status:
        assert not h.value
        return
    block = 2048 + 128 // group * 32 * (3 if zeros else 2)
    assert nb.value == -(-N // 32) * -(-K // 128) * block
    v = [ctypes.c_int() for _ in range(5)]
    assert q.lib().qmv_w4_info(h, *map(ctypes.byref, v)) == 0
    assert [i.value for i in v] == [N, K, group, dt, zeros]
    assert q.lib().qmv_w4_destroy(h) == 0
    assert q.lib().qmv_w4_create(None, 64, 64, 32, F16, 1, None) == -1


def test_w4_calls(q):
    lib = q.lib()
    p = q.W4Pack(64, 256, 128)
    h = p.handle
    # nothing bound yet
    assert lib.qmv_w4_gemv(h, 1, 16, 256, F16, 16, 64, F32, None) == -1
    assert lib.qmv_w4_unpack(h, 16, None) == -1
    assert lib.qmv_w4_pack(h, 16, 16, None, 16, None) == -1          # zero points are missing
    assert lib.qmv_w4_pack(q.W4Pack(64, 256, 128, zeros=False).handle, 16, 16, 16, 16, None) == -1
    assert lib.qmv_w4_pack(h, 12, 16, 16, 16, None) == -3
    assert lib.qmv_w4_pack(h, 16, 16, 16, 24, None) == -3
    assert lib.qmv_w4_bind(h, None) == -1 and lib.qmv_w4_bind(h, 24) == -3
    assert lib.qmv_w4_bind(h, 4096) == 0                               # an address that nothing reads
    for M in (0, -1, 4097):
        assert lib.qmv_w4_gemv(h, M, 16, 256, F16, 16, 64, F32, None) == -1
    assert lib.qmv_w4_gemv(h, 1, None, 256, F16, 16, 64, F32, None) == -1
    assert lib.qmv_w4_gemv(h, 1, 16, 256, F32, 16, 64, F32, None) == -1
    assert lib.qmv_w4_gemv(h, 1, 16, 256, F16, 16, 64, 3, None) == -1
    assert lib.qmv_w4_gemv(h, 1, 16, 255, F16, 16, 64, F32, None) == -4
    assert lib.qmv_w4_gemv(h, 1, 16, 256, F16, 16, 63, F32, None) == -4
    assert lib.qmv_w4_gemv(h, 1, 17, 256, F16, 16, 64, F32, None) == -3
    assert lib.qmv_w4_gemv(h, 1, 16, 256, F16, 18, 64, F32, None) == -3
    assert lib.qmv_w4_gemv(None, 1, 16, 256, F16, 16, 64, F32, None) == -1
    assert lib.qmv_w4_info(None, None, None, None, None, None) == -1
    assert lib.qmv_w4_destroy(None) == -1


def test_block_norm_calls(q):
    def call(M=2, D=64, y=16, ldy=64, yd=F32, r=16, ldr=64, gpo=None, gate=None, ldg=0, gpr=16, eps=1e-6,
             h=32, ldh=64, out=48, ldo=64, dt=F16):
        return q.lib().qmv_block_norm(M, D, y, ldy, yd, r, ldr, gpo, gate, ldg, 1.0, 1.0, gpr, 0.0, eps, h, ldh,
                                      out, ldo, dt, None)

    for kw in (dict(M=0), dict(D=0), dict(y=None), dict(r=None), dict(gpr=None), dict(out=None), dict(yd=3),
               dict(dt=F32), dict(eps=-1.0), dict(eps=float("nan"))):
        assert call(**kw) == -1, kw
    # an output on top of an input or of the other output
    for kw in (dict(out=16), dict(h=48), dict(y=32), dict(gate=48)):
        assert call(**kw) == -1, kw
    assert call(D=65537, ldy=70000, ldr=70000, ldh=70000, ldo=70000) == -2
    for kw in (dict(ldy=63), dict(ldr=63), dict(ldh=63), dict(ldo=63), dict(gate=16, ldg=63), dict(h=16, ldh=65)):
        assert call(**kw) == -4, kw
    for kw in (dict(y=18), dict(y=17, yd=F16), dict(r=17), dict(gpo=17), dict(gate=17), dict(gpr=17), dict(h=17),
               dict(out=17)):
        assert call(**kw) == -3, kw


def test_softmax_calls(q):
    def call(rows=2, V=64, x=16, ldl=64, dt=F32, t=None, t0=1.0, out=32, ldo=64):
        return q.lib().qmv_softmax(rows, V, x, ldl, dt, t, t0, out, ldo, None)

    for kw in (dict(rows=0), dict(V=0), dict(x=None), dict(out=None), dict(dt=3), dict(t0=-0.5),
               dict(t0=float("nan"))):
        assert call(**kw) == -1, kw
    for kw in (dict(ldl=63), dict(ldo=63), dict(out=16, ldo=65), dict(out=16, dt=F16)):
        assert call(**kw) == -4, kw
    for kw in (dict(x=18), dict(x=17, dt=F16), dict(out=34), dict(t=18)):
        assert call(**kw) == -3, kw


def test_verify_calls(q):
    def call(B=2, S=3, V=64, p=16, dq=16, d=16, n=None, ua=16, us=16, tok=16, na=16):
        return q.lib().qmv_verify_draft(B, S, V, p, dq, d, n, ua, us, tok, na, None)

    for kw in (dict(B=0), dict(S=-1), dict(V=0), dict(p=None), dict(d=None), dict(ua=None), dict(us=None),
               dict(tok=None), dict(na=None)):
        assert call(**kw) == -1, kw
    for kw in (dict(B=65536), dict(S=1025), dict(V=(1 << 20) + 1)):
        assert call(**kw) == -2, kw
    for kw in (dict(p=18), dict(dq=18), dict(d=18), dict(n=18), dict(ua=18), dict(us=18), dict(tok=18), dict(na=18)):
        assert call(**kw) == -3, kw


def test_binding_refuses_before_any_call(q):
    f16 = lambda *s: torch.zeros(*s, dtype=torch.float16)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    p = q.W4Pack(64, 256, 128)
    T = torch.zeros
    cases = [
        (lambda: q.W4Pack(64, 256, 128, scale_dtype=torch.float32), "scale_dtype"),
        (lambda: p.pack_weights(T(64, 256, dtype=torch.int8), f16(64, 2), T(64, 2, dtype=torch.uint8)), "codes: expected"),
        (lambda: p.pack_weights(T(64, 255, dtype=torch.uint8), f16(64, 2), T(64, 2, dtype=torch.uint8)), "codes: needs"),
        (lambda: p.pack_weights(T(64, 256, dtype=torch.uint8), f16(64, 2).bfloat16(), None), "scales: expected"),
        (lambda: p.pack_weights(T(64, 256, dtype=torch.uint8), f16(64, 2), None), "zeros: given exactly"),
        (lambda: p.pack_weights(T(64, 256, dtype=torch.uint8), f16(64, 2), T(64, 1, dtype=torch.uint8)), "zeros: needs"),
        (lambda: p.pack_weights(T(64, 256, dtype=torch.uint8), f16(64, 2), T(64, 2, dtype=torch.uint8)), "CUDA"),
        (lambda: p.bind_packed(T(16, dtype=torch.uint8)), "packed: needs"),
        (lambda: p.unpack_codes(), "holds no weights"),
        (lambda: q.qmv_w4_gemv(p, T(1, 256)), "x: expected"),
        (lambda: q.qmv_w4_gemv(p, f16(1, 255)), r"x: expected \[1, 256\]"),
        (lambda: q.qmv_w4_gemv(p, f16(256, 2).t()), "rows must be contiguous"),
        (lambda: q.qmv_w4_gemv(p, f16(1, 256).expand(4, 256)), "rows overlap"),
        (lambda: q.qmv_w4_gemv(p, f16(1, 256)), "holds no weights"),
        (lambda: q.qmv_block_norm(f16(2, 64), T(2, 64), T(64)), "residual: expected"),
        (lambda: q.qmv_block_norm(f16(2, 64), f16(2, 64), T(64)), "gamma_pre: expected"),
        (lambda: q.qmv_block_norm(f16(2, 63), f16(2, 64), f16(64)), "y: expected"),
        (lambda: q.qmv_block_norm(f16(2, 64), f16(2, 64), f16(64), gamma_post=f16(63)), "gamma_post: needs"),
        (lambda: q.qmv_block_norm(f16(2, 64), f16(2, 64), f16(64), gate=f16(1, 64)), "gate: expected"),
        (lambda: q.qmv_block_norm(f16(2, 64), f16(2, 64), f16(64), h_out=T(2, 64)), "h_out: expected"),
        (lambda: q.qmv_block_norm(f16(2, 64), f16(2, 64), f16(64)), "CUDA"),
        (lambda: q.qmv_softmax(T(2, 3, 4)), "logits: expected"),
        (lambda: q.qmv_softmax(T(2, 64), temperature=T(3)), "temperature: needs 2"),
        (lambda: q.qmv_softmax(T(2, 64), out=f16(2, 64)), "out: expected"),
        (lambda: q.qmv_verify_draft(T(2, 64), None, i32(2, 0), T(2, 0), T(2)), "target: expected"),
        (lambda: q.qmv_verify_draft(T(2, 4, 8), T(2, 4, 8), i32(2, 3), T(2, 3), T(2)), "draft_probs: needs 48"),
        (lambda: q.qmv_verify_draft(T(2, 4, 8), None, T(2, 3), T(2, 3), T(2)), "draft: expected"),
        (lambda: q.qmv_verify_draft(T(2, 4, 8), None, i32(2, 3), T(2, 2), T(2)), "u_accept: needs"),
        (lambda: q.qmv_verify_draft(T(2, 4, 8), None, i32(2, 3), T(2, 3), T(3)), "u_sample: needs"),
        (lambda: q.qmv_verify_draft(T(2, 4, 8), None, i32(2, 3), T(2, 3), T(2), n_draft=i32(3)), "n_draft: needs"),
        (lambda: q.qmv_verify_draft(T(8, 4, 2).permute(2, 1, 0), None, i32(2, 3), T(2, 3), T(2)), "contiguous"),
        (lambda: q.qmv_verify_draft(T(2, 4, 8), None, i32(2, 3), T(2, 3), T(2)), "CUDA"),
    ]
    for call, msg in cases:
        with pytest.raises(ValueError, match=msg):
            call()


def test_outputs_on_top_of_inputs(q):
    # every call here is in order but for an output that shares memory with an input or
    # the other output; addresses that nothing reads
    lib, M, D, at = q.lib(), 2, 64, 1 << 20
    far = [at + 65536 * i for i in range(12)]
    p = q.W4Pack(64, 256, 128)
    assert lib.qmv_w4_bind(p.handle, far[0]) == 0
    nb = p.packed_bytes
    row = 2 * 256 * 2                                    # bytes of x, M = 2
    for x, y in ((far[1], far[1]), (far[1], far[1] + row - 2), (far[1] + 254, far[1]), (far[1], far[0] + nb - 4)):
        assert lib.qmv_w4_gemv(p.handle, 2, x, 256, F16, y, 64, F16, None) == -1, (x, y)
    # columns that cross the next row's, and strides that differ
    assert lib.qmv_w4_gemv(p.handle, 2, far[1], 320, F16, far[1] + 2 * 257, 320, F16, None) == -1
    assert lib.qmv_w4_gemv(p.handle, 2, far[1], 320, F16, far[1] + 2 * 256, 321, F16, None) == -1
    assert lib.qmv_w4_unpack(p.handle, far[0] + nb - 1, None) == -1
    for codes, scales, zeros in ((far[2] + 2048, far[3], far[4]), (far[1], far[2], far[4]), (far[1], far[3], far[2] + 64)):
        assert lib.qmv_w4_pack(p.handle, codes, scales, zeros, far[2], None) == -1

    def norm(y=far[0], r=far[1], gpo=far[2], gate=far[3], ldg=D, gpr=far[4], h=far[5], out=far[6], ldo=D):
        return lib.qmv_block_norm(M, D, y, D, F16, r, D, gpo, gate, ldg, 1.0, 1.0, gpr, 0.0, 1e-6, h, D, out, ldo,
                                  F16, None)

    n = 2 * M * D
    for base in (far[0], far[1], far[2], far[3], far[4]):
        last = base + (n if base in (far[0], far[1], far[3]) else 2 * D) - 2
        for o in (base, last, base - n + 2):
            assert norm(out=o) == -1, (base, o)
            if (base, o) != (far[1], far[1]):            # h_out may be the residual itself
                assert norm(h=o) == -1, (base, o)
    assert norm(out=far[5] + 2) == -1
    assert norm(out=far[3] + 2 * D - 2, ldg=0) == -1
    assert norm(out=far[0] + 2, ldo=D + 1) == -1

    def softmax(x=far[0], dt=F32, t=far[1], out=far[2], ldo=D):
        return lib.qmv_softmax(M, D, x, D, dt, t, 1.0, out, ldo, None)

    for o in (far[0] + 4, far[0] + 4 * M * D - 4, far[0] - 4 * M * D + 4, far[1], far[1] + 4):
        assert softmax(out=o) == -1, o
    assert softmax(dt=F16, out=far[0] + 2 * M * D - 4) == -1

    B, S, V = 2, 3, 64
    args = dict(p=far[0], dq=far[1], d=far[2], n=far[3], ua=far[4], us=far[5], tok=far[6], na=far[7])
    sizes = dict(p=B * (S + 1) * V, dq=B * S * V, d=B * S, n=B, ua=B * S, us=B)
    verify = lambda **kw: lib.qmv_verify_draft(B, S, V, *{**args, **kw}.values(), None)
    for name, size in sizes.items():
        for o in (args[name], args[name] + 4 * size - 4):
            assert verify(tok=o) == -1 and verify(na=o) == -1, name
    assert verify(na=far[6] + 4 * (B * (S + 1) - 1)) == -1
