"""The decode-step calls on other streams, in captured graphs, on several host threads, next to each
other, and after refused launches."""
import subprocess
import sys
import threading

import pytest
import torch

from conftest import ROOT
from gpu_util import GuardBuf, qmv
from test_gpu_step import BF16, F16, F32, gen, make_w4
from test_gpu_token import distinct, draw_ref, logits_like, randn

pytestmark = pytest.mark.gpu


def calls(seed=1):
    """One call of each operator, each with inputs of its own, as functions of a stream."""
    q = qmv()
    M, E, T, R, K, V = 9, 16, 4, 128, 512, 70000
    p, _, _ = make_w4(E * R, K, 64, True, BF16, seed)
    ids = distinct(M, T, E, seed)
    x, w = randn(seed, M, K).to(BF16), torch.rand(M, T, generator=gen(seed), device="cuda")
    gated = randn(seed, M, T, 2 * K).to(F16)
    qkv = randn(seed, M, 6 * 128)
    g = (1 + 0.1 * randn(seed, 128)).to(F16)
    rope, pos = q.Rope(128), torch.arange(M, device="cuda", dtype=torch.int32) * 7 + seed
    logits, bias = randn(seed, M, E), 0.1 * randn(seed + 1, E)
    big = logits_like(seed, M, V)
    u = torch.rand(M, generator=gen(seed), device="cuda")
    ws = q.qmv_w4_experts_workspace(p, R, M, T)
    return [
        lambda s=None: q.qmv_qk_norm_rope(qkv, 4, 2, 128, rope, pos, g, g, stream=s),
        lambda s=None: q.qmv_route(logits, T, score=q.QMV_SCORE_SIGMOID, bias=bias, groups=4, group_k=2, group_top=2, stream=s),
        lambda s=None: q.qmv_w4_experts(p, R, ids, x, workspace=ws, stream=s),
        lambda s=None: q.qmv_w4_experts(p, R, ids, gated, weights=w, act=q.QMV_ACT_GELU, stream=s),
        lambda s=None: q.qmv_sample(big, u, 0.8, 40, 0.9, stream=s),
        lambda s=None: q.qmv_sample(big, u, 0.8, 0, 0.9, 0.001, stream=s),
    ]


def tensors(r):
    return list(r) if isinstance(r, tuple) else [r]


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(tensors(a), tensors(b)))


def test_other_streams_and_raw_handles():
    for f in calls():
        ref = f()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        a = f(s)
        with torch.cuda.stream(s):
            b = f()
        c = f(s.cuda_stream)
        torch.cuda.synchronize()
        assert same(ref, a) and same(ref, b) and same(ref, c)


def test_streams_at_once_and_memory_that_is_freed_early():
    fs = calls()
    refs = [f() for f in fs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in fs]
    outs = []
    for _ in range(5):
        for s, f in zip(streams, fs):
            outs.append((f, f(s)))
        # what these leave is handed out again while they may still run
        torch.full((1 << 20,), 7.0, device="cuda")
    torch.cuda.synchronize()
    for f, o in outs:
        assert same(refs[fs.index(f)], o)


def test_inputs_that_are_freed_right_after_the_call():
    q = qmv()
    s = torch.cuda.Stream()
    for i in range(8):
        x, u = logits_like(i, 6, 50000), torch.rand(6, generator=gen(i), device="cuda")
        ref = q.qmv_sample(x, u, 0.9, 20, 0.9)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(2_000_000)
        out = q.qmv_sample(x, u, 0.9, 20, 0.9, stream=s)
        del x, u
        junk = [torch.zeros(6 * 50000, device="cuda"), torch.zeros(6, device="cuda")]
        torch.cuda.synchronize()
        assert torch.equal(ref, out)
        del junk


def test_captured_replayed_and_with_changed_inputs():
    q = qmv()
    M, E, T, R, K, V = 5, 12, 3, 64, 256, 9000
    p, _, _ = make_w4(E * R, K, 128, False, F16, 4)
    x, logits, big = randn(1, M, K).to(F16), randn(2, M, E), logits_like(3, M, V)
    u = torch.rand(M, generator=gen(4), device="cuda")
    ws = q.qmv_w4_experts_workspace(p, R, M, T)

    def step():
        ids, w = q.qmv_route(logits, T)
        return (*[ids, w], q.qmv_w4_experts(p, R, ids, x, weights=w, workspace=ws), q.qmv_sample(big, u, 0.7, 0, 0.8))

    step()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):                      # two graphs of one workspace, one after the other
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    for i in range(4):
        x.copy_(randn(10 + i, M, K))
        logits.copy_(randn(20 + i, M, E))
        big.copy_(logits_like(30 + i, M, V))
        ref = step()
        for g, o in zip(graphs, outs):
            g.replay()
            torch.cuda.synchronize()
            assert all(same(a, b) for a, b in zip(ref, o))


def test_ids_and_logits_from_the_kernel_before():
    # the products read ids ahead of their wait for the kernel that makes x: those come from further back;
    # without such a kernel they come from the one before
    q = qmv()
    M, E, T, R, K = 4, 32, 4, 64, 256
    for dt in (F16, BF16):
        p, _, _ = make_w4(E * R, K, 64, True, dt, 6)
        x = randn(1, M, K).to(dt)
        outs, idss = [], []
        q.qmv_set_pdl(True)
        try:
            for i in range(20):
                logits = randn(50 + i, M, E)
                ids, w = q.qmv_route(logits, T)
                outs.append((q.qmv_w4_experts(p, R, ids, x), q.qmv_w4_experts(p, R, ids, x, weights=w)))
                idss.append((ids, w))
        finally:
            q.qmv_set_pdl(False)
        torch.cuda.synchronize()
        for (ids, w), (a, b) in zip(idss, outs):
            torch.cuda.synchronize()
            assert torch.equal(a, q.qmv_w4_experts(p, R, ids, x)) and torch.equal(b, q.qmv_w4_experts(p, R, ids, x, weights=w))


def test_weights_bound_again_between_calls():
    q = qmv()
    p, _, _ = make_w4(8 * 32, 256, 64, True, F16, 1)
    p2, _, _ = make_w4(8 * 32, 256, 64, True, F16, 2)
    ids, x = distinct(3, 2, 8, 1), randn(1, 3, 256).to(F16)
    a, b = q.qmv_w4_experts(p, 32, ids, x), q.qmv_w4_experts(p2, 32, ids, x)
    p.bind_packed(p2.packed.clone())
    assert torch.equal(q.qmv_w4_experts(p, 32, ids, x), b) and not torch.equal(a, b)


def test_several_host_threads():
    fs = calls()
    refs = [f() for f in fs]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                mine = calls()                 # workspaces of its own
                for _ in range(6):
                    for k, f in enumerate(mine):
                        if not same(f(), refs[k]):
                            wrong.append((i, k))
            s.synchronize()
        except Exception as e:              # noqa: BLE001
            wrong.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not wrong, wrong[:4]
    assert qmv().qmv_device_error(clear=True) == 0


@pytest.mark.parametrize("M,T,weighted,act", [(3, 2, False, 0), (40, 4, True, 1), (200, 4, True, 0), (200, 4, False, 2)])
def test_experts_workspace_bounds_and_contents(M, T, weighted, act):
    q = qmv()
    E, R, K = 12, 64, 320
    p, _, _ = make_w4(E * R, K, 32, True, BF16, 3)
    ids = distinct(M, T, E, 2)
    x = randn(1, M, T, K * (2 if act else 1)).to(BF16)
    w = torch.rand(M, T, generator=gen(5), device="cuda") if weighted else None
    n = q.qmv_w4_experts_workspace_bytes(p, R, M, T)
    outs = []
    for fill in (0x00, 0x5A, 0xFF):
        g = GuardBuf(n, fill=fill)
        outs.append(q.qmv_w4_experts(p, R, ids, x, weights=w, act=act, workspace=g.view(torch.uint8, (n,))))
        torch.cuda.synchronize()
        g.check("workspace")
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    assert torch.equal(outs[0], q.qmv_w4_experts(p, R, ids, x, weights=w, act=act))
    with pytest.raises(ValueError, match="workspace"):
        q.qmv_w4_experts(p, R, ids, x, weights=w, act=act, workspace=torch.empty(n - 1, dtype=torch.uint8, device="cuda"))


def test_outputs_over_inputs_are_refused():
    q = qmv()
    x = randn(1, 4, 512).to(F16)
    with pytest.raises(q.QmvError):
        q.qmv_qk_norm_rope(x, 2, 1, 128, q=x[:, 128:384])
    logits = randn(1, 4, 64)
    with pytest.raises(q.QmvError):
        q.qmv_route(logits, 8, weights=logits.view(-1)[:32].view(4, 8))
    u = torch.rand(4, device="cuda")
    with pytest.raises(q.QmvError):
        q.qmv_sample(logits, u, tokens=u.view(torch.int32))
    for bad in (dict(temperature=-1.0), dict(top_k=-1), dict(top_p=1.5), dict(min_p=-0.5), dict(top_p=float("nan"))):
        with pytest.raises(q.QmvError):
            q.qmv_sample(logits, u, **bad)
    for bad in (dict(score=2), dict(groups=5), dict(groups=4, group_k=5), dict(groups=4, group_k=1, group_top=3), dict(groups=64)):
        with pytest.raises(q.QmvError):
            q.qmv_route(logits, 8, **bad)
    with pytest.raises(q.QmvError):
        q.qmv_route(logits, 65)
    with pytest.raises(q.QmvError):
        q.qmv_route(logits, 0)


def test_views_that_the_fast_form_leaves_to_the_other():
    q = qmv()
    wide = logits_like(1, 6, 3000)
    u = torch.rand(12, generator=gen(1), device="cuda")
    a = q.qmv_sample(wide[:, 100:2900], u[::2].contiguous(), 0.8, 30, 0.9)
    b = q.qmv_sample(wide[:, 100:2900].contiguous(), u[::2].contiguous(), 0.8, 30, 0.9)
    assert torch.equal(a, b)
    assert torch.equal(q.qmv_route(wide[:, :64], 4)[0], q.qmv_route(wide[:, :64].contiguous(), 4)[0])
    x = randn(2, 6, 1024).to(BF16)
    r, pos = q.Rope(64), torch.arange(6, device="cuda", dtype=torch.int32)
    for s, t in zip(q.qmv_qk_norm_rope(x[:, 8:776], 4, 2, 128, r, pos), q.qmv_qk_norm_rope(x[:, 8:776].contiguous(), 4, 2, 128, r, pos)):
        assert torch.equal(s, t)
    with pytest.raises(ValueError):
        q.qmv_sample(wide[:, ::2], u[:6])
    with pytest.raises(ValueError):
        q.qmv_route(wide.t(), 4)


def test_the_python_form_gives_the_same(monkeypatch):
    q = qmv()
    assert not isinstance(q._host, q._NoHost)
    p, _, _ = make_w4(6 * 64, 256, 64, True, BF16, 2)
    x, g = randn(1, 9, 512), (randn(2, 64) * 0.2).to(BF16)
    r, pos = q.Rope(64, scaling=q.QMV_SCALE_NTK, factor=4.0), torch.arange(9, device="cuda", dtype=torch.int32)
    bias, lg = randn(3, 6), logits_like(4, 9, 5003)
    u, per = torch.rand(9, generator=gen(5), device="cuda"), torch.rand(9, generator=gen(6), device="cuda")

    def run():
        out = list(q.qmv_qk_norm_rope(x, 4, 2, 64, r, pos, g, g, 1.0, 1e-5, q.QMV_BF16))
        out += q.qmv_qk_norm_rope(x.to(F16), 4, 0, 64)[:1]
        ids, w = q.qmv_route(x[:, :6].contiguous(), 2, q.QMV_SCORE_SIGMOID, bias, 3, 2, 2, True, 2.5)
        out += [ids, w, q.qmv_w4_experts(p, 64, ids, x[:, :256].to(BF16).contiguous()),
                q.qmv_w4_experts(p, 64, ids, x.to(BF16), weights=w, act=q.QMV_ACT_SILU, y_dtype=q.QMV_BF16)]
        return out + [q.qmv_sample(lg, u, 0.7, 40, 0.9, 0.01), q.qmv_sample(lg, u, per, 0, per, per * 0.1)]

    ref = run()
    monkeypatch.setattr(q, "_host", q._NoHost())
    for a, b in zip(run(), ref):
        assert a.dtype == b.dtype and a.shape == b.shape and torch.equal(a, b)


# As for the calls before these: the legacy stream may not be used while a stream that waits for it is
# captured, so the runtime refuses the launch and nothing runs on the device.
REFUSED = """
import sys; sys.path[:0] = [{root!r}, {root!r} + '/tests']
import ctypes
import torch
from bit_weight_only_packed_gb300 import qmv as q
from test_gpu_step import make_w4, F16
lib, rt = q.lib(), ctypes.CDLL('libcudart.so.13')
p, _, _ = make_w4(4 * 32, 256, 128, True, F16, 1)
x = torch.ones(4, 512, device='cuda', dtype=F16)
ids, w = torch.zeros(4, 2, device='cuda', dtype=torch.int32), torch.ones(4, 2, device='cuda')
y = torch.empty(4, 2, 32, device='cuda')
ws = q.qmv_w4_experts_workspace(p, 32, 4, 2)
lg, u, tok = torch.ones(4, 64, device='cuda'), torch.zeros(4, device='cuda'), torch.empty(4, device='cuda', dtype=torch.int32)
oq, ok = torch.empty(4, 128, device='cuda', dtype=F16), torch.empty(4, 64, device='cuda', dtype=F16)
a = lambda t: t.data_ptr()
CALLS = {{
    'rope': lambda s: lib.qmv_qk_norm_rope(4, 2, 1, 64, a(x), 512, q.QMV_F16, None, None, 0, 0, 1.0, None, None, 0.0, 1e-6, a(oq),
                                           128, a(ok), 64, q.QMV_F16, s),
    'route': lambda s: lib.qmv_route(4, 64, 2, a(lg), 64, q.QMV_F32, 0, None, 1, 1, 1, 1, 1.0, a(ids), a(w), s),
    'experts': lambda s: lib.qmv_w4_experts(p.handle, 32, 4, 2, a(ids), None, a(x), 512, 0, q.QMV_F16, 0, a(y), 32, q.QMV_F32, a(ws),
                                            ws.numel(), s),
    'sample': lambda s: lib.qmv_sample(4, 64, a(lg), 64, q.QMV_F32, None, 1.0, None, 0, None, 1.0, None, 0.0, a(u), a(tok), s),
}}
call = CALLS[{name!r}]
assert call(torch.cuda.current_stream().cuda_stream) == 0
torch.cuda.synchronize()
side, graph = ctypes.c_void_p(), ctypes.c_void_p()
assert rt.cudaStreamCreate(ctypes.byref(side)) == 0             # one that waits for the legacy stream
assert rt.cudaStreamBeginCapture(side, 0) == 0
rc = call(None)
left = rt.cudaPeekAtLastError()
rt.cudaStreamEndCapture(side, ctypes.byref(graph))              # the capture was given up
assert rc == q.QMV_ERR_CUDA and q.qmv_last_cuda_error() != 0, rc
print('left', left)
"""


@pytest.mark.parametrize("name", ["rope", "route", "experts", "sample"])
def test_a_refused_launch_leaves_no_error_behind(name):
    r = subprocess.run([sys.executable, "-c", REFUSED.format(root=ROOT, name=name)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "left 0" in r.stdout, r.stdout


# ------------------------------------------------------------ the largest --

def test_sample_offsets_past_32_bits():
    # the last rows of 4.4 G logits in 16 bits lie past 2^31 elements
    q = qmv()
    rows, V = 16800, 262144
    x = torch.full((rows, V), -20.0, dtype=BF16, device="cuda")
    at = torch.randint(0, V, (rows,), generator=gen(1), device="cuda")
    x.scatter_(1, at[:, None], 5.0)
    u = torch.rand(rows, generator=gen(2), device="cuda") * 0.5
    assert torch.equal(q.qmv_sample(x, u, 0.5, 8).long(), at)
    last = x[-3:].clone()
    assert q.qmv_sample(x, u, 0.9, 0, 0.9)[-3:].tolist() == [draw_ref(last[i].float().cpu().numpy(), u[-3 + i].item(), 0.9, 0, 0.9, 0.0)
                                                             for i in range(3)]


def test_rope_and_route_offsets_past_32_bits():
    q = qmv()
    M, D = 70000, 128
    x = torch.zeros(M, 256 * D, dtype=F16, device="cuda")          # 2.3 G elements a tensor
    x[-2:] = randn(1, 2, 256 * D).to(F16)
    pos = torch.arange(M, device="cuda", dtype=torch.int32)
    r = q.Rope(D)
    a = q.qmv_qk_norm_rope(x, 250, 6, D, r, pos)
    b = q.qmv_qk_norm_rope(x[-2:], 250, 6, D, r, pos[-2:])
    assert torch.equal(a[0][-2:], b[0]) and torch.equal(a[1][-2:], b[1]) and not bool(a[0][1000].any())
    del a, x
    M, E = 2_200_000, 1024
    lg = torch.zeros(M, E, dtype=BF16, device="cuda")
    lg[-5:] = randn(2, 5, E).to(BF16)
    ids, w = q.qmv_route(lg, 4)
    i2, w2 = q.qmv_route(lg[-5:], 4)
    assert torch.equal(ids[-5:], i2) and torch.equal(w[-5:], w2) and ids[7].tolist() == [0, 1, 2, 3]


def test_experts_most_of_everything():
    # the most pairs, and a weight buffer past 2^31 bytes whose last experts are taken
    q = qmv()
    M, T, E, R, K = 4096, 8, 16, 32, 64
    p, _, w = make_w4(E * R, K, 64, True, F16, 1, exact=True)
    ids = distinct(M, T, E, 1)
    x = torch.randint(-2, 3, (M, K), generator=gen(1), device="cuda").to(F16)
    y = q.qmv_w4_experts(p, R, ids, x).double()
    full = torch.einsum("mk,erk->mer", x.double(), w.view(E, R, K))
    assert torch.equal(y, full.gather(1, ids.long()[:, :, None].expand(M, T, R)))
    E, R, K, group = 520, 2048, 4096, 128
    nb = q.W4Pack(E * R, K, group, F16, False).packed_bytes
    assert nb > 2 ** 31
    big = q.W4Pack(E * R, K, group, F16, False)
    one, _, wl = make_w4(R, K, group, False, F16, 9, exact=True)
    packed = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    packed[-one.packed.numel():] = one.packed
    big.bind_packed(packed)
    x = torch.randint(-2, 3, (2, K), generator=gen(2), device="cuda").to(F16)
    y = q.qmv_w4_experts(big, R, torch.tensor([[519, 0], [3, 519]], device="cuda", dtype=torch.int32), x)
    ref = x.double() @ wl.t()
    assert torch.equal(y[0, 0].double(), ref[0]) and torch.equal(y[1, 1].double(), ref[1])
    assert not bool(y[0, 1].any()) and not bool(y[1, 0].any())
