"""Edges of the decode-step operators that their other tests leave out, each against 64 bits or
the definition in the header."""
import math

import pytest
import torch

from gpu_util import GuardBuf, qmv
from test_gpu_step import BF16, EPS, F16, F32, TINY, code, gen, make_w4
from test_gpu_token import act_ref, check_route, distinct, randn, route_ref

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------- route --

def check_shares(x, T, score, bias=None, renorm=True, scale=1.0):
    """check_route without its smallest sum of 1e-300: weights over their sum in 64 bits, 0 where that is 0."""
    q = qmv()
    ids, w = q.qmv_route(x, T, score=score, bias=bias, renormalise=renorm, scale=scale)
    ref, _ = route_ref(x, T, score, bias, 1, 1, 1, renorm, scale)
    assert torch.equal(ids, ref)
    v = x.double()
    s = 1 / (1 + torch.exp(-v)) if score else torch.softmax(v, 1)
    rw = s.gather(1, ref.long())
    if renorm:
        total = rw.sum(1, keepdim=True)
        rw = torch.where(total > 0, rw / total, 0.0)
    tol = rw * scale * 2.0 ** -20 + 2.0 ** -126 * scale
    assert bool(((w.double() - rw * scale).abs() <= tol).all()), float(((w.double() - rw * scale).abs() / tol).max())


@pytest.mark.parametrize("T", [1, 8, 40])
@pytest.mark.parametrize("scale", [1.0, 2.5])
@pytest.mark.parametrize("level", [-5.0, -17.0, -40.0, -87.0, -89.0, -100.0, -104.0, -150.0, -700.0, -800.0])
def test_route_weights_of_small_scores(level, scale, T):
    # scores near or below the smallest fp32 number: their shares of their sum are as large as any
    E = 64
    x = level - 3 * torch.rand(20, E, generator=gen(T), device="cuda")
    check_shares(x, T, 1, None, True, scale)
    check_shares(x, T, 1, None, False, scale)
    # the same of a softmax, where the bias takes experts far below the largest: every row has one logit of 0
    y = torch.cat((torch.zeros(20, 1, device="cuda"), x), 1)
    bias = torch.ones(E + 1, device="cuda") + 0.1 * torch.rand(E + 1, generator=gen(9), device="cuda")
    bias[0] = -5.0
    check_shares(y, T, 0, bias, True, scale)
    check_shares(y, T, 1, bias, True, scale)
    # and small ones beside one that is not
    bias[0] = 5.0
    check_shares(y, T, 1, bias, True, scale)


@pytest.mark.parametrize("level", [-12.2, -14.9, -16.4])
@pytest.mark.parametrize("score", [0, 1])
def test_route_small_weights_beside_a_small_sum(level, score):
    # shares that are numbers, of scores that are not quite: e^-80 and less of a sum of about 2^-20 or 2^-24
    x = level - 80 - 8 * torch.rand(400, 28, generator=gen(3), device="cuda")
    x[:, 5] = level - 0.1 * torch.rand(400, generator=gen(4), device="cuda")
    x[:, 23:] = -0.3 * torch.rand(400, 5, generator=gen(5), device="cuda")
    bias = torch.ones(28, device="cuda") + 0.1 * torch.rand(28, generator=gen(9), device="cuda")
    bias[23:] = -5.0
    for scale in (1.0, 1e-3):
        check_shares(x, 20, score, bias, True, scale)


@pytest.mark.parametrize("T", [8, 40])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_weights_far_below_the_largest(renorm, T):
    # the distance to the largest logit has to be known to 2^-21, which its fp32 difference does not say beyond 8
    E = 41
    x = -16 - 60 * torch.rand(300, E, generator=gen(T), device="cuda")
    x[:, 7] = torch.rand(300, generator=gen(1), device="cuda") + 0.3
    check_shares(x, T, 0, None, renorm)
    bias = torch.zeros(E, device="cuda")
    bias[7] = -5.0
    bias[20:] = 1.0
    check_shares(x, min(T, 20), 0, bias, renorm)
    x[:, 7] = -20 - torch.rand(300, generator=gen(2), device="cuda")
    check_shares(x, T, 1, None, renorm)


@pytest.mark.parametrize("per", [4, 8, 5])
@pytest.mark.parametrize("score", [0, 1])
def test_route_groups_with_fewer_than_two_experts(score, per):
    # such a group counts as -inf, whatever its only expert's rank is
    q = qmv()
    groups, M = 4, 6
    E = groups * per
    x = randn(per, M, E)
    x[:, 1:per] = -math.inf                     # the first group has its first expert alone
    bias = torch.zeros(E, device="cuda")
    bias[0] = math.inf
    for group_k in (1, 2, 3):
        ids, w = q.qmv_route(x, 3, score=score, bias=bias, groups=groups, group_k=group_k, group_top=2)
        rest, rw = q.qmv_route(x[:, per:].contiguous(), 3, score=score, bias=bias[per:].contiguous(), groups=3, group_k=group_k, group_top=2)
        assert torch.equal(ids, rest + per), (ids, rest)
    ids, _ = q.qmv_route(x, 3, score=score, bias=bias, groups=groups, group_k=4, group_top=2)
    assert bool((ids[:, 0] == 0).all())         # where all groups stay it comes first


@pytest.mark.parametrize("dt", [F32, F16, BF16])
def test_route_scores_that_64_bits_cannot_tell_apart(dt):
    q = qmv()
    # sigmoid scores of 1, softmax scores of 0, in 64 bits: without a bias the logit decides, with a bias of 0 the index
    x = torch.tensor([[41.0, 43.0, 40.0, 42.0, -3.0, 44.0, 40.0, 43.0]], device="cuda").to(dt)
    zero = torch.zeros(8, device="cuda")
    assert q.qmv_route(x, 4, score=1)[0].tolist() == [[5, 1, 7, 3]]
    assert q.qmv_route(x, 4, score=1, bias=zero)[0].tolist() == [[0, 1, 2, 3]]
    y = torch.tensor([[2.0, -1.0, 3.0, 900.0, 4.0, 1.0, 5.0, 0.0]], device="cuda").to(dt)
    assert q.qmv_route(y, 4, score=0)[0].tolist() == [[3, 6, 4, 2]]
    assert q.qmv_route(y, 4, score=0, bias=zero)[0].tolist() == [[3, 0, 1, 2]]
    # groups of two go by their scores' sum, where the first of those that are equal stays; of one by the logit
    for bias, first in ((None, 1), (zero, 0)):
        assert q.qmv_route(x, 2, score=1, bias=bias, groups=4, group_k=1, group_top=2)[0].tolist() == [[first, 1 - first]]
    assert q.qmv_route(x, 2, score=1, groups=4, group_k=1, group_top=1)[0].tolist() == [[5, 4]]
    assert q.qmv_route(x, 2, score=1, bias=zero, groups=4, group_k=1, group_top=1)[0].tolist() == [[0, 1]]


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("E,T", [(8, 1), (30, 3), (64, 1), (64, 8), (300, 5), (300, 31), (1000, 16), (64, 40), (1000, 33)])
def test_route_equal_experts_hide_no_larger_one(E, T, score):
    # a few logits many times over, and a bias beside which fp32 cannot tell them apart: equal ones fill
    # the last places and the next, behind which one that is larger in 64 bits may follow
    step = 2.0 ** -14 if score else 2.0 ** -8
    x = torch.randint(0, 4, (400, E), generator=gen(E + T), device="cuda").float() * step
    check_route(x, T, score, torch.full((E,), 1024.0, device="cuda"))
    few = torch.full((400, E), -30.0, device="cuda")
    few[:, :: max(E // 8, 1)] = x[:, :: max(E // 8, 1)]
    check_route(few, min(T, 7), score, torch.full((E,), 1024.0, device="cuda"))


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("groups,per,group_k", [(4, 2, 1), (8, 4, 3), (8, 8, 1), (5, 3, 2), (32, 8, 12)])
def test_route_equal_groups_hide_no_larger_one(groups, per, group_k, score):
    # groups of the same two logits, and some whose sum of scores is larger by less than fp32 can tell
    g = gen(groups + per)
    x = torch.full((400, groups, per), -4.0, device="cuda")
    x[:, :, 0], x[:, :, 1] = 3 + torch.rand(400, 1, generator=g, device="cuda"), 2 + torch.rand(400, 1, generator=g, device="cuda")
    x[:, :, 1] += 2.0 ** -22 * torch.randint(0, 2, (400, groups), generator=g, device="cuda")
    order = torch.rand(400, groups, per, generator=g, device="cuda").argsort(2)
    check_route(x.gather(2, order).view(400, -1), 2, score, None, groups, group_k, 2)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("groups,per,group_k,group_top", [(1, 64, 1, 1), (8, 8, 1, 1), (8, 8, 3, 2), (32, 2, 5, 2), (4, 250, 2, 1), (5, 3, 2, 2),
                                                            (3, 1, 1, 1), (8, 1, 2, 1), (6, 4, 2, 1), (4, 4, 1, 2)])
def test_route_biases_of_any_size(groups, per, group_k, group_top, score):
    # infinite ones, and such whose sum of two is infinite in fp32 and not in 64 bits
    E = groups * per
    x = randn(E, 50, E)
    for seed, some in enumerate((0.03, 0.3, 0.9)):
        for sizes in ([math.inf], [3e38], [-3e38], [3e38, -3e38, 2e38], [math.inf, 3e38, -2e38], [1e30, -1e30]):
            g = gen(seed)
            bias = 0.1 * torch.randn(E, generator=g, device="cuda")
            at = torch.rand(E, generator=g, device="cuda") < some
            which = torch.randint(0, len(sizes), (E,), generator=g, device="cuda")
            bias = torch.where(at, torch.tensor(sizes, device="cuda")[which], bias)
            check_route(x, min(6, group_k * per), score, bias, groups, group_k, group_top)


@pytest.mark.parametrize("groups,group_k,group_top", [(1, 1, 1), (4, 2, 2)])
@pytest.mark.parametrize("T", [4, 12, 33])
def test_route_scores_near_the_smallest_numbers(T, groups, group_k, group_top):
    # sigmoid scores from e^-690 to e^-744, which a bias of 0 leaves as they are
    q = qmv()
    E = 128
    x = -690 - torch.rand(60, E, generator=gen(T), device="cuda").mul(27).round() * 2
    bias = torch.zeros(E, device="cuda")
    ids, _ = q.qmv_route(x, T, score=1, bias=bias, groups=groups, group_k=group_k, group_top=group_top)
    assert torch.equal(ids, route_ref(x, T, 1, bias, groups, group_k, group_top, False, 1.0)[0])


# --------------------------------------------------------------- experts --

def one_to_one(dt):
    """A pack whose product with x is x: 32 rows of 32, code 9 on the diagonal and 8, which is zero, elsewhere."""
    codes = torch.full((32, 32), 8, device="cuda", dtype=torch.uint8)
    codes.fill_diagonal_(9)
    return qmv().W4Pack(32, 32, 32, dt, False).pack_weights(codes, torch.ones(32, 1, device="cuda", dtype=dt))


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("act", [1, 2])
@pytest.mark.parametrize("M", [16, 700])
def test_experts_gates_far_below_zero(M, act, dt):
    # the activation there is a small number, and as many bits of it are right as of any other
    q = qmv()
    g = torch.linspace(-95.0 if act == 1 else -10.0, 3.0, M, device="cuda").to(dt)
    x = torch.cat((g[:, None].expand(M, 32), torch.ones(M, 32, device="cuda", dtype=dt)), 1).contiguous()
    y = q.qmv_w4_experts(one_to_one(dt), 32, torch.zeros(M, 1, device="cuda", dtype=torch.int32), x[:, None], act=act)[:, 0].double()
    v = act_ref(x, act)
    if act == 2:                                # (1 + tanh t) / 2 = 1 / (1 + exp(-2 t)), without its cancellation
        a = x[:, :32].double()
        v = a / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)))
    # The exponent t is formed by up to five roundings: t 2^-21 of the exponential; that itself, a sum, a product,
    # a quotient: 2^-21 in all.  An exponential below 2^-126 is a multiple of 2^-149, of which g are taken.
    a = x[:, :32].double().abs()
    t = a if act == 1 else 2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)
    near = v.abs() * (t * 2.0 ** -21 + 2.0 ** -21) + a * 2.0 ** -149
    tol = near + (v.abs() + near) * EPS[dt] + TINY[dt]
    err = (y - v).abs()
    assert bool((err <= tol).all()), (float((err / tol).max()), x[(err / tol).max(1).values.argmax(), 0].item())


@pytest.mark.parametrize("dt", [F16, BF16])
def test_experts_ids_and_weights_written_again_in_place(dt):
    # a decode loop keeps its buffers: each step's ids and weights lie where the last one's lay
    q = qmv()
    M, E, T, R, K, steps = 4, 32, 4, 64, 256, 150
    p, _, _ = make_w4(E * R, K, 64, True, dt, 6)
    x = randn(1, M, K).to(dt)
    logits = randn(2, steps, M, E)
    ids, w = torch.empty(M, T, device="cuda", dtype=torch.int32), torch.empty(M, T, device="cuda")
    ws = q.qmv_w4_experts_workspace(p, R, M, T)
    torch.cuda.synchronize()
    outs = []
    for i in range(steps):
        q.qmv_route(logits[i], T, ids=ids, weights=w)
        outs.append((q.qmv_w4_experts(p, R, ids, x, weights=w, workspace=ws), q.qmv_w4_experts(p, R, ids, x, workspace=ws)))
    torch.cuda.synchronize()
    for i in range(steps):
        a, b = q.qmv_route(logits[i], T)
        torch.cuda.synchronize()
        assert torch.equal(outs[i][0], q.qmv_w4_experts(p, R, a, x, weights=b)), i
        assert torch.equal(outs[i][1], q.qmv_w4_experts(p, R, a, x)), i


@pytest.mark.parametrize("xdt", [F16, BF16])
@pytest.mark.parametrize("M,T,weighted,per_pair,act", [
    (3, 2, False, False, 0), (3, 2, True, False, 0), (40, 4, True, True, 1), (40, 4, False, False, 0), (40, 4, False, False, 2), (200, 4, True, False, 0),
])
def test_experts_scratch_of_its_form_is_enough(M, T, weighted, per_pair, act, xdt):
    # the form's own bytes, any contents, nothing written outside; the same bits as with a workspace for every form
    q = qmv()
    E, R, K = 12, 64, 320
    p, _, _ = make_w4(E * R, K, 32, True, xdt, 3)
    ids = distinct(M, T, E, 2)
    width = K * (2 if act else 1)
    x = randn(1, *((M, T, width) if per_pair else (M, width))).to(xdt)
    w = torch.rand(M, T, generator=gen(5), device="cuda") if weighted else None
    ref = q.qmv_w4_experts(p, R, ids, x, weights=w, act=act, workspace=q.qmv_w4_experts_workspace(p, R, M, T))
    n = q.lib().qmv_w4_experts_form_bytes(p.handle, R, M, T, int(weighted), x.data_ptr(), width, int(per_pair), code(xdt), act)
    st = torch.cuda.current_stream().cuda_stream
    for fill in (0x00, 0x5A, 0xFF):
        ws = GuardBuf(n, fill=fill) if n else None
        y = torch.full_like(ref, 7.0)
        rc = q.lib().qmv_w4_experts_form(p.handle, R, M, T, ids.data_ptr(), w.data_ptr() if weighted else None, x.data_ptr(), width,
                                         int(per_pair), code(xdt), act, y.data_ptr(), R, q.QMV_F32,
                                         ws.view(torch.uint8, (n,)).data_ptr() if n else None, n, st)
        torch.cuda.synchronize()
        assert rc == 0 and torch.equal(y, ref)
        if n:
            ws.check("workspace")
    assert torch.equal(q.qmv_w4_experts(p, R, ids, x, weights=w, act=act), ref)


@pytest.mark.parametrize("form", ["cpp", "python"])
def test_experts_take_no_more_memory_than_their_form(form, monkeypatch):
    q = qmv()
    if form == "python":
        monkeypatch.setattr(q, "_host", q._NoHost())
    M, T, E, R, K = 1024, 8, 16, 1024, 512
    p, _, _ = make_w4(E * R, K, 128, False, F16, 3)
    ids = distinct(M, T, E, 2)
    w = torch.rand(M, T, generator=gen(5), device="cuda")
    # rows of y, and what the call may take beside them: the pairs in order, rows of x, products
    order = 256 + 20 * M * T
    for dt, weights, most in ((F16, None, order), (BF16, None, order + M * (2 * K + 4)), (F16, w, order + M * T * R * 4)):
        x = randn(1, M, K).to(dt)
        torch.cuda.synchronize()
        # what was asked for: a block that is handed out may be up to 1 MB larger, since less is not split off
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_stats()["requested_bytes.all.current"]
        y = q.qmv_w4_experts(p, R, ids, x, weights=weights)
        taken = torch.cuda.memory_stats()["requested_bytes.all.peak"] - before - y.numel() * 4
        assert taken <= most + 1280, (dt, taken, most)         # five regions, each rounded up to 256 bytes
        del y, x


@pytest.mark.parametrize("M,T", [(3, 2), (100, 2)])
def test_experts_of_the_largest_x(M, T):
    # bf16 rows from 2^121 on, whose products are numbers again
    q = qmv()
    E, R, K, group = 4, 64, 512, 64
    p, _, w = make_w4(E * R, K, group, True, BF16, 5)
    ids = distinct(M, T, E, 2)
    x = (randn(3, M, K) * 2.0 ** torch.linspace(115, 125, M, device="cuda")[:, None]).to(BF16)
    y = q.qmv_w4_experts(p, R, ids, x)
    u, wr = x.double(), w.view(E, R, K)
    ref, A = torch.einsum("mk,erk->mer", u, wr), torch.einsum("mk,erk->mer", u.abs(), wr.abs())
    pick = ids.long()[:, :, None].expand(M, T, R)
    # the products' fp32 sums, as for x of any size (test_experts_general)
    tol = (A.gather(1, pick) + u.abs().sum(1)[:, None, None] * 30 * 0.02) * (17 * 8 + K // group + 32) * 2.0 ** -23
    assert float((ref.abs().gather(1, pick) + tol).max()) < 3.4e38      # numbers of fp32, to the last bit of what they may be off
    assert bool(((y.double() - ref.gather(1, pick)).abs() <= tol).all()), y[~torch.isfinite(y)].numel()
