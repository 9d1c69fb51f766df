"""The operators of a decode step around its matvecs, as measured cases.

After the fused q/k/v matvec the heads are normed and rotated; ahead of a
mixture of experts the tokens are routed, and the chosen experts' 4-bit weights
are multiplied with them; behind the lm_head the next token is drawn:

  rope     norms of query and key heads and their position rotation, in one pass
  route    experts of a token and their weights, from the router's logits
  experts  products of 4-bit expert weights with the tokens routed to them, with
           the gated activation in front or the weighted sum behind
  sample   a token a row of logits: temperature, top-k, top-p, min-p, from given
           random numbers

`run` computes them with elementary torch operations where `own` is false, and
with the library's calls where it is true.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ------------------------------------------------------------------ cases --

def _rope(M, nq, nk, D, rot, x, y, layout, norm, scaling, far, **kw):
    return dict(op="rope", M=M, nq=nq, nk=nk, D=D, rot=rot, x=x, y=y, layout=layout, norm=norm, scaling=scaling, far=far, **kw)


def _route(M, E, T, x, score, bias, groups, group_k, group_top, renorm, **kw):
    return dict(op="route", M=M, E=E, T=T, x=x, score=score, bias=bias, groups=groups, group_k=group_k,
                group_top=group_top, renorm=renorm, **kw)


def _experts(M, T, E, R, K, group, zeros, x, y, act, combine, **kw):
    return dict(op="experts", M=M, T=T, E=E, R=R, K=K, group=group, zeros=zeros, x=x, y=y, act=act, combine=combine, **kw)


def _sample(rows, V, x, per_row, top_k, top_p, min_p, **kw):
    return dict(op="sample", rows=rows, V=V, x=x, per_row=per_row, top_k=top_k, top_p=top_p, min_p=min_p, **kw)


def listed():
    return [
        # one token of a small layer, from the matvec's fp32 sums: latency
        _rope(1, 8, 1, 256, 256, "f32", "f16", "half", True, "none", 8192, name="rope 1 token"),
        # a batch of verified chunks with half of each head turned, pairs side by side, odd heads
        _rope(77, 12, 3, 72, 40, "f16", "f16", "interleaved", True, "linear", 200000, name="rope 77 tokens odd"),
        # a prefill chunk of a wide layer far into a long context
        _rope(8192, 32, 8, 256, 256, "bf16", "bf16", "half", True, "yarn", 1000000, name="rope 8192 tokens"),
        # one token, a plain router
        _route(1, 64, 8, "f32", "softmax", False, 1, 1, 1, True, name="route 1 token"),
        # a batch, experts in groups, an odd number of them
        _route(129, 156, 6, "f16", "sigmoid", True, 12, 3, 2, True, name="route 129 tokens odd"),
        # a prefill chunk over many experts, balanced by a bias
        _route(16384, 256, 8, "f32", "sigmoid", True, 8, 4, 2, True, name="route 16384 tokens"),
        # one token's gate and up products: eight experts' weights
        _experts(1, 8, 64, 2048, 2048, 128, True, "f16", "f32", "none", False, name="experts gate-up 1 token"),
        # the down products of a verified chunk, summed by the router's weights
        _experts(8, 8, 64, 2048, 1024, 128, True, "bf16", "bf16", "silu", True, name="experts down 8 tokens"),
        # a batch that reaches nearly all of many experts
        _experts(64, 8, 128, 2048, 2048, 64, False, "bf16", "bf16", "none", False, name="experts gate-up 64 tokens"),
        # one sequence at its next token
        _sample(1, 262144, "f32", False, 64, 0.95, 0.0, name="sample 1 row"),
        # a batch whose sequences have settings of their own, an odd vocabulary
        _sample(64, 50257, "f16", True, 50, 0.9, 0.05, name="sample 64 rows odd"),
        # a batch over the largest vocabulary, cut by probability alone
        _sample(128, 262144, "f32", False, 0, 0.9, 0.0, name="sample 128 rows"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "route", "experts", "experts", "sample"])
    if op == "rope":
        D = 2 * _log(rng, 16, 128)
        nk = _log(rng, 1, 8)
        nq = nk * rng.randint(1, 8)
        rot = D if rng.random() < 0.5 else 2 * rng.randint(1, D // 2)
        return _rope(_log(rng, 1, min(8192, 50_000_000 // ((nq + nk) * D))), nq, nk, D, rot, rng.choice(["f32", "f16", "bf16"]),
                     rng.choice(["f16", "bf16"]), rng.choice(["half", "interleaved"]), rng.random() < 0.7,
                     rng.choice(["none", "linear", "ntk", "yarn"]) if rot > 2 else "none", _log(rng, 100, 1_000_000))
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        per = _log(rng, max(2, 8 // groups), 512 // groups)
        group_k = rng.randint(1, groups)
        E = groups * per
        return _route(_log(rng, 1, min(16384, 4_000_000 // E)), E, rng.randint(1, min(16, group_k * per)),
                      rng.choice(["f32", "f16", "bf16"]), rng.choice(["softmax", "sigmoid"]), rng.random() < 0.5, groups,
                      group_k, rng.choice([1, 2]), rng.random() < 0.7)
    if op == "experts":
        E = _log(rng, 4, 128)
        K, R = 32 * _log(rng, 4, 128), 32 * _log(rng, 2, 128)
        while E * K * R > 500_000_000:
            E //= 2
        act = rng.choice(["none", "none", "silu", "gelu"])
        return _experts(_log(rng, 1, 64), rng.randint(1, min(8, E)), E, R, K, rng.choice([32, 64, 128]), rng.random() < 0.5,
                        rng.choice(["f16", "bf16"]), rng.choice(["f32", "f16", "bf16"] if act == "none" else ["f16", "bf16"]),
                        act, rng.random() < 0.5)
    V = _log(rng, 100, 262144)
    return _sample(_log(rng, 1, min(512, 33_000_000 // V)), V, rng.choice(["f32", "f16", "bf16"]), rng.random() < 0.5,
                   rng.choice([0, 1, 20, 100, 1000]), rng.choice([1.0, 0.95, 0.7]), rng.choice([0.0, 0.0, 0.02]))


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


# What a long context changes: positions 8 times as far as the ROPE_LENGTH that
# a model was trained on.
ROPE_BASE, ROPE_FACTOR, ROPE_LENGTH = 10000.0, 8.0, 8192


def _frequencies(rot, scaling):
    """Angle a position of each pair, and what the rotated elements are scaled by."""
    n, b, f = rot // 2, ROPE_BASE, ROPE_FACTOR
    if scaling == "ntk":
        b *= f ** (rot / (rot - 2))
    w = [b ** (-2.0 * i / rot) for i in range(n)]
    if scaling == "linear":
        return [v / f for v in w], 1.0
    if scaling != "yarn":
        return w, 1.0
    # pairs that turn more than 32 times in the old length stay, those that turn less
    # than once are stretched, between them a ramp
    at = [rot * math.log(ROPE_LENGTH / (turns * 2 * math.pi)) / (2 * math.log(b)) for turns in (32.0, 1.0)]
    lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
    ramp = [min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0) for i in range(n)]
    return [v / f * r + v * (1 - r) for v, r in zip(w, ramp)], 0.1 * math.log(f) + 1.0


def _logits(g, rows, V):
    """Logits as a language model gives them: most of a row near its middle, a
    few tokens that stand out."""
    x = _randn(g, rows, V) * 2.0
    top = torch.randint(0, V, (rows, 8), generator=g, device="cuda")
    x.scatter_add_(1, top, 6.0 + 5.0 * _rand(g, rows, 8))
    return x


def _inputs(c, seed):
    g = _gen(seed)
    if c["op"] == "rope":
        # what the q/k/v matvec leaves: query heads, key heads, value heads
        d = {"qkv": (_randn(g, c["M"], (c["nq"] + 2 * c["nk"]) * c["D"]) * 1.5).to(DT[c["x"]]),
             "positions": torch.randint(0, c["far"], (c["M"],), generator=g, device="cuda", dtype=torch.int32),
             "gamma_q": None, "gamma_k": None}
        if c["norm"]:
            d["gamma_q"], d["gamma_k"] = ((1.0 + 0.1 * _randn(g, c["D"])).to(DT[c["y"]]) for _ in range(2))
        return d
    if c["op"] == "route":
        d = {"logits": (_randn(g, c["M"], c["E"]) * 1.5).to(DT[c["x"]]), "bias": None}
        if c["bias"]:
            d["bias"] = 0.1 * _randn(g, c["E"])
        return d
    if c["op"] == "experts":
        N, K, G = c["E"] * c["R"], c["K"], -(-c["K"] // c["group"])
        dt = DT[c["x"]]
        d = {"codes": torch.randint(0, 16, (N, K), generator=g, device="cuda", dtype=torch.uint8),
             "scales": (0.005 + 0.015 * _rand(g, N, G)).to(dt), "zeros": None}
        if c["zeros"]:
            d["zeros"] = torch.randint(4, 12, (N, G), generator=g, device="cuda", dtype=torch.uint8)
        # a token's experts are distinct, and all about equally sought
        order = _rand(g, c["M"], c["E"]).argsort(1)
        d["ids"] = order[:, :c["T"]].to(torch.int32).contiguous()
        w = _rand(g, c["M"], c["T"]) + 0.1
        d["weights"] = w / w.sum(1, keepdim=True) if c["combine"] else None
        shape = (c["M"], K) if c["act"] == "none" else (c["M"], c["T"], 2 * K)
        d["x"] = _randn(g, *shape).to(dt)
        return d
    rows = c["rows"]
    d = {"logits": _logits(g, rows, c["V"]).to(DT[c["x"]]), "u": _rand(g, rows), "temperature": 0.8, "top_k": c["top_k"],
         "top_p": c["top_p"], "min_p": c["min_p"]}
    if c["per_row"]:
        d["temperature"] = 0.5 + _rand(g, rows)
        d["top_p"] = (c["top_p"] - 0.1 * _rand(g, rows))
        d["min_p"] = c["min_p"] * _rand(g, rows)
        if c["top_k"]:
            d["top_k"] = torch.randint(1, 2 * c["top_k"], (rows,), generator=g, device="cuda", dtype=torch.int32)
    return d


def prepare(case, seed):
    c = case
    s = dict(_inputs(c, seed), case=c)
    if c["op"] == "rope":
        # a program keeps the frequencies of its positions
        if own:
            q = _library()
            s["rope"] = q.Rope(c["rot"], base=ROPE_BASE, layout=getattr(q, "QMV_ROPE_" + c["layout"].upper()),
                               scaling=getattr(q, "QMV_SCALE_" + c["scaling"].upper()), factor=ROPE_FACTOR,
                               original_length=ROPE_LENGTH)
        else:
            w, s["amplitude"] = _frequencies(c["rot"], c["scaling"])
            s["inv_freq"] = torch.tensor(w, dtype=torch.float64, device="cuda")
    if c["op"] == "experts" and own:
        # and its weights packed, with scratch for its largest batch
        q = _library()
        p = q.W4Pack(c["E"] * c["R"], c["K"], c["group"], DT[c["x"]], c["zeros"])
        s["pack"] = p.pack_weights(s.pop("codes"), s.pop("scales"), s.pop("zeros"))
        s["workspace"] = q.qmv_w4_experts_workspace(p, c["R"], c["M"], c["T"])
    return s


# ------------------------------------------------------------ plain forms --

def _plain_rope(s):
    c = s["case"]
    M, nq, nk, D, rot = c["M"], c["nq"], c["nk"], c["D"], c["rot"]
    # angles of far positions need 64 bits
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    cos = (angle.cos() * s["amplitude"]).float()[:, None]
    sin = (angle.sin() * s["amplitude"]).float()[:, None]
    out = []
    for at, n, gamma in ((0, nq, s["gamma_q"]), (nq, nk, s["gamma_k"])):
        v = s["qkv"][:, at * D:(at + n) * D].float().view(M, n, D)
        if gamma is not None:
            v = v * torch.rsqrt((v * v).mean(2, keepdim=True) + 1e-6) * gamma.float()
        if c["layout"] == "half":
            a, b = v[..., :rot // 2], v[..., rot // 2:rot]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], 2)
        else:
            a, b = v[..., 0:rot:2], v[..., 1:rot:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], 3).view(M, n, rot)
        out.append(torch.cat([turned, v[..., rot:]], 2).to(DT[c["y"]]))
    return out


def _plain_route(s):
    c = s["case"]
    M, E, T = c["M"], c["E"], c["T"]
    # an expert's place hangs on differences, so scores are compared in 64 bits
    x = s["logits"].double()
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-x))
    else:
        e = torch.exp(x - x.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    rank = score if s["bias"] is None else score + s["bias"].double()
    if c["groups"] > 1:
        parts = rank.view(M, c["groups"], -1)
        best = parts.sort(dim=2, descending=True, stable=True).values[..., :c["group_top"]].sum(2)
        chosen = best.sort(dim=1, descending=True, stable=True).indices[:, :c["group_k"]]
        keep = torch.zeros(M, c["groups"], dtype=torch.bool, device="cuda").scatter_(1, chosen, True)
        rank = torch.where(keep[:, :, None], parts, -math.inf).view(M, E)
    ids = rank.sort(dim=1, descending=True, stable=True).indices[:, :T]
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return ids.to(torch.int32), (w * 2.5).float()


def _act(kind, x):
    """The gated activation of [.., gate | up]."""
    a, b = x.chunk(2, -1)
    if kind == "silu":
        return a / (1.0 + torch.exp(-a)) * b
    t = 0.7978845608028654 * (a + 0.044715 * a * a * a)
    return a / (1.0 + torch.exp(-2.0 * t)) * b            # (1 + tanh t) / 2 = 1 / (1 + exp(-2 t))


def _plain_experts(s):
    c = s["case"]
    M, T, R, K = c["M"], c["T"], c["R"], c["K"]
    at = torch.arange(K, device="cuda") // c["group"]
    x = s["x"].float()
    if c["act"] != "none":
        x = _act(c["act"], x).to(DT[c["x"]]).float()      # the product takes it as it is stored
    x = x.view(M, -1, K).expand(M, T, K).reshape(M * T, K)
    ids = s["ids"].view(-1).long()
    y = torch.zeros(M * T, R, device="cuda")
    for e in range(c["E"]):
        rows = slice(e * R, (e + 1) * R)
        z = s["zeros"][rows].float()[:, at] if c["zeros"] else 8.0
        w = (s["codes"][rows].float() - z) * s["scales"][rows].float()[:, at]
        y += (x * (ids == e)[:, None]) @ w.t()
    y = y.view(M, T, R)
    if c["combine"]:
        y = (y * s["weights"][:, :, None]).sum(1)
    return y.to(DT[c["y"]])


# 2^f for |f| <= 1/2, interpolated at Chebyshev nodes: part of the definition
EXP2 = [1.0, 0.6931471824645996, 0.2402234971523285, 0.055503811687231064, 0.00966636836528778, 0.0013381302123889327]


def _weights(x, top, t):
    """exp((x - top) / t) in whole units of 2^-42 of the largest, so that sums do not
    depend on their order: every step is one fp32 operation."""
    rate = torch.full_like(t, 1.4426950408889634) / t.clamp(min=2.0 ** -100)
    z = torch.where(x == top, 0.0, (top - x) * rate).clamp(max=64.0)
    n = z.round()
    f = (n - z).double()
    p = torch.full_like(z, EXP2[-1])
    for k in EXP2[-2::-1]:
        p = (p.double() * f + k).float()                  # a fused multiply-add
    return torch.where(x > -math.inf, torch.floor(p.double() * torch.exp2(42.0 - n.double())), 0.0).long()


def _share(total, u):
    """floor(total * u) for u in whole units of 2^-31."""
    u = (u.double() * 2.0 ** 31).long().clamp(0, 2 ** 31)
    return ((u * (total >> 32)) << 1) + ((u * (total & 0xffffffff)) >> 31)


def _plain_sample(s):
    x = s["logits"].float()
    rows, V = x.shape

    def setting(v):
        return v if torch.is_tensor(v) else torch.full((rows,), v, device="cuda")

    t, k, top_p, min_p = (setting(s[n]) for n in ("temperature", "top_k", "top_p", "min_p"))
    top = x.amax(1, keepdim=True)
    w = _weights(x, top, t[:, None])
    # every cut keeps the first so many of an order: the largest first, equal ones by id
    order = x.sort(dim=1, descending=True, stable=True).indices
    ws = w.gather(1, order)
    k = torch.where(k > 0, k, V)
    ws = torch.where(torch.arange(V, device="cuda") < k[:, None], ws, 0)
    before = ws.cumsum(1) - ws
    need = torch.where(top_p < 1.0, _share(ws.sum(1), top_p), 2 ** 62)
    first = torch.arange(V, device="cuda") == 0
    ws = torch.where((before < need[:, None]) | first, ws, 0)
    ws = torch.where(ws >= (min_p.double() * 2.0 ** 42).long()[:, None], ws, 0)
    w = torch.zeros_like(w).scatter_(1, order, ws)
    run = w.cumsum(1)
    t = _share(run[:, -1], s["u"])
    return (run <= t[:, None]).sum(1).to(torch.int32)


# -------------------------------------------------------------------- run --

def _library():
    from bit_weight_only_packed_gb300 import qmv
    return qmv


def _own(s):
    q, c = _library(), s["case"]
    code = {"f32": q.QMV_F32, "f16": q.QMV_F16, "bf16": q.QMV_BF16}
    if c["op"] == "rope":
        return q.qmv_qk_norm_rope(s["qkv"], c["nq"], c["nk"], c["D"], s["rope"], s["positions"], gamma_q=s["gamma_q"],
                                  gamma_k=s["gamma_k"], eps=1e-6, y_dtype=code[c["y"]])
    if c["op"] == "route":
        return q.qmv_route(s["logits"], c["T"], score=getattr(q, "QMV_SCORE_" + c["score"].upper()), bias=s["bias"],
                           groups=c["groups"], group_k=c["group_k"], group_top=c["group_top"], renormalise=c["renorm"],
                           scale=2.5)
    if c["op"] == "experts":
        return q.qmv_w4_experts(s["pack"], c["R"], s["ids"], s["x"], weights=s["weights"],
                                act=getattr(q, "QMV_ACT_" + c["act"].upper()), y_dtype=code[c["y"]], workspace=s["workspace"])
    return q.qmv_sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])


PLAIN = {"rope": _plain_rope, "route": _plain_route, "experts": _plain_experts, "sample": _plain_sample}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------- work --

def work(case):
    c = case
    if c["op"] == "rope":
        n = c["M"] * (c["nq"] + c["nk"]) * c["D"]
        return {"bytes": n * (SIZE[c["x"]] + SIZE[c["y"]]) + 4 * c["M"] + 4 * c["rot"], "flops": n * 8.0}
    if c["op"] == "route":
        return {"bytes": c["M"] * (c["E"] * SIZE[c["x"]] + c["T"] * 8), "flops": c["M"] * c["E"] * 8.0}
    if c["op"] == "experts":
        M, T, E, R, K = c["M"], c["T"], c["E"], c["R"], c["K"]
        # the weights of the experts that a batch is expected to reach
        reached = E * (1.0 - (1.0 - T / E) ** M)
        per = R * (K / 2 + -(-K // c["group"]) * (2.5 if c["zeros"] else 2.0))
        x = M * K * 2 if c["act"] == "none" else M * T * K * 4
        y = M * R * (1 if c["combine"] else T) * SIZE[c["y"]]
        return {"bytes": reached * per + x + y + M * T * 8, "flops": 2.0 * M * T * R * K}
    n = c["rows"] * c["V"]
    return {"bytes": n * SIZE[c["x"]] + c["rows"] * 8, "flops": 20.0 * n}


# ------------------------------------------------- definitions in 64 bits --

def _exact_rope(c, d):
    D, rot = c["D"], c["rot"]
    w, amplitude = _frequencies(rot, c["scaling"])
    angle = d["positions"].double()[:, None, None] * torch.tensor(w, dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.full_like(angle, amplitude), angle)
    heads = d["qkv"].double().view(c["M"], -1, D)
    out = []
    for v, gamma in ((heads[:, :c["nq"]], d["gamma_q"]), (heads[:, c["nq"]:c["nq"] + c["nk"]], d["gamma_k"])):
        if gamma is not None:
            v = v / torch.sqrt(v.pow(2).sum(2, keepdim=True) / D + 1e-6) * gamma.double()
        y = v.clone()
        first = slice(0, rot // 2) if c["layout"] == "half" else slice(0, rot, 2)
        second = slice(rot // 2, rot) if c["layout"] == "half" else slice(1, rot, 2)
        z = torch.complex(v[..., first].contiguous(), v[..., second].contiguous()) * turn
        y[..., first], y[..., second] = z.real, z.imag
        out.append(y)
    return out


def _exact_route(c, d):
    x = d["logits"].double()
    p = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, 1)
    key = p.clone() if d["bias"] is None else p + d["bias"].double()
    if c["groups"] > 1:
        g = key.unflatten(1, (c["groups"], -1))
        worth = g.topk(c["group_top"], 2).values.sum(2)
        out = worth.argsort(dim=1, descending=True, stable=True)[:, c["group_k"]:]
        g.scatter_(1, out[:, :, None].expand(-1, -1, g.shape[2]), -math.inf)
    w = p.gather(1, key.argsort(dim=1, descending=True, stable=True)[:, :c["T"]])
    return None, 2.5 * (w / w.sum(1, keepdim=True) if c["renorm"] else w)


def _exact_experts(c, d):
    M, T, R, K, G = c["M"], c["T"], c["R"], c["K"], -(-c["K"] // c["group"])
    x = d["x"].double()
    if c["act"] != "none":
        a, b = x[..., :K], x[..., K:]
        if c["act"] == "silu":
            x = torch.nn.functional.silu(a) * b
        else:
            x = 0.5 * a * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (a + 0.044715 * a.pow(3)))) * b
        x = x.to(DT[c["x"]]).double()
    else:
        x = x[:, None, :].expand(M, T, K)
    y = torch.zeros(M, T, R, dtype=torch.float64, device="cuda")
    for e in d["ids"].unique().tolist():
        m, j = (d["ids"] == e).nonzero(as_tuple=True)
        q = torch.zeros(R, G * c["group"], dtype=torch.float64, device="cuda")
        q[:, :K] = d["codes"][e * R:(e + 1) * R].double()
        q = q.view(R, G, -1) - (d["zeros"][e * R:(e + 1) * R].double()[:, :, None] if c["zeros"] else 8)
        q = (q * d["scales"][e * R:(e + 1) * R].double()[:, :, None]).view(R, -1)[:, :K]
        y[m, j] = x[m, j] @ q.t()
    return torch.einsum("mtr,mt->mr", y, d["weights"].double()) if c["combine"] else y


def exact(case, seed):
    if case["op"] == "sample":
        return None          # whole numbers
    f = {"rope": _exact_rope, "route": _exact_route, "experts": _exact_experts}[case["op"]]
    return f(case, _inputs(case, seed))
