"""The operators of one verification step of drafted tokens, as measured cases.

A chunk of M tokens (the drafted ones and the last accepted one) goes through
a decoder's blocks and is then accepted or refused token by token:

  w4       y = x . W^T for weights in 4 bits with a scale and a zero point a group
  norm     the norm after a block, its gate and residual scale, and the norm
           before the next block
  softmax  rows of logits to probabilities at a temperature
  verify   drafted tokens against the target's probabilities, from given random
           numbers

`run` computes them with elementary torch operations where `own` is false, and
with the library's calls where it is true.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ------------------------------------------------------------------ cases --

def _w4(M, N, K, group, zeros, x, y, **kw):
    return dict(op="w4", M=M, N=N, K=K, group=group, zeros=zeros, x=x, y=y, **kw)


def _norm(M, D, y, dtype, post, gate, **kw):
    return dict(op="norm", M=M, D=D, y=y, dtype=dtype, post=post, gate=gate, **kw)


def _softmax(rows, V, x, per_row, **kw):
    return dict(op="softmax", rows=rows, V=V, x=x, per_row=per_row, **kw)


def _verify(B, S, V, q, ragged, **kw):
    return dict(op="verify", B=B, S=S, V=V, q=q, ragged=ragged, **kw)


def listed():
    return [
        # an output projection for one token: the smallest weights, where latency counts
        _w4(1, 2048, 2048, 128, True, "f16", "f16", name="w4 o-proj 1 token"),
        # the widest product of a layer for one token, gate and up in one
        _w4(1, 43008, 5376, 128, True, "bf16", "bf16", name="w4 gate-up 1 token"),
        # a down projection for a chunk of eight tokens: few rows, long sums
        _w4(8, 5376, 21504, 64, False, "f16", "f16", name="w4 down 8 tokens"),
        # logits of five verified tokens: the most weights of a step, in short groups
        _w4(5, 262144, 2048, 32, False, "bf16", "f32", name="w4 lm-head 5 tokens"),
        # sizes that fill no tile, and a batch of chunks
        _w4(19, 4099, 4128, 128, True, "f16", "f32", name="w4 odd 19 tokens"),
        # between two blocks for one token: latency
        _norm(1, 2048, "f32", "f16", True, "none", name="norm 1 token"),
        # a batch of verified chunks, with an odd width and a gate a channel
        _norm(77, 5381, "f16", "bf16", True, "channel", name="norm 77 tokens odd"),
        # a prefill chunk, a gate a token and channel
        _norm(4096, 4096, "bf16", "bf16", True, "token", name="norm 4096 tokens"),
        # one sequence's verified tokens
        _softmax(5, 262144, "f32", False, name="softmax 1x5"),
        # a batch of sequences with temperatures of their own, an odd vocabulary
        _softmax(384, 50257, "f16", True, name="softmax 64x6 odd"),
        # one sequence, drafted by a model
        _verify(1, 4, 262144, True, False, name="verify 1x4"),
        # a batch, some sequences with fewer drafted tokens
        _verify(48, 5, 262144, True, True, name="verify 48x5 ragged"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["w4", "w4", "norm", "softmax", "verify"])
    if op == "w4":
        M = _log(rng, 1, 32)
        K = 32 * _log(rng, 4, 672)
        N = _log(rng, 64, min(262144, 230_000_000 // K))
        return _w4(M, N, K, rng.choice([32, 64, 128]), rng.random() < 0.5, rng.choice(["f16", "bf16"]),
                   rng.choice(["f32", "f16", "bf16"]))
    if op == "norm":
        D = _log(rng, 64, 16384)
        return _norm(_log(rng, 1, 16_000_000 // D), D, rng.choice(["f32", "f16", "bf16"]),
                     rng.choice(["f16", "bf16"]), rng.random() < 0.7, rng.choice(["none", "channel", "token"]))
    if op == "softmax":
        V = _log(rng, 100, 262144)
        return _softmax(_log(rng, 1, min(2048, 19_000_000 // V)), V, rng.choice(["f32", "f16", "bf16"]),
                        rng.random() < 0.5)
    V = _log(rng, 100, 262144)
    S = rng.randint(1, 8)
    return _verify(_log(rng, 1, min(256, max(2, 75_000_000 // (V * (S + 1))))), S, V, rng.random() < 0.7,
                   rng.random() < 0.5)


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _logits(g, rows, V):
    """Logits as a language model gives them: most of a row near its middle, a
    few tokens that stand out."""
    x = _randn(g, rows, V) * 2.0
    top = torch.randint(0, V, (rows, 8), generator=g, device="cuda")
    x.scatter_add_(1, top, 6.0 + 5.0 * _rand(g, rows, 8))
    return x


def _inputs(c, seed):
    g = _gen(seed)
    if c["op"] == "w4":
        G = -(-c["K"] // c["group"])
        dt = DT[c["x"]]
        d = {"x": _randn(g, c["M"], c["K"]).to(dt),
             "codes": torch.randint(0, 16, (c["N"], c["K"]), generator=g, device="cuda", dtype=torch.uint8),
             "scales": (0.005 + 0.015 * _rand(g, c["N"], G)).to(dt), "zeros": None}
        if c["zeros"]:
            d["zeros"] = torch.randint(4, 12, (c["N"], G), generator=g, device="cuda", dtype=torch.uint8)
        return d
    if c["op"] == "norm":
        dt, M, D = DT[c["dtype"]], c["M"], c["D"]
        d = {"y": (_randn(g, M, D) * 0.7).to(DT[c["y"]]), "residual": (_randn(g, M, D) * 3.0).to(dt),
             "gamma_pre": (1.0 + 0.1 * _randn(g, D)).to(dt), "gamma_post": None, "gate": None,
             "residual_scale": 0.9, "branch_scale": 0.5}
        if c["post"]:
            d["gamma_post"] = (1.0 + 0.1 * _randn(g, D)).to(dt)
        if c["gate"] != "none":
            shape = (M, D) if c["gate"] == "token" else (D,)
            d["gate"] = torch.sigmoid(_randn(g, *shape)).to(dt)
        return d
    if c["op"] == "softmax":
        return {"logits": _logits(g, c["rows"], c["V"]).to(DT[c["x"]]),
                "temperature": 0.5 + _rand(g, c["rows"]) if c["per_row"] else 0.8}
    B, S, V = c["B"], c["S"], c["V"]
    lt = _logits(g, B * (S + 1), V)
    target = torch.softmax(lt, 1).view(B, S + 1, V)
    d = {"target": target, "draft_probs": None, "n_draft": None}
    ld = lt.view(B, S + 1, V)[:, :S] + 0.6 * _randn(g, B, S, V)
    q = torch.softmax(ld, 2)
    # drafted tokens are drawn from the draft's probabilities (the greedy one
    # where there are none)
    if c["q"]:
        d["draft_probs"] = q.contiguous()
        at = torch.log(-torch.log(_rand(g, B, S, V).clamp_(1e-7, 1 - 1e-7)))
        d["draft"] = (torch.log(q + 1e-30) - at).argmax(2).to(torch.int32)
    else:
        d["draft"] = q.argmax(2).to(torch.int32)
    if c["ragged"]:
        d["n_draft"] = torch.randint(0, S + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    d["u_accept"], d["u_sample"] = _rand(g, B, S), _rand(g, B)
    return d


def prepare(case, seed):
    s = dict(_inputs(case, seed), case=case)
    if case["op"] == "w4" and own:
        # a program keeps the weights packed
        from bit_weight_only_packed_gb300 import qmv
        p = qmv.W4Pack(case["N"], case["K"], case["group"], DT[case["x"]], case["zeros"])
        s["pack"] = p.pack_weights(s.pop("codes"), s.pop("scales"), s.pop("zeros"))
    return s


# ------------------------------------------------------------ plain forms --

def _plain_w4(s):
    c = s["case"]
    at = torch.arange(c["K"], device="cuda") // c["group"]
    z = s["zeros"].float()[:, at] if c["zeros"] else 8.0
    w = (s["codes"].float() - z) * s["scales"].float()[:, at]
    return (s["x"].float() @ w.t()).to(DT[c["y"]])


def _plain_norm(s):
    c = s["case"]
    eps, dt = 1e-6, DT[c["dtype"]]
    u = s["y"].float()
    if s["gamma_post"] is not None:
        u = u * torch.rsqrt((u * u).mean(1, keepdim=True) + eps) * s["gamma_post"].float()
    if s["gate"] is not None:
        u = u * s["gate"].float()
    h = (s["residual_scale"] * s["residual"].float() + s["branch_scale"] * u).to(dt)
    f = h.float()
    return h, (f * torch.rsqrt((f * f).mean(1, keepdim=True) + eps) * s["gamma_pre"].float()).to(dt)


def _plain_softmax(s):
    t = s["temperature"]
    x = s["logits"].float()
    e = torch.exp((x - x.amax(1, keepdim=True)) / (t[:, None] if torch.is_tensor(t) else t))
    return e / e.sum(1, keepdim=True)


def _plain_verify(s):
    p, q, draft = s["target"], s["draft_probs"], s["draft"].long()
    B, S = draft.shape
    V = p.shape[2]
    rows, at = torch.arange(B, device="cuda"), torch.arange(S + 1, device="cuda")
    n = torch.full((B,), S, device="cuda") if s["n_draft"] is None else s["n_draft"].long()
    d = draft.clamp(0, V - 1)[:, :, None]
    pd = p[:, :S].gather(2, d)[:, :, 0].double()
    qd = 1.0 if q is None else q.gather(2, d)[:, :, 0].double()
    good = (s["u_accept"].double() * qd < pd) & (at[:S] < n[:, None]) & (draft >= 0) & (draft < V)
    acc = good.long().cumprod(1).sum(1)
    last = acc.clamp(max=S - 1)
    pj = p[rows, acc]
    if q is None:
        qj = (torch.arange(V, device="cuda") == draft[rows, last][:, None]).float()
    else:
        qj = q[rows, last]
    rest = torch.relu(pj - qj)
    # weights are whole multiples of 2^-42, so that sums do not depend on their order
    unit = 2.0 ** 42
    wp, wr = (pj.clamp(0, 1).double() * unit).long(), (rest.clamp(0, 1).double() * unit).long()
    use = (acc < n) & (wr.sum(1) > 0)
    w = torch.where(use[:, None], wr, wp)
    total = w.sum(1)
    u = (s["u_sample"].double() * 2.0 ** 31).long().clamp(0, 2 ** 31 - 1)
    t = ((u * (total >> 32)) << 1) + ((u * (total & 0xffffffff)) >> 31)
    new = (w.cumsum(1) <= t[:, None]).sum(1)
    new = torch.where(total > 0, new, torch.full_like(new, -1))
    kept = torch.cat([draft, draft[:, :1]], 1)
    tokens = torch.where(at < acc[:, None], kept, torch.where(at == acc[:, None], new[:, None], -1))
    return tokens.to(torch.int32), acc.to(torch.int32)


# -------------------------------------------------------------------- run --

def _library():
    from bit_weight_only_packed_gb300 import qmv
    return qmv


def _own(s):
    q, c = _library(), s["case"]
    if c["op"] == "w4":
        return q.qmv_w4_gemv(s["pack"], s["x"], y_dtype={"f32": q.QMV_F32, "f16": q.QMV_F16, "bf16": q.QMV_BF16}[c["y"]])
    if c["op"] == "norm":
        return q.qmv_block_norm(s["y"], s["residual"], s["gamma_pre"], gamma_post=s["gamma_post"], gate=s["gate"],
                                residual_scale=s["residual_scale"], branch_scale=s["branch_scale"], eps=1e-6)
    if c["op"] == "softmax":
        return q.qmv_softmax(s["logits"], s["temperature"])
    return q.qmv_verify_draft(s["target"], s["draft_probs"], s["draft"], s["u_accept"], s["u_sample"],
                              n_draft=s["n_draft"])


PLAIN = {"w4": _plain_w4, "norm": _plain_norm, "softmax": _plain_softmax, "verify": _plain_verify}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------- work --

def work(case):
    c = case
    if c["op"] == "w4":
        M, N, K = c["M"], c["N"], c["K"]
        G = -(-K // c["group"])
        b = N * K / 2 + 2 * N * G + (N * G / 2 if c["zeros"] else 0) + 2 * M * K + SIZE[c["y"]] * M * N
        return {"bytes": b, "flops": 2.0 * M * N * K}
    if c["op"] == "norm":
        M, D = c["M"], c["D"]
        b = M * D * (SIZE[c["y"]] + 6 + (2 if c["gate"] == "token" else 0)) + 2 * D * (1 + c["post"] + (c["gate"] == "channel"))
        return {"bytes": b, "flops": M * D * (12.0 if c["post"] else 8.0)}
    if c["op"] == "softmax":
        n = c["rows"] * c["V"]
        return {"bytes": n * (SIZE[c["x"]] + 4), "flops": 5.0 * n}
    # the row of the target that the new token is drawn from, and the draft's
    # where a token was refused (nearly every sequence)
    n = c["B"] * c["V"]
    return {"bytes": n * (8 if c["q"] else 4) + c["B"] * c["S"] * 16, "flops": 4.0 * n}


# ------------------------------------------------- definitions in 64 bits --

def _exact_w4(c, d):
    N, K, group = c["N"], c["K"], c["group"]
    G = -(-K // group)
    x = torch.zeros(c["M"], G * group, dtype=torch.float64, device="cuda")
    x[:, :K] = d["x"].double()
    y = torch.zeros(c["M"], N, dtype=torch.float64, device="cuda")
    rows = max(1, (1 << 27) // (G * group))
    for n in range(0, N, rows):
        q = torch.zeros(min(rows, N - n), G * group, dtype=torch.float64, device="cuda")
        q[:, :K] = d["codes"][n:n + rows].double()
        q = q.view(-1, G, group) - (d["zeros"][n:n + rows].double()[:, :, None] if c["zeros"] else 8)
        q *= d["scales"][n:n + rows].double()[:, :, None]
        y[:, n:n + rows] = x @ q.view(q.shape[0], -1).t()
    return y


def _exact_norm(c, d):
    def rms(v, gamma):
        return v / torch.sqrt(v.pow(2).sum(1, keepdim=True) / v.shape[1] + 1e-6) * gamma.double()

    v = d["y"].double()
    v = rms(v, d["gamma_post"]) if c["post"] else v
    v = v if d["gate"] is None else v * d["gate"].double()
    h = d["residual"].double() * d["residual_scale"] + v * d["branch_scale"]
    # the second norm is defined on h as it is stored
    return h, rms(h.to(DT[c["dtype"]]).double(), d["gamma_pre"])


def _exact_softmax(c, d):
    t = d["temperature"]
    return torch.softmax(d["logits"].double() / (t.double()[:, None] if c["per_row"] else t), 1)


def exact(case, seed):
    if case["op"] == "verify":
        return None          # whole numbers
    f = {"w4": _exact_w4, "norm": _exact_norm, "softmax": _exact_softmax}[case["op"]]
    return f(case, _inputs(case, seed))
