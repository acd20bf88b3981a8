"""The operators that surround the intra-chunk step, as a user's program calls them, with a
plain form of each in elementary torch operations and a 64-bit definition to compare with.

Ops (the case's "op"):
  train       the gated delta-rule recurrence over whole sequences, forward and backward
  prefill     the same recurrence forward only, from a given state, with the final state
  step        its single-token form: one token for each of N requests, states updated in place
  norm_train  layer norm forward and backward with the weight's and bias's gradients
  norm        layer norm forward alone
"""

import torch

own = False

K = 128  # channels of q and k, and of v
_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------- cases
def _rec(name, op, T, H, HV=0, B=1, lens="", dtype="bf16", lo=-0.5):
    c = {"op": op, "B": B, "T": T, "H": H, "HV": HV or H, "lens": lens, "dtype": dtype, "lo": lo}
    return {"name": name, **c} if name else c


def _norm(name, op, rows, width, dtype="bf16"):
    c = {"op": op, "rows": rows, "width": width, "dtype": dtype}
    return {"name": name, **c} if name else c


def listed():
    return [
        # a small model's training step, far too few heads to fill the card
        _rec("train_small", "train", 1024, 4, B=2),
        # the library's headline workload: one layer of a training step
        _rec("train_headline", "train", 4096, 16, B=8),
        # documents of very different lengths packed into one row, value heads in groups of 2,
        # gates that forget within a few tokens
        _rec("train_packed", "train", 9467, 4, 8, lens="1,17,640,63,129,4096,65,2500,1956",
             dtype="fp16", lo=-8.0),
        # one very long prompt
        _rec("prefill_long", "prefill", 32768, 32, lo=-1.0),
        # a short prompt that continues a conversation
        _rec("prefill_short", "prefill", 37, 16),
        # a serving batch's prompts, packed, grouped value heads
        _rec("prefill_packed", "prefill", 7011, 8, 16,
             lens="5,1031,64,1,777,2048,333,128,15,2609", dtype="fp16"),
        # one user's decoding
        {"name": "step_one", "op": "step", "N": 1, "H": 16, "HV": 16, "dtype": "bf16", "lo": -0.5},
        # decoding for a full serving batch
        {"name": "step_batch", "op": "step", "N": 256, "H": 16, "HV": 32, "dtype": "bf16",
         "lo": -0.5},
        # the norm in front of the headline layer: 16 heads of 128
        _norm("norm_train_hidden", "norm_train", 32768, 2048),
        # the norm of each head's output of the headline layer
        _norm("norm_train_heads", "norm_train", 524288, 128),
        # an odd width, rows that start at no round address
        _norm("norm_train_odd", "norm_train", 2021, 1111, "fp16"),
        # the norm in front of one decoded token of four requests
        _norm("norm_token", "norm", 4, 2048),
    ]


def _log(rng, lo, hi, times=1):
    n = times * max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))
    return n if n != 24 * K else n + times


def draw(rng):
    op = rng.choice(["train", "train", "prefill", "step", "norm_train", "norm_train", "norm"])
    dtype = rng.choice(["bf16", "fp16"])
    if op in ("norm", "norm_train"):
        width = rng.choice([K, _log(rng, 16, 16384), _log(rng, 1, 64, K)])
        rows = _log(rng, 1, min(524288, (1 << 26) // width))
        return _norm("", op, rows, width, rng.choice([dtype, "fp32"]))
    H = _log(rng, 1, 16)
    HV = H * rng.choice([1, 1, 2, 4])
    lo = rng.choice([-0.1, -0.5, -1.0, -8.0])
    if op == "step":
        return {"op": op, "N": _log(rng, 1, 8192 // HV), "H": H, "HV": HV, "dtype": dtype, "lo": lo}
    most = 262144 if op == "train" else 524288  # token-heads
    if rng.random() < 0.4:
        n = rng.randint(1, 9)
        lens = [_log(rng, 1, max(1, most // HV // n // 2)) for _ in range(n)]
        return _rec("", op, sum(lens), H, HV, 1, ",".join(map(str, lens)), dtype, lo)
    T = _log(rng, 1, 8192)
    T = min(T, most // HV)
    return _rec("", op, T, H, HV, _log(rng, 1, max(1, min(16, most // HV // T))), "", dtype, lo)


# ---------------------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dt = _DT[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, device=dev, generator=gen)

    def uniform(*shape):
        return torch.rand(*shape, device=dev, generator=gen)

    s = {"op": case["op"]}
    if case["op"] in ("norm", "norm_train"):
        rows, width = case["rows"], case["width"]
        # activations carry a mean and a few large channels
        s["x"] = (normal(rows, width) * (1 + 3 * uniform(width)) + 0.5 * normal(width)).to(dt)
        s["weight"] = (1 + 0.2 * normal(width)).to(dt)
        s["bias"] = (0.2 * normal(width)).to(dt)
        if case["op"] == "norm_train":
            s["dy"] = normal(rows, width).to(dt)
        return s

    H, HV = case["H"], case["HV"]
    lead = (case["N"],) if case["op"] == "step" else (case["B"], case["T"])

    def unit(*shape):
        x = normal(*shape)
        return (x / x.square().sum(-1, keepdim=True).sqrt()).to(dt)

    s["q"], s["k"] = unit(*lead, H, K), unit(*lead, H, K)
    s["v"] = normal(*lead, HV, K).to(dt)
    s["gate"] = case["lo"] * uniform(*lead, HV, K)  # per-step log2 decay of each channel
    s["beta"] = uniform(*lead, HV)
    s["scale"] = K ** -0.5
    if case["op"] == "step":
        s["state"] = normal(case["N"], HV, K, K)
        return s
    s["lens"], s["cu_seqlens"] = None, None
    if case["lens"]:
        s["lens"] = [int(n) for n in case["lens"].split(",")]
        ends = torch.tensor([0] + s["lens"]).cumsum(0)
        s["cu_seqlens"] = ends.to(torch.int32).to(dev)
    if case["op"] == "train":
        s["do"] = normal(*lead, HV, K).to(dt)
    else:
        s["initial_state"] = normal(len(s["lens"]) if s["lens"] else case["B"], HV, K, K)
    return s


# ---------------------------------------------------------------------------- run
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import gated_delta_rule_intra_gb300 as kda

    if s["op"] == "norm":
        return {"y": kda.kda_layer_norm_fwd(s["x"], s["weight"], s["bias"])[0]}
    if s["op"] == "norm_train":
        y, mean, rstd = kda.kda_layer_norm_fwd(s["x"], s["weight"], s["bias"])
        dx, dw, db = kda.kda_layer_norm_bwd(s["dy"], s["x"], s["weight"], mean, rstd)
        return {"y": y, "dx": dx, "dweight": dw, "dbias": db}
    args = (s["q"], s["k"], s["v"], s["gate"], s["beta"])
    if s["op"] == "step":
        return {"o": kda.kda_step(*args, s["state"], scale=s["scale"]), "state": s["state"]}
    if s["op"] == "prefill":
        o, final, _ = kda.kda_chunk_fwd(*args, scale=s["scale"], initial_state=s["initial_state"],
                                        output_final_state=True, cu_seqlens=s["cu_seqlens"])
        return {"o": o, "state": final}
    o, _, saved = kda.kda_chunk_fwd(*args, scale=s["scale"], cu_seqlens=s["cu_seqlens"], save=True)
    dq, dk, dv, dgate, dbeta, _ = kda.kda_chunk_bwd(*args, s["do"], saved, scale=s["scale"],
                                                    cu_seqlens=s["cu_seqlens"])
    return {"o": o, "dq": dq, "dk": dk, "dv": dv, "dgate": dgate, "dbeta": dbeta}


def _run_plain(s):
    if s["op"] in ("norm", "norm_train"):
        return _plain_norm(s)
    if s["op"] == "step":
        return _plain_step(s)
    args = [s[n].float() for n in ("q", "k", "v", "gate", "beta")]
    dt = s["q"].dtype
    if s["op"] == "prefill":
        with torch.no_grad():
            o, final = _plain_recurrence(*args, s["scale"], s["initial_state"], s["lens"])
        return {"o": o.to(dt), "state": final}
    args = [x.detach().requires_grad_() for x in args]
    o, _ = _plain_recurrence(*args, s["scale"], None, s["lens"])
    grads = torch.autograd.grad(o, args, s["do"].float())
    return {"o": o.detach().to(dt),
            **{n: g.to(dt) for n, g in zip(("dq", "dk", "dv", "dgate", "dbeta"), grads)}}


def _plain_norm(s):
    x, w, dt = s["x"].float(), s["weight"].float(), s["x"].dtype
    centred = x - x.mean(-1, keepdim=True)
    rstd = (centred.square().mean(-1, keepdim=True) + 1e-5).rsqrt()
    xhat = centred * rstd
    y = (xhat * w + s["bias"].float()).to(dt)
    if s["op"] == "norm":
        return {"y": y}
    dy = s["dy"].float()
    wdy = dy * w
    dx = rstd * (wdy - wdy.mean(-1, keepdim=True) - xhat * (wdy * xhat).mean(-1, keepdim=True))
    return {"y": y, "dx": dx.to(dt), "dweight": (dy * xhat).sum(0), "dbias": dy.sum(0)}


def _plain_step(s):
    q, k, v = (s[n].float() for n in ("q", "k", "v"))
    G = v.shape[1] // q.shape[1]
    q, k = (x.repeat_interleave(G, 1)[..., None] for x in (q, k))
    S = s["state"] * torch.exp2(s["gate"])[..., None]
    e = (v - (S * k).sum(-2)) * s["beta"][..., None]
    S = S + k * e[..., None, :]
    s["state"].copy_(S)
    o = s["scale"] * (S * q).sum(-2)
    return {"o": o.to(s["q"].dtype), "state": s["state"]}


def _plain_recurrence(q, k, v, gate, beta, scale, S, lens):
    """o and the final state in chunks of 16 tokens.  What does not depend on the state is
    computed for all chunks at once; the state goes from chunk to chunk in a loop, which the
    recurrence itself asks for."""
    C = 16
    B, T, HV = beta.shape
    G = HV // q.shape[2]
    q, k = (x.repeat_interleave(G, 2) if G > 1 else x for x in (q, k))
    if lens:  # the packed sequences as a batch padded at its end
        n = torch.tensor(lens, device=q.device)
        longest = max(lens)
        at = torch.arange(longest, device=q.device)
        inside = at < n[:, None]
        token = ((n.cumsum(0) - n)[:, None] + at).clamp(max=T - 1)
        q, k, v, gate, beta = (x[0][token] * inside.reshape(*inside.shape, *[1] * (x.dim() - 2))
                               for x in (q, k, v, gate, beta))
        B, Tp = len(lens), longest
    else:
        Tp = T
    NC = -(-Tp // C)

    def chunks(x):  # [B, T, HV, ...] -> [B, HV, NC, C, ...], zeros behind the end
        x = torch.cat([x, x.new_zeros(B, NC * C - Tp, *x.shape[2:])], 1) if NC * C > Tp else x
        return x.unflatten(1, (NC, C)).movedim(3, 1)

    q, k, v, gate = (chunks(x) for x in (q, k, v, gate))
    beta = chunks(beta[..., None])
    g = gate.cumsum(-2)
    r = torch.arange(C, device=q.device)
    later = (r[:, None] >= r)[..., None]
    E = torch.exp2((g[..., :, None, :] - g[..., None, :, :]).masked_fill(~later, float("-inf")))
    kE = k[..., None, :, :] * E
    P = scale * (q[..., :, None, :] * kE).sum(-1)
    L = beta * (k[..., :, None, :] * kE).sum(-1) * (r[:, None] > r)
    del E, kE
    eye = torch.eye(C, device=q.device)
    L2 = L @ L
    L4 = L2 @ L2
    inv = (eye - L) @ (eye + L2) @ (eye + L4) @ (eye + L4 @ L4)  # (I + L)^-1, as L^16 = 0
    Tb = inv * beta.transpose(-1, -2)
    up = torch.exp2(g)
    qw, kw = scale * q * up, k * up
    last = g[..., -1:, :]
    kd = (k * torch.exp2(last - g)).transpose(-1, -2)
    decay = torch.exp2(last).transpose(-1, -2)
    if S is None:
        S = q.new_zeros(B, HV, K, K)
    out = []
    for qw_c, kw_c, kd_c, v_c, P_c, T_c, a_c in zip(*(x.unbind(2) for x in (qw, kw, kd, v, P, Tb,
                                                                           decay))):
        N = T_c @ (v_c - kw_c @ S)
        out.append(qw_c @ S + P_c @ N)
        S = a_c * S + kd_c @ N
    o = torch.stack(out, 2).movedim(1, 3).flatten(1, 2)[:, :Tp]
    return (o[inside][None] if lens else o), S


# ---------------------------------------------------------------------------- cost
def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    if case["op"] in ("norm", "norm_train"):
        n, w = case["rows"] * case["width"], case["width"]
        if case["op"] == "norm":
            return {"bytes": 2 * n * e + 2 * w * e, "flops": 7 * n}
        # x and dy read, y and dx written; weight and bias in, their gradients out in fp32
        return {"bytes": 4 * n * e + 2 * w * e + 8 * w, "flops": 20 * n}
    H, HV = case["H"], case["HV"]
    tokens = case["N"] if case["op"] == "step" else case["B"] * case["T"]
    qk, val, gates = tokens * H * K * e, tokens * HV * K * e, tokens * HV * (K * 4 + 4)
    states = {"step": case.get("N", 0), "train": 0}.get(
        case["op"], len(case.get("lens", "").split(",")) if case.get("lens") else case.get("B", 0))
    states *= 2 * HV * K * K * 4  # read and written
    if case["op"] == "train":
        # q, k, v, do, gate, beta read once; o and a gradient for each of the five written
        moved = 4 * qk + 4 * val + gates + tokens * HV * (K * e + e)
        return {"bytes": moved, "flops": tokens * HV * K * K * (7 + 17)}
    return {"bytes": 2 * qk + 2 * val + gates + states, "flops": tokens * HV * K * K * 7}


# ---------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "norm_train"):
        return _exact_norm(s)
    if case["op"] == "step":
        r = _exact_tokens({**s, **{n: s[n][:, None] for n in ("q", "k", "v", "gate", "beta")},
                           "initial_state": s["state"], "lens": None})
        return {"o": r["o"][:, 0], "state": r["state"]}
    rows, longest = (len(s["lens"]), max(s["lens"])) if s["lens"] else (case["B"], case["T"])
    if longest > 40000 or rows * case["HV"] * longest * (2 if "do" in s else 0) > 1.1e6:
        return None  # the states of every token would not fit, or the time
    r = _exact_tokens(s)
    names = ("o", "dq", "dk", "dv", "dgate", "dbeta") if "do" in s else ("o", "state")
    return {n: r[n] for n in names}


def _exact_norm(s):
    x, w, b = s["x"].double(), s["weight"].double(), s["bias"].double()
    width = x.shape[1]
    mu = x.sum(1) / width
    sigma = ((x * x).sum(1) / width - mu * mu + 1e-5).sqrt()
    y = (x - mu[:, None]) / sigma[:, None] * w + b
    if "dy" not in s:
        return {"y": y}
    dy = s["dy"].double()
    z = (x - mu[:, None]) / sigma[:, None]
    dz = dy * w
    dsum, dzz = dz.sum(1) / width, (dz * z).sum(1) / width
    dx = (dz - dsum[:, None] - z * dzz[:, None]) / sigma[:, None]
    return {"y": y, "dx": dx, "dweight": (dy * z).sum(0), "dbias": dy.sum(0)}


def _exact_tokens(s):
    """Token by token from the definition, and its adjoint token by token backwards:
    S~ = a S, e = v - S~^T k, S' = S~ + beta k e^T, o = scale S'^T q."""
    f = torch.float64
    q, k, v, gate, beta = (s[n].to(f) for n in ("q", "k", "v", "gate", "beta"))
    H, HV = q.shape[2], v.shape[2]
    spans = [(b, 0, q.shape[1]) for b in range(q.shape[0])]
    if s["lens"]:
        ends = [sum(s["lens"][:i + 1]) for i in range(len(s["lens"]))]
        spans = [(0, e - n, n) for e, n in zip(ends, s["lens"])]
    Tm, N = max(n for _, _, n in spans), len(spans)

    def rows(x):  # sequences side by side, zeros (no decay, no write) behind their ends
        x = x.repeat_interleave(HV // x.shape[2], 2)
        y = x.new_zeros(Tm, N, *x.shape[2:])
        for i, (b, at, n) in enumerate(spans):
            y[:n, i] = x[b, at:at + n]
        return y.flatten(1, 2)

    def back(y, like, heads):
        y = y.reshape(Tm, N, HV, *y.shape[2:])
        x = y.new_zeros(*like.shape[:2], *y.shape[2:])
        for i, (b, at, n) in enumerate(spans):
            x[b, at:at + n] = y[:n, i]
        return x.unflatten(2, (heads, -1)).sum(3)

    q, k, v, a, beta = rows(q), rows(k), rows(v), torch.exp2(rows(gate)), rows(beta)
    M = q.shape[1]
    S = s["initial_state"].to(f).flatten(0, 1).clone() if s.get("initial_state") is not None \
        else q.new_zeros(M, K, K)
    grads = "do" in s
    before = q.new_empty(Tm, M, K, K) if grads else None
    o, es = torch.empty_like(v), torch.empty_like(v)
    for t in range(Tm):
        if grads:
            before[t] = S
        S = a[t, :, :, None] * S
        es[t] = v[t] - torch.bmm(k[t, :, None], S)[:, 0]
        S = torch.baddbmm(S, k[t, :, :, None], (beta[t, :, None] * es[t])[:, None])
        o[t] = s["scale"] * torch.bmm(q[t, :, None], S)[:, 0]
    found = {"o": back(o, s["v"], HV), "state": S.reshape(N, HV, K, K)}
    if not grads:
        return found
    do = rows(s["do"].to(f))
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg, db = torch.empty_like(a), torch.empty_like(beta)
    dS = torch.zeros_like(S)
    ln2 = 0.6931471805599453
    for t in reversed(range(Tm)):
        kt, n = k[t, :, :, None], (beta[t, :, None] * es[t])[:, None]
        decayed = a[t, :, :, None] * before[t]
        dS = torch.baddbmm(dS, q[t, :, :, None], s["scale"] * do[t][:, None])
        after = torch.baddbmm(decayed, kt, n)
        dq[t] = s["scale"] * torch.bmm(after, do[t][:, :, None])[..., 0]
        dn = torch.bmm(kt.mT, dS)
        db[t] = (dn[:, 0] * es[t]).sum(-1)
        dv[t] = beta[t, :, None] * dn[:, 0]
        dk[t] = torch.bmm(dS, n.mT)[..., 0] - torch.bmm(decayed, dv[t][:, :, None])[..., 0]
        dS = torch.baddbmm(dS, kt, dv[t][:, None], alpha=-1)
        dg[t] = ln2 * (dS * decayed).sum(-1)
        dS = a[t, :, :, None] * dS
    for name, y, like, heads in (("dq", dq, s["q"], H), ("dk", dk, s["k"], H),
                                 ("dv", dv, s["v"], HV), ("dgate", dg, s["v"], HV),
                                 ("dbeta", db, s["v"], HV)):
        found[name] = back(y, like, heads)
    return found
