"""The operators of a layer with a selective state-space scan, and the matrix products around it and
around the recurrence, as a user's program calls them, with a plain form of each in elementary torch
operations and a 64-bit definition to compare with.

Ops (the case's "op"):
  conv_train    short causal convolution with its activation, forward and backward
  conv          the same forward only, from given last inputs, with the new ones (a prompt)
  conv_step     its single-token form: one token for each of N requests, last inputs in place
  scan_train    selective state-space scan with skip and gate, forward and backward
  scan          the same forward only, from a given state, with the final one (a prompt)
  scan_step     its single-token form, states updated in place
  linear        matrix product with bias, activation and residual
  linear_train  the same, forward and backward
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------- cases
def _conv(name, op, T, D, W, B=1, lens="", dtype="bf16", act="silu"):
    c = {"op": op, "B": B, "T": T, "D": D, "W": W, "lens": lens, "dtype": dtype, "act": act}
    return {"name": name, **c} if name else c


def _scan(name, op, T, D, N=16, G=1, B=1, lens="", dtype="bf16"):
    c = {"op": op, "B": B, "T": T, "D": D, "N": N, "G": G, "lens": lens, "dtype": dtype}
    return {"name": name, **c} if name else c


def _linear(name, op, M, K, N, act="", bias=True, residual=False, dtype="bf16"):
    c = {"op": op, "M": M, "K": K, "N": N, "act": act, "bias": bias, "residual": residual,
         "dtype": dtype}
    return {"name": name, **c} if name else c


_PACKED = "1,17,640,63,129,4096,65,2500,1956"


def listed():
    return [
        # the convolution of q, k and v together in the library's headline layer: 16 heads of 128
        _conv("conv_train_headline", "conv_train", 4096, 6144, 4, B=8),
        # documents of very different lengths packed into one row, an odd number of channels
        _conv("conv_train_packed", "conv_train", 9467, 1111, 3, lens=_PACKED, dtype="fp16"),
        # one token of a few requests
        _conv("conv_step_few", "conv_step", 4, 4096, 4),
        # one layer of a training step: width 2048, twice that inside
        _scan("scan_train", "scan_train", 2048, 4096, B=4),
        # packed documents, input and output vectors in two groups
        _scan("scan_train_packed", "scan_train", 9467, 1000, G=2, lens=_PACKED, dtype="fp16"),
        # one very long prompt
        _scan("scan_long", "scan", 32768, 4096),
        # a short prompt that continues a conversation
        _scan("scan_short", "scan", 37, 2048),
        # decoding for a full serving batch
        _scan("scan_step_batch", "scan_step", 256, 4096),
        # the way into a wide hidden layer, of the headline workload's tokens
        _linear("linear_wide", "linear", 32768, 2048, 8192, act="silu"),
        # the way out of a layer for one token of four requests, onto the residual stream
        _linear("linear_token", "linear", 4, 4096, 2048, bias=False, residual=True),
        # a hidden layer's training step
        _linear("linear_train", "linear_train", 8192, 2048, 8192, act="gelu"),
        # sizes that are a multiple of nothing, onto the residual stream
        _linear("linear_train_odd", "linear_train", 2021, 1111, 1540, act="silu", residual=True,
                dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def _lens(rng, most):
    n = rng.randint(1, 9)
    return [_log(rng, 1, max(1, most // n // 2)) for _ in range(n)]


def draw(rng):
    op = rng.choice(["conv_train", "conv", "conv_step", "scan_train", "scan_train", "scan",
                     "scan_step", "linear", "linear", "linear_train"])
    dtype = rng.choice(["bf16", "fp16"])
    if op.startswith("linear"):
        most = 1 << (37 if op == "linear_train" else 39)  # multiplications
        K, N = (rng.choice([_log(rng, 1, 8192), 8 * _log(rng, 1, 1024)]) for _ in range(2))
        return _linear("", op, _log(rng, 1, max(1, min(32768, most // (K * N)))), K, N,
                       act=rng.choice(["", "silu", "gelu", "relu"]), bias=rng.random() < 0.6,
                       residual=rng.random() < 0.5, dtype=dtype)
    if op.startswith("conv"):
        D = rng.choice([_log(rng, 1, 8192), 64 * _log(rng, 1, 128)])
        make = lambda *a, **k: _conv("", op, *a, act=rng.choice(["silu", ""]),  # noqa: E731
                                     dtype=rng.choice([dtype, "fp32"]), **k)
        width, most = rng.choice([2, 3, 4, 4]), (1 << 27) // D
    else:
        D = rng.choice([_log(rng, 1, 2048) * 2, 64 * _log(rng, 1, 64)])
        G = rng.choice([1, 1, 2])
        make = lambda *a, **k: _scan("", op, *a, G=G, dtype=dtype, **k)  # noqa: E731
        width = rng.choice([4, 7, 8, 16, 16, 32])
        most = (1 << (29 if op == "scan_train" else 31)) // (D * width)
    if op.endswith("step"):
        return make(_log(rng, 1, max(1, min(512, (1 << 24) // (D * width)))), D, width)
    most = max(1, min(most, 65536))
    if rng.random() < 0.4:
        lens = _lens(rng, most)
        return make(sum(lens), D, width, lens=",".join(map(str, lens)))
    T = _log(rng, 1, min(most, 16384))
    return make(T, D, width, B=_log(rng, 1, max(1, min(16, most // T))))


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

    s = {"op": case["op"], "lens": None, "cu_seqlens": None}
    if case["op"].startswith("linear"):
        M, K, N = case["M"], case["K"], case["N"]
        s["act"] = case["act"] or None
        s["x"], s["weight"] = normal(M, K).to(dt), (normal(N, K) * K ** -0.5).to(dt)
        s["bias"] = (0.2 * normal(N)).to(dt) if case["bias"] else None
        s["residual"] = normal(M, N).to(dt) if case["residual"] else None
        if case["op"] == "linear_train":
            s["dy"] = normal(M, N).to(dt)
        return s
    step = case["op"].endswith("step")
    B, T, D = case["B"], case["T"], case["D"]
    lead = (T,) if step else (B, T)
    if case["lens"]:
        s["lens"] = [int(n) for n in case["lens"].split(",")]
        ends = torch.tensor([0] + s["lens"]).cumsum(0)
        s["cu_seqlens"] = ends.to(torch.int32).to(dev)
    seqs = T if step else len(s["lens"]) if s["lens"] else B
    train = case["op"].endswith("train")
    if train:
        s["dy"] = normal(*lead, D).to(dt)
    if case["op"].startswith("conv"):
        s["act"] = case["act"] or None
        # one half of what the projection in front of it writes
        s["x"] = normal(*lead, 2 * D).to(dt)[..., :D]
        s["weight"] = (normal(D, case["W"]) * case["W"] ** -0.5).to(dt)
        s["bias"] = (0.2 * normal(D)).to(dt)
        if not train:
            s["state"] = normal(seqs, case["W"] - 1, D).to(dt)
        return s
    N, G = case["N"], case["G"]
    s["u"] = normal(*lead, D).to(dt)
    s["z"] = normal(*lead, 2 * D).to(dt)[..., D:]  # the projection's other half
    s["delta"] = (0.5 * normal(*lead, D)).to(dt)
    # step sizes between 0.001 and 0.1 before the inputs' share, through the softplus
    dt0 = torch.exp(uniform(D) * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
    s["delta_bias"] = dt0 + torch.log(-torch.expm1(-dt0))
    # input and output vectors are slices of one projection, behind the step sizes' low rank
    rank = 8 * max(1, D // 128)
    bc = normal(*lead, rank + 2 * G * N).to(dt)
    s["B"] = bc[..., rank:rank + G * N].unflatten(-1, (G, N))
    s["C"] = bc[..., rank + G * N:].unflatten(-1, (G, N))
    s["A"] = -torch.arange(1, N + 1, device=dev) * torch.exp(0.1 * normal(D, N))
    s["skip"] = 1 + 0.2 * normal(D)
    if not train:
        s["state"] = normal(seqs, D, N)
    return s


# ---------------------------------------------------------------------------- run
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import gated_delta_rule_intra_gb300 as kda

    op = s["op"]
    if op == "linear":
        return {"y": kda.kda_linear_fwd(s["x"], s["weight"], s["bias"], s["residual"],
                                        activation=s["act"])[0]}
    if op == "linear_train":
        y, saved = kda.kda_linear_fwd(s["x"], s["weight"], s["bias"], s["residual"],
                                      activation=s["act"], save=True)
        dx, dw, db = kda.kda_linear_bwd(s["dy"], s["x"], s["weight"], saved, activation=s["act"],
                                        bias_grad=s["bias"] is not None)
        return _present(y=y, dx=dx, dweight=dw, dbias=db)
    if op == "conv_step":
        return {"y": kda.kda_conv_step(s["x"], s["state"], s["weight"], s["bias"],
                                       activation=s["act"]), "state": s["state"]}
    if op == "conv":
        y, last = kda.kda_conv_fwd(s["x"], s["weight"], s["bias"], s["state"],
                                   activation=s["act"], output_final_state=True,
                                   cu_seqlens=s["cu_seqlens"])
        return {"y": y, "state": last}
    if op == "conv_train":
        y, _ = kda.kda_conv_fwd(s["x"], s["weight"], s["bias"], activation=s["act"],
                                cu_seqlens=s["cu_seqlens"])
        dx, dw, db, _ = kda.kda_conv_bwd(s["dy"], s["x"], s["weight"], s["bias"],
                                         activation=s["act"], cu_seqlens=s["cu_seqlens"])
        return {"y": y, "dx": dx, "dweight": dw, "dbias": db}
    args = (s["u"], s["delta"], s["A"], s["B"], s["C"])
    more = (s["skip"], s["z"], s["delta_bias"])
    if op == "scan_step":
        return {"y": kda.kda_scan_step(*args, s["state"], *more), "state": s["state"]}
    if op == "scan":
        y, final, _ = kda.kda_scan_fwd(*args, *more, s["state"], output_final_state=True,
                                       cu_seqlens=s["cu_seqlens"])
        return {"y": y, "state": final}
    y, _, saved = kda.kda_scan_fwd(*args, *more, save=True, cu_seqlens=s["cu_seqlens"])
    grads = kda.kda_scan_bwd(s["dy"], *args, saved, *more, cu_seqlens=s["cu_seqlens"])
    return {"y": y, **dict(zip(_SCAN_GRADS, grads))}


_SCAN_GRADS = ("du", "ddelta", "dA", "dB", "dC", "dD", "dz", "ddelta_bias")
_SCAN_INPUTS = ("u", "delta", "A", "B", "C", "skip", "z", "delta_bias")


def _present(**outputs):
    return {n: t for n, t in outputs.items() if t is not None}


def _act(x, act):
    if act == "silu":
        return x * torch.sigmoid(x)
    if act == "gelu":
        return 0.5 * x * (1 + torch.erf(x * 0.5 ** 0.5))
    return x.clamp(min=0) if act == "relu" else x


def _run_plain(s):
    op = s["op"]
    if op.startswith("linear"):
        return _plain_linear(s)
    if op == "conv_step":
        x, st = s["x"].float(), s["state"].float()
        window = torch.cat([st, x[:, None]], 1)
        y = (window * s["weight"].float().T).sum(1) + s["bias"].float()
        s["state"].copy_(window[:, 1:])
        return {"y": _act(y, s["act"]).to(s["x"].dtype), "state": s["state"]}
    if op == "scan_step":
        u, z = s["u"].float(), s["z"].float()
        d = s["delta"].float() + s["delta_bias"]
        d = d.clamp(min=0) + torch.log1p(torch.exp(-d.abs()))
        Bm, Cm = (s[n].float().repeat_interleave(u.shape[1] // s[n].shape[1], 1) for n in "BC")
        h = s["state"] * torch.exp(d[..., None] * s["A"]) + (d * u)[..., None] * Bm
        s["state"].copy_(h)
        y = ((h * Cm).sum(-1) + s["skip"] * u) * _act(z, "silu")
        return {"y": y.to(s["u"].dtype), "state": s["state"]}
    if op.startswith("conv"):
        dt, train = s["x"].dtype, op == "conv_train"
        leaf = [s[n].float().detach().requires_grad_(train) for n in ("x", "weight", "bias")]
        y, last = _plain_conv(*leaf, s.get("state"), s["lens"], s["act"])
        if not train:
            return {"y": y.to(dt), "state": last}
        dx, dw, db = torch.autograd.grad(y, leaf, s["dy"].float())
        return {"y": y.detach().to(dt), "dx": dx.to(dt), "dweight": dw, "dbias": db}
    dt, train = s["u"].dtype, op == "scan_train"
    leaf = [s[n].float().detach().requires_grad_(train) for n in _SCAN_INPUTS]
    y, final = _plain_scan(*leaf, s.get("state"), s["lens"])
    if not train:
        return {"y": y.to(dt), "state": final}
    grads = torch.autograd.grad(y, leaf, s["dy"].float())
    return {"y": y.detach().to(dt),
            **{n: g.to(s[i].dtype) for n, i, g in zip(_SCAN_GRADS, _SCAN_INPUTS, grads)}}


def _plain_linear(s):
    x, w, dt = s["x"].float(), s["weight"].float(), s["x"].dtype
    pre = x @ w.T
    if s["bias"] is not None:
        pre = pre + s["bias"].float()
    y = _act(pre, s["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    if s["op"] == "linear":
        return {"y": y.to(dt)}
    g = s["dy"].float()
    if s["act"] == "relu":
        g = g * (pre > 0)
    elif s["act"] == "silu":
        sig = torch.sigmoid(pre)
        g = g * sig * (1 + pre * (1 - sig))
    elif s["act"] == "gelu":
        g = g * (0.5 * (1 + torch.erf(pre * 0.5 ** 0.5))
                 + pre * torch.exp(-0.5 * pre * pre) * (2 * math.pi) ** -0.5)
    return _present(y=y.to(dt), dx=(g @ w).to(dt), dweight=(g.T @ x).to(dt),
                    dbias=g.sum(0).to(dt) if s["bias"] is not None else None)


def _batch(lens, T, device):
    """Packed sequences as a batch padded at its end: (token [n, longest], inside)."""
    n = torch.tensor(lens, device=device)
    at = torch.arange(max(lens), device=device)
    return ((n.cumsum(0) - n)[:, None] + at).clamp(max=T - 1), at < n[:, None]


def _plain_conv(x, w, b, state, lens, act):
    T, W = x.shape[1], w.shape[1]
    if lens:
        token, inside = _batch(lens, T, x.device)
        x = x[0][token]
    front = x.new_zeros(x.shape[0], W - 1, x.shape[2]) if state is None else state.float()
    full = torch.cat([front, x], 1)
    y = b
    for j in range(W):
        y = y + full[:, j:j + x.shape[1]] * w[:, j]
    y = _act(y, act)
    last = None
    if state is not None:  # the last W - 1 inputs of every sequence
        n = torch.tensor(lens or [T] * x.shape[0], device=x.device)
        rows = n[:, None] + torch.arange(W - 1, device=x.device)
        last = full.gather(1, rows[..., None].expand(-1, -1, x.shape[2])).to(state.dtype)
    return (y[inside][None] if lens else y), last


def _plain_scan(u, delta, A, Bm, Cm, skip, z, delta_bias, h0, lens):
    """Pieces of C tokens: every piece from a zero state, all pieces side by side; then the states
    from piece to piece in a loop; then what each piece's first state adds to its tokens."""
    T, D, N = u.shape[1], u.shape[2], A.shape[1]
    d = delta + delta_bias
    d = d.clamp(min=0) + torch.log1p(torch.exp(-d.abs()))
    x = d * u
    C = max(1, min(64, int(T ** 0.5)))

    def pieces(t):  # [B, T, ...] -> C tensors [B, pieces, ...], zeros behind the end
        if lens:
            t = t[0][token] * inside.reshape(*inside.shape, *[1] * (t.dim() - 2))
        more = -t.shape[1] % C
        if more:
            t = torch.cat([t, t.new_zeros(t.shape[0], more, *t.shape[2:])], 1)
        return t.unflatten(1, (-1, C)).unbind(2)

    if lens:
        token, inside = _batch(lens, T, u.device)
    per = D // Bm.shape[2]
    groups = lambda t: t.unflatten(-1, (-1, per))  # noqa: E731   [.., D] -> [.., G, D / G]
    A = A.unflatten(0, (-1, per))
    h, total, local, decay = 0, 0, [], []
    for d_t, x_t, B_t in zip(pieces(groups(d)), pieces(groups(x)), pieces(Bm)):
        total = total + d_t
        h = h * torch.exp(d_t[..., None] * A) + x_t[..., None] * B_t[..., None, :]
        local.append(h)
        decay.append(total)
    B, NP = h.shape[:2]
    H = h.new_zeros(B, *h.shape[2:]) if h0 is None else h0.unflatten(1, (-1, per))
    before = []
    for p, (last, a) in enumerate(zip(h.unbind(1), torch.exp(total[..., None] * A).unbind(1))):
        before.append(H)
        H = a * H + last
    before = torch.stack(before, 1)
    out = [((h_t + torch.exp(s_t[..., None] * A) * before) * C_t[..., None, :]).sum(-1)
           for h_t, s_t, C_t in zip(local, decay, pieces(Cm))]
    y = torch.stack(out, 2).flatten(1, 2).flatten(-2)
    y = y[:, :max(lens)][inside][None] if lens else y[:, :T]
    return (y + skip * u) * _act(z, "silu"), H.flatten(1, 2)


# ---------------------------------------------------------------------------- cost
def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    op, train = case["op"], case["op"].endswith("train")
    if op.startswith("linear"):
        M, K, N = case["M"], case["K"], case["N"]
        x, w, y = M * K * e, N * K * e, M * N * e
        moved = x + w + y * (2 if case["residual"] else 1) + (N * e if case["bias"] else 0)
        # the backward also reads dy and writes dx, dweight and dbias
        moved += train * (y + x + w + (N * e if case["bias"] else 0))
        return {"bytes": moved, "flops": 2 * M * K * N * (3 if train else 1)}
    tokens = case["T"] * (1 if op.endswith("step") else case["B"])
    seqs = case["T"] if op.endswith("step") else \
        len(case["lens"].split(",")) if case["lens"] else case["B"]
    D = case["D"]
    row = tokens * D * e
    if op.startswith("conv"):
        W = case["W"]
        params = D * (W + 1)
        if train:  # x and dy read, y and dx written; the parameters' gradients in fp32
            return {"bytes": 4 * row + params * (e + 4), "flops": tokens * D * (6 * W + 12)}
        return {"bytes": 2 * row + params * e + 2 * seqs * (W - 1) * D * e,
                "flops": tokens * D * (2 * W + 5)}
    N, G = case["N"], case["G"]
    params = D * (N + 2) * 4
    if train:  # u, delta, z and dy read, y and three gradients written, B and C and theirs
        return {"bytes": 8 * row + 4 * tokens * G * N * e + 2 * params,
                "flops": tokens * D * (N * 22 + 40)}
    return {"bytes": 4 * row + 2 * tokens * G * N * e + params + 2 * seqs * D * N * 4,
            "flops": tokens * D * (N * 7 + 15)}


# ---------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f = {n: t.double() if torch.is_tensor(t) and t.is_floating_point() else t
         for n, t in s.items()}
    op = case["op"]
    if op.startswith("linear"):
        return _exact_linear(f)
    if op.endswith("step"):  # a sequence of one token for each request
        for n in ("x", "u", "z", "delta", "B", "C"):
            if n in f:
                f[n] = f[n][:, None]
        r = _exact_conv(f) if op == "conv_step" else _exact_scan(f)
        return {"y": r["y"][:, 0], "state": r["state"]}
    if op.startswith("conv"):
        return _exact_conv(f)
    spans = _spans(f, "u")
    longest, n = max(c for _, _, c in spans), len(spans)
    if longest > 70000 or case["op"] == "scan_train" and longest * n * case["D"] * case["N"] > 1.5e9:
        return None  # the time, or the states of every token, would be too much
    return _exact_scan(f)


def _spans(f, name):
    B, T = f[name].shape[:2]
    if not f["lens"]:
        return [(b, 0, T) for b in range(B)]
    at, out = 0, []
    for n in f["lens"]:
        out.append((0, at, n))
        at += n
    return out


def _slopes(x, act):
    """The activation and its derivative."""
    if act == "silu":
        e = 1 / (1 + torch.exp(-x))
        return x * e, e + x * e * (1 - e)
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-x / math.sqrt(2))
        return x * cdf, cdf + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    if act == "relu":
        return torch.where(x > 0, x, 0.0), (x > 0).double()
    return x, torch.ones_like(x)


def _exact_linear(f):
    pre = torch.einsum("mk,nk->mn", f["x"], f["weight"])
    if f["bias"] is not None:
        pre += f["bias"]
    y, slope = _slopes(pre, f["act"])
    if f["residual"] is not None:
        y = y + f["residual"]
    if "dy" not in f:
        return {"y": y}
    g = f["dy"] * slope
    return _present(y=y, dx=torch.einsum("mn,nk->mk", g, f["weight"]),
                    dweight=torch.einsum("mn,mk->nk", g, f["x"]),
                    dbias=torch.einsum("mn->n", g) if f["bias"] is not None else None)


def _exact_conv(f):
    x, w = f["x"], f["weight"]
    W = w.shape[1]
    y = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    dx, dw, db = torch.zeros_like(y), torch.zeros_like(w), torch.zeros_like(f["bias"])
    last = None if f.get("state") is None else torch.empty_like(f["state"])
    spans = _spans(f, "x")
    for i, (b, at, n) in enumerate(spans):
        seq = torch.zeros(n + W - 1, x.shape[2], dtype=torch.float64, device=x.device)
        if last is not None:
            seq[:W - 1] = f["state"][i]
        seq[W - 1:] = x[b, at:at + n]
        window = seq.unfold(0, W, 1)  # [n, D, W]
        out, slope = _slopes(torch.einsum("tdw,dw->td", window, w) + f["bias"], f["act"])
        y[b, at:at + n] = out
        if last is not None:
            last[i] = seq[n:]
        if "dy" in f:
            g = f["dy"][b, at:at + n] * slope
            db += g.sum(0)
            dw += torch.einsum("td,tdw->dw", g, window)
            for t in range(min(W, n)):  # an input reaches the token `t` behind it
                dx[b, at:at + n - t] += g[t:] * w[:, W - 1 - t]
    if "dy" in f:
        return {"y": y, "dx": dx, "dweight": dw, "dbias": db}
    return {"y": y, "state": last}


def _exact_scan(f):
    """Token by token, h = exp(delta A) h + delta u B, and its adjoint token by token backwards."""
    spans = _spans(f, "u")
    Tm, S = max(n for _, _, n in spans), len(spans)
    D, N = f["A"].shape
    G = f["B"].shape[2]

    def rows(x):  # [Tm, S, ...]: sequences side by side, zeros behind their ends
        y = x.new_zeros(Tm, S, *x.shape[2:])
        for i, (b, at, n) in enumerate(spans):
            y[:n, i] = x[b, at:at + n]
        return y

    def back(y, like):
        x = torch.zeros(like.shape, dtype=torch.float64, device=like.device)
        for i, (b, at, n) in enumerate(spans):
            x[b, at:at + n] = y[:n, i]
        return x

    raw = f["delta"] + f["delta_bias"]
    step = torch.where(raw > 0, raw + torch.log1p(torch.exp(-raw)), torch.log1p(torch.exp(raw)))
    u, d, z = rows(f["u"]), rows(step), rows(f["z"])
    Bv, Cv = rows(f["B"]), rows(f["C"])
    A = f["A"]
    h = f["state"].clone() if f.get("state") is not None else u.new_zeros(S, D, N)
    grads = "dy" in f
    hs = u.new_empty(Tm, S, D, N) if grads else None
    y = torch.empty_like(u)

    def wide(v):  # [S, G, N] -> [S, D, N]
        return v.repeat_interleave(D // G, 1)

    for t in range(Tm):
        if grads:
            hs[t] = h
        h = torch.addcmul((d[t] * u[t])[..., None] * wide(Bv[t]), torch.exp(d[t][..., None] * A), h)
        y[t] = torch.einsum("sdn,sdn->sd", h, wide(Cv[t]))
    full = y + f["skip"] * u
    gate, slope = _slopes(z, "silu")
    found = {"y": back(full * gate, f["u"]), "state": h}
    if not grads:
        return found
    dout = rows(f["dy"])
    dy = dout * gate
    du, dd = dy * f["skip"], torch.empty_like(d)
    dB, dC = torch.empty_like(Bv), torch.empty_like(Cv)
    dA, carry = torch.zeros_like(A), torch.zeros_like(h)

    def fold(v):  # [S, D, N] -> [S, G, N]
        return v.reshape(S, G, D // G, N).sum(2)

    for t in reversed(range(Tm)):
        decayed = torch.exp(d[t][..., None] * A) * hs[t]
        b = wide(Bv[t])
        h = decayed + (d[t] * u[t])[..., None] * b
        g = torch.addcmul(carry, dy[t][..., None], wide(Cv[t]))
        dC[t] = fold(dy[t][..., None] * h)
        dB[t] = fold(g * (d[t] * u[t])[..., None])
        gb, gp = (g * b).sum(-1), g * decayed
        du[t] += d[t] * gb
        dd[t] = u[t] * gb + (gp * A).sum(-1)
        dA += torch.einsum("sdn,sd->dn", gp, d[t])
        carry = g * torch.exp(d[t][..., None] * A)
    ddelta = back(dd, f["u"]) / (1 + torch.exp(-raw))
    if f["lens"]:  # nothing comes from behind a sequence's end: its rows there are zeros
        ddelta = ddelta * back(rows(torch.ones_like(f["u"])), f["u"])
    return {"y": found["y"], "du": back(du, f["u"]), "ddelta": ddelta, "dA": dA,
            "dB": back(dB, f["B"]), "dC": back(dC, f["C"]), "dD": (dy * u).sum((0, 1)),
            "dz": back(dout * full * slope, f["u"]), "ddelta_bias": ddelta.sum((0, 1))}
