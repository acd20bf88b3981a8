"""The short convolution, the selective scan and the matrix product with its epilogue from their
definitions in 64 bits (gradients by autograd through them), and small inputs for their tests."""

import torch

F64 = torch.float64
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32

# An output that is rounded once is within the type's unit roundoff (half a step: eps / 2) of the exact
# one in the 2-norm; what is computed in FP32 on the way adds its own: sums of up to some thousand terms
# of random sign and exponentials of 2^-22, 4e-6.
UNIT = {BF: 2.0 ** -8, HF: 2.0 ** -11, F32: 0.0}
SUMS = 4e-6


def tol(dtype):
    return UNIT[dtype] + SUMS


def rel(got, ref):
    got, ref = got.detach().cpu().double(), ref.detach().cpu().double()
    assert got.shape == ref.shape, (got.shape, ref.shape)
    assert torch.isfinite(got).all()
    return float((got - ref).norm() / ref.norm().clamp(min=1e-30)) if ref.numel() else 0.0


def cuda(x):
    return {n: t.cuda() if torch.is_tensor(t) else t for n, t in x.items()}


def spans(B, T, lens=None, start=0):
    """(batch, first token, tokens) of every sequence."""
    if lens is None:
        return [(b, 0, T) for b in range(B)]
    out = []
    for n in lens:
        out.append((0, start, n))
        start += n
    return out


def cu(lens, start=0):
    return (torch.tensor([0] + list(lens)).cumsum(0) + start).to(torch.int32).cuda()


def act64(x, act):
    if act == "silu":
        return x * torch.sigmoid(x)
    if act == "gelu":
        return 0.5 * x * torch.erfc(-x * 0.5 ** 0.5)
    return torch.relu(x) if act == "relu" else x


def normal(gen, *shape):
    return torch.randn(*shape, generator=gen)


# ---------------------------------------------------------------------------- convolution
def make_conv(B, T, D, W, dtype=BF, wdtype=None, seqs=None, seed=0):
    g = torch.Generator().manual_seed(seed)
    wdtype = wdtype or dtype
    seqs = B if seqs is None else seqs
    return {"x": normal(g, B, T, D).to(dtype), "weight": (normal(g, D, W) * W ** -0.5).to(wdtype),
            "bias": (0.3 * normal(g, D)).to(wdtype), "dy": normal(g, B, T, D).to(dtype),
            "initial": normal(g, seqs, W - 1, D).to(dtype),
            "dfinal": normal(g, seqs, W - 1, D).to(dtype)}


def conv64(x, weight, bias, initial, act, lens=None, start=0):
    """(y, final states); tensors in 64 bits, which may require gradients."""
    B, T, D = x.shape
    W = weight.shape[1]
    y, finals = torch.zeros(B, T, D, dtype=F64), []
    for i, (b, at, n) in enumerate(spans(B, T, lens, start)):
        front = torch.zeros(W - 1, D, dtype=F64) if initial is None else initial[i]
        seq = torch.cat([front, x[b, at:at + n]])
        pre = sum(seq[j:j + n] * weight[:, j] for j in range(W))
        if bias is not None:
            pre = pre + bias
        rows = torch.zeros(B, T, D, dtype=F64)
        y = y + rows.index_put((torch.tensor(b), torch.arange(at, at + n)), act64(pre, act))
        finals.append(seq[n:])
    return y, torch.stack(finals)


# ---------------------------------------------------------------------------- scan
SCAN = ("u", "delta", "A", "B", "C", "D", "z", "delta_bias")


def make_scan(B, T, D, N, G=1, dtype=BF, seqs=None, seed=0):
    g = torch.Generator().manual_seed(seed)
    seqs = B if seqs is None else seqs
    return {"u": normal(g, B, T, D).to(dtype), "delta": (0.5 * normal(g, B, T, D)).to(dtype),
            "A": -torch.arange(1, N + 1) * torch.exp(0.2 * normal(g, D, N)),
            "B": normal(g, B, T, G, N).to(dtype), "C": normal(g, B, T, G, N).to(dtype),
            "D": 1 + 0.3 * normal(g, D), "z": normal(g, B, T, D).to(dtype),
            "delta_bias": normal(g, D) - 3, "dy": normal(g, B, T, D).to(dtype),
            "initial": normal(g, seqs, D, N), "dfinal": normal(g, seqs, D, N)}


def scan64(u, delta, A, Bm, Cm, D=None, z=None, delta_bias=None, initial=None, softplus=True,
           lens=None, start=0):
    """(y, final states) token by token; tensors in 64 bits, which may require gradients."""
    batch, T, width = u.shape
    per = width // Bm.shape[2]
    s = delta if delta_bias is None else delta + delta_bias
    if softplus:
        s = torch.clamp(s, min=0) + torch.log1p(torch.exp(-s.abs()))
    rows, finals = {}, []
    for i, (b, at, n) in enumerate(spans(batch, T, lens, start)):
        h = torch.zeros(width, A.shape[1], dtype=F64) if initial is None else initial[i]
        for t in range(at, at + n):
            Bt, Ct = (v[b, t].repeat_interleave(per, 0) for v in (Bm, Cm))
            h = torch.exp(s[b, t][:, None] * A) * h + (s[b, t] * u[b, t])[:, None] * Bt
            rows[b, t] = (h * Ct).sum(-1)
        finals.append(h)
    none = torch.zeros(width, dtype=F64)
    if T == 0:
        return torch.zeros(batch, 0, width, dtype=F64), torch.stack(finals)
    y = torch.stack([torch.stack([rows.get((b, t), none) for t in range(T)]) for b in range(batch)])
    inside = torch.zeros(batch, T, 1, dtype=F64)
    for b, t in rows:
        inside[b, t] = 1
    if D is not None:
        y = y + D * u * inside
    return (y if z is None else y * act64(z, "silu")), torch.stack(finals)


# ---------------------------------------------------------------------------- matrix product
def make_linear(M, K, N, dtype=BF, seed=0, lead=None):
    g = torch.Generator().manual_seed(seed)
    lead = (M,) if lead is None else lead
    return {"x": normal(g, *lead, K).to(dtype), "weight": (normal(g, N, K) * K ** -0.5).to(dtype),
            "bias": (0.3 * normal(g, N)).to(dtype), "residual": normal(g, *lead, N).to(dtype),
            "dy": normal(g, *lead, N).to(dtype)}


def leaves(x, names):
    return {n: x[n].detach().cpu().to(F64).requires_grad_() for n in names}
