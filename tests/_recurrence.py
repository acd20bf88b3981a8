"""The gated delta-rule recurrence token by token in 64 bits (autograd through the definition),
and small inputs for its tests."""

import torch

F64 = torch.float64
NAMES = ("q", "k", "v", "gate", "beta")
GRADS = ("dq", "dk", "dv", "dgate", "dbeta")

# Unit roundoff of the 16-bit types (2^-p, p = significand bits): an output that is rounded
# once is within this of the exact one in the 2-norm.  On top: states and sums are FP32 with
# operands of 16 bits, 3 * 2^-17 (rms) a product and a handful of products in a chain: 1e-5 for
# what stays in FP32; gradients subtract terms of the same size (the gate's): 1e-4.
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
STATE_TOL = 1e-5
EXTRA = 1e-4


def make(T, H, HV, B=1, dtype=torch.bfloat16, lo=-0.5, seed=0, lead=None):
    gen = torch.Generator().manual_seed(seed)
    lead = (B, T) if lead is None else lead

    def normal(*s):
        return torch.randn(*s, generator=gen)

    def unit(*s):
        x = normal(*s)
        return (x / x.norm(dim=-1, keepdim=True)).to(dtype)

    return {"q": unit(*lead, H, 128), "k": unit(*lead, H, 128),
            "v": normal(*lead, HV, 128).to(dtype),
            "gate": lo * torch.rand(*lead, HV, 128, generator=gen),
            "beta": torch.rand(*lead, HV, generator=gen)}


def states(n, HV, seed=1):
    return torch.randn(n, HV, 128, 128, generator=torch.Generator().manual_seed(seed))


def forward64(x, scale=128 ** -0.5, S0=None, lens=None):
    """(o, final states) in 64 bits from the definition; x's tensors may require gradients."""
    q, k, v, gate, beta = (x[n].to(F64) for n in NAMES)
    HV = v.shape[2]
    q, k = (t.repeat_interleave(HV // t.shape[2], 2) for t in (q, k))
    B, T = q.shape[:2]
    spans = [(b, 0, T) for b in range(B)]
    if lens is not None:
        at = [sum(lens[:i]) for i in range(len(lens))]
        spans = [(0, a, n) for a, n in zip(at, lens)]
    rows = {}
    finals = []
    for i, (b, at, n) in enumerate(spans):
        S = torch.zeros(HV, 128, 128, dtype=F64) if S0 is None else S0[i].to(F64)
        for t in range(at, at + n):
            S = torch.exp2(gate[b, t])[..., None] * S
            e = v[b, t] - torch.einsum("hkv,hk->hv", S, k[b, t])
            S = S + k[b, t][..., None] * (beta[b, t][..., None] * e)[:, None, :]
            rows[b, t] = scale * torch.einsum("hkv,hk->hv", S, q[b, t])
        finals.append(S)
    zero = torch.zeros(HV, 128, dtype=F64)
    o = torch.stack([torch.stack([rows.get((b, t), zero) for t in range(T)])
                     for b in range(B)]) if T else torch.zeros(B, 0, HV, 128, dtype=F64)
    return o, torch.stack(finals)


def gradients64(x, do, scale=128 ** -0.5, S0=None, dfinal=None, lens=None):
    """Gradients of <o, do> + <final, dfinal> for the five inputs and the initial states."""
    leaf = {n: x[n].to(F64).requires_grad_() for n in NAMES}
    s0 = None if S0 is None else S0.to(F64).requires_grad_()
    o, final = forward64(leaf, scale, s0, lens)
    loss = (o * do.to(F64)).sum()
    if dfinal is not None:
        loss = loss + (final * dfinal.to(F64)).sum()
    ins = [leaf[n] for n in NAMES] + ([] if s0 is None else [s0])
    got = torch.autograd.grad(loss, ins, allow_unused=True)
    got = [torch.zeros_like(i) if g is None else g for g, i in zip(got, ins)]
    return got[:5], (got[5] if s0 is not None else None)


def rel(got, ref):
    got, ref = got.detach().cpu().to(F64), ref.detach().cpu().to(F64)
    assert got.shape == ref.shape
    assert torch.isfinite(got).all()
    return float((got - ref).norm() / ref.norm().clamp(min=1e-30))


def cuda(x):
    return {n: t.cuda() for n, t in x.items()} if isinstance(x, dict) else x.cuda()


def cu(lens, start=0):
    return torch.tensor([start] + lens).cumsum(0).to(torch.int32).cuda()
