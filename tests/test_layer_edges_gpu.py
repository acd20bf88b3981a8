"""Convolution, scan and matrix product where they leave their usual course: the bounds-checked build,
other streams, graphs, the binding's two ways in, infinities, and gradients against differences."""

import threading

import pytest
import torch

import gated_delta_rule_intra_gb300 as kda
from gated_delta_rule_intra_gb300 import conv, linear, scan
from tests._layer import (BF, F32, F64, HF, SCAN, conv64, cu, cuda, make_conv, make_linear, make_scan,
                          rel, scan64, tol)
from tests.test_recurrence_edges_gpu import _debug

pytestmark = pytest.mark.gpu


def all_conv(x, packed=None, act="silu", states=False):
    i, f = (x["initial"], x["dfinal"]) if states else (None, None)
    y, last = kda.kda_conv_fwd(x["x"], x["weight"], x["bias"], i, activation=act, output_final_state=states,
                               cu_seqlens=packed)
    out = kda.kda_conv_bwd(x["dy"], x["x"], x["weight"], x["bias"], i, f, activation=act,
                           output_d_initial_state=states, cu_seqlens=packed)
    return [t for t in (y, last, *out) if t is not None]


def all_scan(x, packed=None, states=False):
    ins, more = [x[n] for n in SCAN[:5]], [x[n] for n in SCAN[5:]]
    i, f = (x["initial"], x["dfinal"]) if states else (None, None)
    y, last, saved = kda.kda_scan_fwd(*ins, *more, i, save=True, output_final_state=states, cu_seqlens=packed)
    out = kda.kda_scan_bwd(x["dy"], *ins, saved, *more, f, output_d_initial_state=states, cu_seqlens=packed)
    return [t for t in (y, last, *out) if t is not None]


def all_linear(x, act="gelu"):
    y, saved = kda.kda_linear_fwd(x["x"], x["weight"], x["bias"], x["residual"], activation=act, save=True)
    return [y, saved, *kda.kda_linear_bwd(x["dy"], x["x"], x["weight"], saved, activation=act)]


# ---------------------------------------------------------------------------- the bounds-checked build
@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("B,T,D,W,lens,start", [
    (2, 67, 264, 4, None, 0), (1, 1, 1, 2, None, 0), (3, 300, 77, 3, None, 0), (2, 2, 6, 4, None, 0),
    (1, 330, 129, 4, [5, 0, 1, 100, 200], 11), (1, 40, 8, 2, [], 0), (1, 700, 1032, 4, [96, 97, 500], 0)])
def test_debug_build_of_the_convolution(B, T, D, W, lens, start, dtype):
    lens = [3, 0, 30] if lens == [] else lens
    x = cuda(make_conv(B, T, D, W, dtype, seqs=None if lens is None else len(lens), seed=T))
    c = None if lens is None else cu(lens, start)
    _debug(lambda: all_conv(x, c))
    _debug(lambda: all_conv(x, c, None, True))


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("B,T,D,N,G,lens,start", [
    (2, 67, 64, 16, 1, None, 0), (1, 1, 1, 1, 1, None, 0), (2, 33, 77, 5, 1, None, 0), (1, 40, 66, 64, 3, None, 0),
    (1, 100, 33, 16, 1, [5, 0, 16, 17, 33], 11), (1, 900, 64, 16, 2, None, 0), (1, 1200, 24, 30, 1, [700, 1, 450], 7)])
def test_debug_build_of_the_scan(B, T, D, N, G, lens, start, dtype):
    x = cuda(make_scan(B, T, D, N, G, dtype, seqs=None if lens is None else len(lens), seed=T))
    c = None if lens is None else cu(lens, start)
    _debug(lambda: all_scan(x, c))
    _debug(lambda: all_scan(x, c, True))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("M,K,N", [(1, 1, 1), (7, 72, 40), (16, 77, 33), (17, 8, 8), (130, 77, 129), (300, 520, 136),
                                   (40, 4096, 64), (2048, 256, 2560)])
def test_debug_build_of_the_product(M, K, N, dtype):
    x = cuda(make_linear(M, K, N, dtype, seed=M))
    _debug(lambda: all_linear(x))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,N,R", [(64, 16, 5), (33, 7, 3), (512, 16, 130)])
def test_debug_build_of_single_tokens(D, N, R, dtype):
    c, s = cuda(make_conv(1, R, D, 4, dtype, seqs=R + 2)), cuda(make_scan(1, R, D, N, 1, dtype, seqs=R + 2))
    idx = torch.randperm(R + 2, generator=torch.Generator().manual_seed(1))[:R].to(torch.int32)
    idx[1] = -1
    idx = idx.cuda()
    ins, more = [s[n][0] if s[n].dim() > 2 else s[n] for n in SCAN[:5]], [s["D"], s["z"][0], s["delta_bias"]]

    def call():
        cs, ss = c["initial"].clone(), s["initial"].clone()
        y = kda.kda_conv_step(c["x"][0], cs, c["weight"], c["bias"], activation="silu", state_indices=idx)
        return y, cs, kda.kda_scan_step(*ins, ss, *more, state_indices=idx), ss

    _debug(call)


# ---------------------------------------------------------------------------- sizes
@pytest.mark.parametrize("M,K,N", [(5, 1111, 70), (16, 2049, 130), (1, 8191, 24)])
def test_few_rows_of_an_odd_contraction(M, K, N):
    """They take the tensor-memory kernel, the contraction cut into parts: with its workspace."""
    x = make_linear(M, K, N, BF, seed=K)
    c = cuda(x)
    copies = 3 if K % 8 else 0
    assert kda.load_library().kda_linear_fwd_workspace_bytes(M, K, N, copies) >= \
        2 * (M + N) * K + 4 * 2 * M * N  # the rows' copies, two parts at least
    y = kda.kda_linear_fwd(c["x"], c["weight"], c["bias"])[0]
    assert rel(y, x["x"].to(F64) @ x["weight"].to(F64).T + x["bias"].to(F64)) <= tol(BF)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("M,K,N", [(1, 2048, 8), (3, 2056, 40), (8, 4104, 2449), (9, 2048, 2432), (16, 6136, 4864),
                                   (5, 8192, 17)])
def test_few_rows_of_a_long_contraction(M, K, N, dtype):
    """Chunks of 1024 k that end in the middle, several times 16 columns a CTA, columns behind the last."""
    x = make_linear(M, K, N, dtype, seed=N)
    c = cuda(x)
    y, saved = kda.kda_linear_fwd(c["x"], c["weight"], c["bias"], c["residual"], activation="relu", save=True)
    pre = x["x"].to(F64) @ x["weight"].to(F64).T + x["bias"].to(F64)
    assert rel(saved, pre) <= tol(dtype) and rel(y, torch.relu(pre) + x["residual"].to(F64)) <= tol(dtype)
    _debug(lambda: [kda.kda_linear_fwd(c["x"], c["weight"], c["bias"])[0]])


@pytest.mark.parametrize("M", [17, 23, 31, 47, 64, 90, 120, 127, 129])
def test_rows_of_less_than_a_tile(M):
    """Where x has no rows nothing is copied, and what lies there (NaN from the call before) stays out."""
    bad = torch.full((300, 584), float("nan"), dtype=BF, device="cuda")
    for N in (72, 200):
        x = make_linear(M, 584, N, BF, seed=M)
        c = cuda(x)
        kda.kda_linear_fwd(bad, c["weight"])
        y = kda.kda_linear_fwd(c["x"], c["weight"], c["bias"])[0]
        assert rel(y, x["x"].to(F64) @ x["weight"].to(F64).T + x["bias"].to(F64)) <= tol(BF)


def test_more_sequences_than_a_grid_is_high():
    """70,000 sequences of one token, and their states."""
    n, D = 70000, 8
    x = cuda(make_conv(n, 1, D, 4, HF, seed=1))
    y, last = kda.kda_conv_fwd(x["x"], x["weight"], x["bias"], x["initial"], output_final_state=True)
    dx, dw, db, di = kda.kda_conv_bwd(x["dy"], x["x"], x["weight"], x["bias"], x["initial"], x["dfinal"],
                                      output_d_initial_state=True)
    seq = torch.cat([x["initial"], x["x"]], 1).double()
    w, dy, df = x["weight"].double(), x["dy"].double(), x["dfinal"].double()
    assert rel(y[:, 0], (seq * w.T).sum(1) + x["bias"].double()) <= tol(HF)
    assert torch.equal(last, seq[:, 1:].to(HF))
    ds = dy * w.T
    ds[:, 1:] += df
    assert rel(torch.cat([di, dx], 1), ds) <= tol(HF)
    # FP32 sums of 70,000 terms of random sign: their 2^-24 each, some hundred times over
    assert rel(dw, (dy * seq).sum(0).T) <= 1e-5 and rel(db, dy.sum((0, 1))) <= 1e-5
    s = cuda(make_scan(n, 1, D, 4, 1, HF, seed=2))
    ins, more = [s[m] for m in SCAN[:5]], [s[m] for m in SCAN[5:]]
    y, last, saved = kda.kda_scan_fwd(*ins, *more, s["initial"], save=True, output_final_state=True)
    out = kda.kda_scan_bwd(s["dy"], *ins, saved, *more, s["dfinal"], output_d_initial_state=True)
    few = slice(n - 50, n)
    part = {k: (t[few].cpu() if t.shape[0] == n else t.cpu()) for k, t in s.items()}
    h = {k: part[k].to(F64).requires_grad_() for k in (*SCAN, "initial")}
    want, final = scan64(*h.values())
    loss = (want * part["dy"].to(F64)).sum() + (final * part["dfinal"].to(F64)).sum()
    ref = dict(zip(h, torch.autograd.grad(loss, list(h.values()))))
    assert rel(y[few], want) <= tol(HF) and rel(last[few], final) <= 1e-5
    for got, name in zip(out, (*SCAN, "initial")):
        if got.shape[0] == n:
            assert rel(got[few], ref[name]) <= tol(HF) + 1e-5, name


def test_a_scan_of_more_than_2_to_31_elements():
    """The last tokens' results are those of a call on the last tokens alone, from the state that the
    first ones leave (segments differ: FP32 rounding and the type's)."""
    T, D, cut = 540000, 4000, 530000
    gen = torch.Generator("cuda").manual_seed(1)
    u, delta, dy = (torch.randn(1, T, D, device="cuda", generator=gen, dtype=BF) for _ in range(3))
    B, C = (torch.randn(1, T, 1, 2, device="cuda", generator=gen, dtype=BF) for _ in range(2))
    A = -torch.rand(D, 2, device="cuda", generator=gen) - 0.1
    y, last, saved = kda.kda_scan_fwd(u, delta, A, B, C, save=True, output_final_state=True)
    du, dd, _, dB, dC = kda.kda_scan_bwd(dy, u, delta, A, B, C, saved)[:5]
    del saved
    _, state, _ = kda.kda_scan_fwd(*(t[:, :cut] for t in (u, delta)), A, B[:, :cut], C[:, :cut],
                                   output_final_state=True)
    tail = [t[:, cut:] for t in (dy, u, delta, B, C)]
    ty, tl, ts = kda.kda_scan_fwd(*tail[1:3], A, *tail[3:], initial_state=state, save=True, output_final_state=True)
    out = kda.kda_scan_bwd(*tail[:3], A, *tail[3:], ts)
    assert rel(tl, last) <= 1e-5 and rel(ty, y[:, cut:]) <= 2 * tol(BF)
    for got, want in zip((out[0], out[1], out[3], out[4]), (du, dd, dB, dC)):
        assert rel(got, want[:, cut:]) <= 2 * tol(BF)


@pytest.mark.parametrize("D", [4000, 4001])
def test_a_convolution_of_more_than_2_to_31_elements(D):
    """Bit for bit: a token's sums do not depend on where it stands."""
    T, cut = 540000, 530000
    gen = torch.Generator("cuda").manual_seed(3)
    x, dy = (torch.randn(1, T, D, device="cuda", generator=gen, dtype=BF) for _ in range(2))
    w = torch.randn(D, 4, device="cuda", generator=gen)
    y, last = kda.kda_conv_fwd(x, w, activation="silu", output_final_state=True)
    dx = kda.kda_conv_bwd(dy, x, w, activation="silu")[0]
    state = x[:, cut - 3:cut].contiguous()
    ty, tl = kda.kda_conv_fwd(x[:, cut:], w, None, state, activation="silu", output_final_state=True)
    tx = kda.kda_conv_bwd(dy[:, cut:], x[:, cut:], w, None, state, activation="silu")[0]
    assert torch.equal(tl, last) and torch.equal(ty, y[:, cut:]) and torch.equal(tx, dx[:, cut:])


@pytest.mark.parametrize("N", [2048, 2045])
def test_a_product_of_more_than_2_to_31_elements(N):
    M, K = 1100000, 24
    gen = torch.Generator("cuda").manual_seed(2)
    x = torch.randn(M, K, device="cuda", generator=gen, dtype=BF)
    w, b = torch.randn(N, K, device="cuda", generator=gen, dtype=BF), torch.randn(N, device="cuda", generator=gen, dtype=BF)
    y, saved = kda.kda_linear_fwd(x, w, b, activation="silu", save=True)
    dx, _, _ = kda.kda_linear_bwd(y, x, w, saved, activation="silu", weight_grad=False, bias_grad=False)
    for rows in (slice(0, 200), slice(M // 2, M // 2 + 200), slice(M - 200, M)):
        part, _ = kda.kda_linear_fwd(x[rows], w, b, activation="silu")
        dpart = kda.kda_linear_bwd(y[rows], x[rows], w, saved[rows], activation="silu")[0]
        assert rel(part, y[rows]) <= 2 * tol(BF) and rel(dpart, dx[rows]) <= 2 * tol(BF)


# ---------------------------------------------------------------------------- streams and graphs
def jobs():
    c = cuda(make_conv(2, 150, 136, 4, BF, seed=3))
    s = cuda(make_scan(1, 260, 64, 16, 1, BF, seed=4))
    m, o = cuda(make_linear(150, 520, 136, BF, seed=5)), cuda(make_linear(33, 77, 45, HF, seed=6))
    few = cuda(make_linear(5, 4096, 136, BF, seed=7))
    return [lambda: all_conv(c), lambda: all_scan(s), lambda: all_linear(m), lambda: all_linear(o, "silu"),
            lambda: all_linear(few, "relu")]


def test_on_another_stream():
    """Inputs that the stream itself makes, and the same bits as on the current one."""
    c = cuda(make_conv(2, 150, 136, 4, BF, seed=3))
    s = cuda(make_scan(1, 260, 64, 16, 1, BF, seed=4))
    m = cuda(make_linear(150, 520, 136, BF, seed=5))
    ins, more = [s[n] for n in SCAN[:5]], [s[n] for n in SCAN[5:]]
    want = [kda.kda_conv_fwd(c["x"], c["weight"])[0], kda.kda_scan_fwd(*ins, *more)[0],
            kda.kda_linear_fwd(m["x"], m["weight"])[0]]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        big = torch.randn(1 << 26, device="cuda").sort()[0]  # keeps the stream busy
        x, u, a = c["x"] * 1, s["u"] * 1, m["x"] * 1
    got = [kda.kda_conv_fwd(x, c["weight"], stream=side)[0],
           kda.kda_scan_fwd(u, *ins[1:], *more, stream=side.cuda_stream)[0],
           kda.kda_linear_fwd(a, m["weight"], stream=side)[0]]
    side.synchronize()
    assert big.numel() and all(torch.equal(p, q) for p, q in zip(got, want))


def test_calls_side_by_side():
    """Each on a stream of its own, at once, several times: every call has its own workspace."""
    todo = jobs()
    want = [f() for f in todo]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in todo]
    got = []
    for _ in range(4):
        for f, st in zip(todo, streams):
            with torch.cuda.stream(st):
                got.append(f())
    torch.cuda.synchronize()
    for i, outs in enumerate(got):
        for p, q in zip(outs, want[i % len(todo)]):
            assert torch.equal(p, q), i


def test_in_graphs():
    """Captured forward and backward, two graphs alive at once and replayed in turn and side by side."""
    todo = jobs()
    want = [f() for f in todo]
    torch.cuda.synchronize()
    graphs = []
    for f in todo:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = f()
        graphs.append((g, outs))
    streams = [torch.cuda.Stream() for _ in todo]
    for _ in range(3):
        for g, outs in graphs:
            for t in outs:
                t.zero_()
        torch.cuda.synchronize()
        for (g, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for (_, outs), ref in zip(graphs, want):
            assert all(torch.equal(p, q) for p, q in zip(outs, ref))


def test_steps_in_a_graph_go_on_from_where_they_are():
    R, D, N = 3, 72, 16
    c, s = cuda(make_conv(1, R, D, 4, BF, seqs=R)), cuda(make_scan(1, R, D, N, 1, BF, seqs=R))
    ins = [s[n][0] if s[n].dim() > 2 else s[n] for n in SCAN[:5]]

    def step(cs, ss):
        u = kda.kda_conv_step(c["x"][0], cs, c["weight"], c["bias"], activation="silu")
        return kda.kda_scan_step(u, *ins[1:], ss, s["D"], s["z"][0], s["delta_bias"])

    a = (c["initial"].clone(), s["initial"].clone())
    want = [step(*a) for _ in range(4)]
    b = (c["initial"].clone(), s["initial"].clone())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = step(*b)
    for ref in want:
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_from_a_thread_that_has_called_nothing():
    """As autograd's are: such a thread has no current context yet."""
    todo, got = jobs(), {}
    want = [f() for f in todo]
    torch.cuda.synchronize()

    def work(i):
        got[i] = todo[i]()

    for i in range(len(todo)):
        t = threading.Thread(target=work, args=(i,))
        t.start()
        t.join()
    torch.cuda.synchronize()
    for i, outs in enumerate(want):
        assert all(torch.equal(p, q) for p, q in zip(got[i], outs)), i


# ---------------------------------------------------------------------------- the two ways in
def same(a, b):
    assert len(a) == len(b)
    for p, q in zip(a, b):
        assert (p is None and q is None) or torch.equal(p, q)


@pytest.mark.parametrize("lens", [None, [20, 0, 13]])
def test_both_ways_into_the_library_agree(lens):
    """The short way and the checked one give the same bits (they make the same call)."""
    p = None if lens is None else cu(lens, 5)
    x = cuda(make_conv(1, 50, 72, 4, BF, seed=1))
    same(kda.kda_conv_fwd(x["x"], x["weight"], x["bias"], activation="silu", output_final_state=True, cu_seqlens=p),
         conv._conv_fwd(x["x"], x["weight"], x["bias"], None, "silu", True, p, None))
    same(kda.kda_conv_bwd(x["dy"], x["x"], x["weight"], x["bias"], activation="silu", cu_seqlens=p),
         conv._conv_bwd(x["dy"], x["x"], x["weight"], x["bias"], None, None, "silu", False, p, None, True))
    s = cuda(make_scan(1, 50, 72, 16, 2, BF, seed=2))
    ins, more = [s[n] for n in SCAN[:5]], [s[n] for n in SCAN[5:]]
    a = kda.kda_scan_fwd(*ins, *more, save=True, cu_seqlens=p)
    b = scan._scan_fwd(*ins, *more, None, True, False, True, p, None)
    same(a[:2], b[:2])
    same(kda.kda_scan_bwd(s["dy"], *ins, a[2], *more, cu_seqlens=p),
         scan._scan_bwd(s["dy"], *ins, b[2], *more, None, True, False, p))


def test_both_ways_agree_for_products_and_single_tokens():
    for M in (4, 70):
        x = cuda(make_linear(M, 72, 40, BF, seed=M))
        a = kda.kda_linear_fwd(x["x"], x["weight"], x["bias"], x["residual"], activation="gelu", save=True)
        same(a, linear._linear_fwd(x["x"], x["weight"], x["bias"], x["residual"], "gelu", True, None))
        same(kda.kda_linear_bwd(x["dy"], x["x"], x["weight"], a[1], activation="gelu", input_grad=False),
             linear._linear_bwd(x["dy"], x["x"], x["weight"], a[1], "gelu", False, True, True, None))
    c, s = cuda(make_conv(1, 5, 72, 4, BF)), cuda(make_scan(1, 5, 72, 16, 1, BF, seqs=5))
    ca, cb = (torch.ones(5, 3, 72, dtype=BF, device="cuda") for _ in range(2))
    same([kda.kda_conv_step(c["x"][0], ca, c["weight"], activation="silu"), ca],
         [conv._conv_step(c["x"][0], cb, c["weight"], None, "silu", None, None), cb])
    ins = [s[n][0] if s[n].dim() > 2 else s[n] for n in SCAN[:5]]
    sa, sb = s["initial"].clone(), s["initial"].clone()
    same([kda.kda_scan_step(*ins, sa, s["D"], s["z"][0], s["delta_bias"]), sa],
         [scan._scan_step(*ins, sb, s["D"], s["z"][0], s["delta_bias"], True, None, None), sb])


def test_the_checks_name_what_is_wrong():
    x, s, m = (cuda(t) for t in (make_conv(2, 9, 8, 4), make_scan(2, 9, 8, 4, 2), make_linear(9, 16, 24)))
    ins = [s[n] for n in SCAN[:5]]
    saved = kda.kda_scan_fwd(*ins, save=True)[2]
    for match, call in (
            ("dtype", lambda: kda.kda_conv_fwd(x["x"], x["weight"], x["bias"].float())),
            ("float32", lambda: kda.kda_conv_fwd(x["x"], x["weight"].half())),
            ("W 2 to 4", lambda: kda.kda_conv_fwd(x["x"], torch.zeros(8, 5, device="cuda", dtype=BF))),
            ("activation", lambda: kda.kda_conv_fwd(x["x"], x["weight"], activation="gelu")),
            ("B must be 1", lambda: kda.kda_conv_fwd(x["x"], x["weight"], cu_seqlens=cu([3]))),
            ("initial_state", lambda: kda.kda_conv_fwd(x["x"], x["weight"], None, x["initial"][:1])),
            ("evenly spaced", lambda: kda.kda_conv_fwd(x["x"][:, ::2], x["weight"])),
            ("dy", lambda: kda.kda_conv_bwd(x["dy"][:, :8], x["x"], x["weight"])),
            ("contiguous", lambda: kda.kda_conv_step(x["x"][0], x["x"].new_zeros(9, 8, 3).mT, x["weight"])),
            ("state", lambda: kda.kda_conv_step(x["x"][0], x["initial"], x["weight"])),
            ("A must be", lambda: kda.kda_scan_fwd(*ins[:2], torch.zeros(8, 65, device="cuda"), *ins[3:])),
            ("A has dtype", lambda: kda.kda_scan_fwd(*ins[:2], s["A"].to(BF), *ins[3:])),
            ("groups", lambda: kda.kda_scan_fwd(*ins[:3], s["B"][:, :, :1].expand(2, 9, 3, 4), s["C"])),
            ("delta", lambda: kda.kda_scan_fwd(s["u"], s["delta"].float(), *ins[2:])),
            ("not from a forward", lambda: kda.kda_scan_bwd(s["dy"], *ins, saved[:-1])),
            ("state", lambda: kda.kda_scan_step(*(t[0] if t.dim() > 2 else t for t in ins), s["initial"])),
            ("bf16 or fp16", lambda: kda.kda_linear_fwd(m["x"].float(), m["weight"].float())),
            ("weight must be", lambda: kda.kda_linear_fwd(m["x"], m["weight"].T)),
            ("residual", lambda: kda.kda_linear_fwd(m["x"], m["weight"], None, m["residual"][:4])),
            ("bias", lambda: kda.kda_linear_fwd(m["x"], m["weight"], m["bias"].float())),
            ("saved is needed", lambda: kda.kda_linear_bwd(m["dy"], m["x"], m["weight"], activation="relu")),
            ("must not overlap", lambda: kda.kda_linear_fwd(m["x"][:1].expand(9, 16), m["weight"])),
            ("activation", lambda: kda.kda_linear_fwd(m["x"], m["weight"], activation="tanh"))):
        with pytest.raises(ValueError, match=match):
            call()
    for call in (lambda: kda.kda_conv_fwd(x["x"][:1, :1].expand(2, 9, 8), x["weight"]),
                 lambda: kda.kda_conv_bwd(x["dy"][:, :1].expand(2, 9, 8), x["x"], x["weight"]),
                 lambda: kda.kda_scan_fwd(*ins[:3], s["B"][:, :1].expand(2, 9, 2, 4), s["C"]),
                 lambda: kda.kda_linear_bwd(m["dy"][:1].expand(9, 24), m["x"], m["weight"])):
        with pytest.raises(ValueError, match="overlap|evenly spaced"):
            call()
    y = m["x"][:, :8]
    with pytest.raises(kda.KdaError):  # the output is the input's memory
        kda.kda_linear_fwd(m["x"], m["weight"][:8], y=y)


# ---------------------------------------------------------------------------- values
@pytest.mark.parametrize("M", [2, 40])
def test_activations_of_unusual_values(M):
    """pre = the bias alone: the limits at infinity, NaN stays NaN, and far tails in FP32's reach."""
    inf, nan = float("inf"), float("nan")
    v = torch.tensor([inf, nan, 3e38, 100.0, 13.0, 5.0, 0.0, -0.5, -5.0, -13.0, -100.0, -3e38], dtype=BF)
    x, w = torch.zeros(M, 8, dtype=BF, device="cuda"), torch.zeros(12, 8, dtype=BF, device="cuda")
    for act, f in (("silu", lambda t: t * torch.sigmoid(t)), ("relu", torch.relu),
                   ("gelu", lambda t: 0.5 * t * torch.erfc(-t * 0.5 ** 0.5))):
        y, saved = kda.kda_linear_fwd(x, w, v.cuda(), activation=act, save=True)
        want = f(v.double())
        want = torch.where(want.abs() < 2.0 ** -126, torch.zeros_like(want), want)
        for r in (0, M - 1):
            got = y[r].cpu().double()
            assert torch.isnan(got[1]) and got[0] == inf
            keep = [i for i in range(12) if i > 1]
            # a rounding to BF16, and the exponential's argument (some 85 in the tail) to FP32's: 85 * 2^-24
            # relative beside 7e-6
            assert ((got[keep] - want[keep]).abs() <= want[keep].abs() * (2.0 ** -8 + 2e-5) + 2.0 ** -120).all(), act
        same([saved[0][2:].cpu()], [v[2:]])
        dy = torch.ones(M, 12, dtype=BF, device="cuda")
        db = kda.kda_linear_bwd(dy, x, w, saved, activation=act, input_grad=False, weight_grad=False)[2].cpu().double()
        slopes = {"silu": lambda t: torch.sigmoid(t) * (1 + t * (1 - torch.sigmoid(t))),
                  "relu": lambda t: (t > 0).double(),
                  "gelu": lambda t: 0.5 * torch.erfc(-t * 0.5 ** 0.5) + t * torch.exp(-t * t / 2) / (2 * torch.pi) ** 0.5}
        ref = M * slopes[act](v.double())
        ok = [i for i in range(3, 11)]  # (beyond them the formula itself is 0 times infinity)
        assert ((db[ok] - ref[ok]).abs() <= ref[ok].abs() * 2.0 ** -7 + 1e-5 * M).all(), act


def test_nothing_passes_from_one_sequence_to_the_next():
    """NaN and infinities in one packed sequence, in its state and between the sequences stay there."""
    lens = [30, 40, 25]
    c = cuda(make_conv(1, 100, 16, 4, BF, seqs=3, seed=1))
    s = cuda(make_scan(1, 100, 16, 8, 1, BF, seqs=3, seed=2))
    p = cu(lens)
    conv_ref, scan_ref = all_conv(c, p, states=True), all_scan(s, p, states=True)
    for n in ("x", "dy"):
        c[n][:, 30:70], c[n][:, 95:] = float("nan"), float("inf")
    for n in ("u", "delta", "B", "C", "z", "dy"):
        s[n][:, 30:70], s[n][:, 95:] = float("nan"), float("inf")
    c["initial"][1], s["initial"][1], c["dfinal"][1], s["dfinal"][1] = (float("nan"),) * 4
    got, keep = all_conv(c, p, states=True), [*range(30), *range(70, 100)]
    for i in (0, 2):  # y, dx
        assert torch.equal(got[i][:, keep], conv_ref[i][:, keep])
    for i in (1, 5):  # the states and their gradients
        assert torch.equal(got[i][[0, 2]], conv_ref[i][[0, 2]])
    got = all_scan(s, p, states=True)
    for i in (0, 2, 3, 5, 6, 8):  # y, du, ddelta, dB, dC, dz
        assert torch.equal(got[i][:, keep], scan_ref[i][:, keep])
    for i in (1, 10):
        assert torch.equal(got[i][[0, 2]], scan_ref[i][[0, 2]])


# ---------------------------------------------------------------------------- differences
def slope_along(f, args, direction, h=1e-4):
    """d/de of f(args + e direction) by central differences in 64 bits: h^2 = 1e-8 relative."""
    up = f(*(a + h * d for a, d in zip(args, direction)))
    return float((up - f(*(a - h * d for a, d in zip(args, direction)))) / (2 * h))


def against_differences(value, inputs, grads, limit=1e-4):
    """Along a random direction of each input alone; the kernels' FP32 results leave some 1e-5 of the
    directional derivative's scale |gradient| |direction|."""
    gen = torch.Generator().manual_seed(8)
    for i, g in enumerate(grads):
        d = [torch.zeros_like(a) for a in inputs]
        d[i] = torch.randn(inputs[i].shape, generator=gen, dtype=F64)
        got = float((g.cpu().double() * d[i]).sum())
        assert abs(got - slope_along(value, inputs, d)) <= limit * float(g.double().norm().cpu() * d[i].norm())


def test_conv_gradients_against_differences():
    x = make_conv(2, 11, 6, 4, F32, seed=5)
    names = ("x", "weight", "bias", "initial")
    h = [x[n].to(F64) for n in names]
    c = cuda(x)
    dx, dw, db, di = kda.kda_conv_bwd(c["dy"], c["x"], c["weight"], c["bias"], c["initial"], c["dfinal"],
                                      activation="silu", output_d_initial_state=True)

    def value(*a):
        y, final = conv64(*a, "silu")
        return (y * x["dy"].to(F64)).sum() + (final * x["dfinal"].to(F64)).sum()

    against_differences(value, h, (dx, dw, db, di))


def test_scan_gradients_against_differences():
    x = make_scan(2, 19, 6, 5, 2, F32, seed=6)
    names = (*SCAN, "initial")
    h = [x[n].to(F64) for n in names]
    c = cuda(x)
    ins, more = [c[n] for n in SCAN[:5]], [c[n] for n in SCAN[5:]]
    saved = kda.kda_scan_fwd(*ins, *more, c["initial"], save=True)[2]
    grads = kda.kda_scan_bwd(c["dy"], *ins, saved, *more, c["dfinal"], output_d_initial_state=True)

    def value(*a):
        y, final = scan64(*a)
        return (y * x["dy"].to(F64)).sum() + (final * x["dfinal"].to(F64)).sum()

    against_differences(value, h, grads)


def test_linear_gradients_against_differences():
    x = make_linear(21, 24, 32, HF, seed=7)
    h = [x[n].to(F64) for n in ("x", "weight", "bias")]
    c = cuda(x)
    saved = kda.kda_linear_fwd(c["x"], c["weight"], c["bias"], activation="gelu", save=True)[1]
    grads = kda.kda_linear_bwd(c["dy"], c["x"], c["weight"], saved, activation="gelu")

    def value(a, w, b):
        pre = a @ w.T + b
        return (0.5 * pre * torch.erfc(-pre * 0.5 ** 0.5) * x["dy"].to(F64)).sum()

    # FP16 gradients: five roundings of 2^-11 at most, of components that the direction sums with random
    # signs; the scale |gradient| |direction| is what they are relative to
    against_differences(value, h, grads, 5 * 2.0 ** -11)
