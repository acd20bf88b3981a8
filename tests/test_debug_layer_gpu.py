"""The bounds-checked build's checks of the convolution, the scan and the matrix product are there: with
every extent one less (KDA_DBG_SHORT) each call reports, and leaves the last row or element of every
output as it was."""

import pytest
import torch

import gated_delta_rule_intra_gb300 as kda
from tests._layer import BF, F32, HF, SCAN, cu, cuda, make_conv, make_linear, make_scan

pytestmark = pytest.mark.gpu

STORE, LOAD, SHORT = 1, 2, 8


def short(call, want):
    """The call with every extent one less, its outputs made of memory that is all ones (NaN in each
    type); which of them are not None keep their last element."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    ones = [torch.full((size,), 255, dtype=torch.uint8, device="cuda")
            for size, n in ((1 << 19, 64), (1 << 16, 64), (1 << 13, 128), (1 << 9, 1024)) for _ in range(n)]
    del ones  # the outputs come from here, whatever their size
    word = torch.full((1,), SHORT, dtype=torch.int32, device="cuda")
    with kda.use_library(kda.DEBUG_LIB_PATH):
        kda.kda_debug_set_flags(word)
        try:
            outs = call()
            torch.cuda.synchronize()
        finally:
            kda.kda_debug_set_flags(None)
    assert word.item() == SHORT | want, hex(word.item())
    for i, t in enumerate(outs):
        assert t is None or torch.isnan(t.flatten()[-1].float()), i


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("B,T,D,W", [(2, 67, 264, 4), (3, 300, 77, 3), (1, 2, 6, 2)])
def test_the_convolution_reports(B, T, D, W, dtype):
    x = cuda(make_conv(B, T, D, W, dtype, seed=T))
    short(lambda: kda.kda_conv_fwd(x["x"], x["weight"], x["bias"], x["initial"], activation="silu",
                                   output_final_state=True), STORE | LOAD)
    short(lambda: kda.kda_conv_bwd(x["dy"], x["x"], x["weight"], x["bias"], x["initial"], x["dfinal"],
                                   activation="silu", output_d_initial_state=True), STORE | LOAD)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,D,N,G", [(2, 67, 64, 16, 1), (2, 33, 77, 5, 1), (1, 900, 64, 16, 2), (1, 40, 66, 64, 3)])
def test_the_scan_reports(B, T, D, N, G, dtype):
    x = cuda(make_scan(B, T, D, N, G, dtype, seed=T))
    ins, more = [x[n] for n in SCAN[:5]], [x[n] for n in SCAN[5:]]
    short(lambda: kda.kda_scan_fwd(*ins, *more, x["initial"], save=True, output_final_state=True)[:2], STORE | LOAD)
    saved = kda.kda_scan_fwd(*ins, *more, x["initial"], save=True)[2]
    short(lambda: kda.kda_scan_bwd(x["dy"], *ins, saved, *more, x["dfinal"], output_d_initial_state=True), STORE | LOAD)


def test_packed_sequences_report():
    p = cu([20, 0, 59], 11)
    x, s = cuda(make_conv(1, 90, 72, 4, BF, seqs=3)), cuda(make_scan(1, 90, 72, 16, 1, BF, seqs=3))
    ins, more = [s[n] for n in SCAN[:5]], [s[n] for n in SCAN[5:]]
    short(lambda: kda.kda_conv_fwd(x["x"], x["weight"], cu_seqlens=p)[:1], STORE | LOAD)
    short(lambda: kda.kda_scan_fwd(*ins, *more, cu_seqlens=p)[:1], STORE | LOAD)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,N,R", [(64, 16, 5), (33, 7, 3), (512, 16, 130)])
def test_single_tokens_report(D, N, R, dtype):
    c, s = cuda(make_conv(1, R, D, 4, dtype, seqs=R)), cuda(make_scan(1, R, D, N, 1, dtype, seqs=R))
    ins, more = [s[n][0] if s[n].dim() > 2 else s[n] for n in SCAN[:5]], [s["D"], s["z"][0], s["delta_bias"]]
    state = c["initial"].clone()
    short(lambda: [kda.kda_conv_step(c["x"][0], state, c["weight"], c["bias"])], STORE | LOAD)
    assert torch.equal(state[-1], c["initial"][-1])
    state = s["initial"].clone()
    short(lambda: [kda.kda_scan_step(*ins, state, *more)], STORE)
    assert torch.equal(state[-1, -1], s["initial"][-1, -1])


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("M,K,N", [
    (300, 520, 137),   # results by elements, the residual by words
    (130, 77, 133),    # x and the weight copied first
    (40, 4096, 63),    # the contraction cut into parts
    (5, 72, 40),       # few rows
    (16, 4096, 40),    # few rows of a long contraction
])
def test_the_product_reports(M, K, N, dtype):
    x = cuda(make_linear(M, K, N, dtype, seed=M))
    short(lambda: kda.kda_linear_fwd(x["x"], x["weight"], x["bias"], x["residual"], activation="silu", save=True),
          STORE | LOAD)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("M,K,N", [(300, 521, 136), (130, 77, 129), (4096, 63, 40)])
def test_the_products_gradients_report(M, K, N, dtype):
    """(K is odd: dx and dweight do not leave by tensor maps, which need no checks.)"""
    x = cuda(make_linear(M, K, N, dtype, seed=M))
    saved = kda.kda_linear_fwd(x["x"], x["weight"], x["bias"], activation="silu", save=True)[1]
    short(lambda: kda.kda_linear_bwd(x["dy"], x["x"], x["weight"], saved, activation="silu"), STORE | LOAD)
    short(lambda: kda.kda_linear_bwd(x["dy"], x["x"], x["weight"], saved, activation="silu", input_grad=False,
                                     bias_grad=False), STORE | LOAD)
    short(lambda: kda.kda_linear_bwd(x["dy"], x["x"], x["weight"], saved, activation="silu", input_grad=False,
                                     weight_grad=False)[2:], STORE | LOAD)
