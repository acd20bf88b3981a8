"""The recurrence's states, packed calls and workspaces, and layer norm, through the bounds-checked
debug build: no index outside its buffer, and the same results."""

import pytest
import torch

import gated_delta_rule_intra_gb300 as kda
from tests._recurrence import NAMES, cu, cuda, make, states
from tests.test_layer_norm_gpu import make as make_norm
from tests.test_recurrence_edges_gpu import _debug

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T,H,HV,lens", [(67, 2, 4, None), (33, 80, 160, None),
                                         (200, 2, 6, [63, 1, 0, 65, 71]),
                                         (193, 1, 1, [64, 64, 65])])
def test_states_and_their_gradients(T, H, HV, lens, dtype):
    x = cuda(make(T, H, HV, dtype=dtype, seed=T))
    a, c, n = [x[k] for k in NAMES], None if lens is None else cu(lens), len(lens or [0])
    S0, dS = states(n, HV).cuda(), states(n, HV, seed=2).cuda()

    def call():
        o, final, saved = kda.kda_chunk_fwd(*a, initial_state=S0, output_final_state=True,
                                            save=True, cu_seqlens=c)
        return (o, final, *kda.kda_chunk_bwd(*a, x["v"], saved, d_final_state=dS,
                                             output_d_initial_state=True, cu_seqlens=c))

    _debug(call)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("HV", [3, 8])
def test_tokens_in_no_sequence(HV, dtype):
    x = cuda(make(90, 1, HV, dtype=dtype, seed=7))
    a, c = [x[k] for k in NAMES], cu([20, 0, 45], start=11)

    def call():
        o, _, saved = kda.kda_chunk_fwd(*a, save=True, cu_seqlens=c)
        return (o, *kda.kda_chunk_bwd(*a, x["v"], saved, cu_seqlens=c)[:5])

    _debug(call)


@pytest.mark.parametrize("dtype", [BF, HF, torch.float32])
@pytest.mark.parametrize("rows,width,total", [(1, 8, 8), (37, 128, 128), (37, 129, 129),
                                              (700, 2048, 2048), (19, 200, 1000), (19, 77, 81),
                                              (5, 8192, 8192), (5, 9001, 9001)])
def test_layer_norm(rows, width, total, dtype):
    x, dy, w, b = (t.cuda() for t in make_norm(rows, total, dtype))
    x, dy, w, b = x[:, :width], dy[:, :width], w[:width].to(dtype), b[:width].to(dtype)
    y, dx = (torch.zeros(rows, total, dtype=dtype, device="cuda")[:, :width] for _ in range(2))

    def call():
        _, mean, rstd = kda.kda_layer_norm_fwd(x, w, b, y=y)
        _, dw, db = kda.kda_layer_norm_bwd(dy, x, w, mean, rstd, dx=dx)
        return y.clone(), mean, rstd, dx.clone(), dw, db

    _debug(call)
