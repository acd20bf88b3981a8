"""Choices of a caller (no call reaches CUDA): the size of `saved` chooses the kernels of a BF16 call
without a state, KDA_GATE_GRADS_FP32 the type of dgate and dbeta."""

import ctypes

import pytest

from gated_delta_rule_intra_gb300.recurrence import ChunkBwdOpts
from tests.test_ops_abi_host import (ERR_ALIGN, ERR_CUDA, ERR_DEVICE, ERR_OVERLAP,  # noqa: F401
                                     ERR_WORKSPACE, at, fwd, lib)


@pytest.mark.parametrize("cu,num_seqs", [(0, 0), (at(11), 2)])
def test_either_size_is_taken_without_a_state(lib, cu, num_seqs):  # noqa: F811
    import torch
    if torch.cuda.is_available():
        pytest.skip("these addresses exist nowhere: only where no device accepts the call")
    less, more = (lib.kda_chunk_saved_bytes(1, 64, 2, num_seqs, 0, s) for s in (0, 1))
    assert less < more
    kw = dict(saved=at(10), cu=cu, num_seqs=num_seqs)
    for size in (less, more):
        assert fwd(lib, saved_bytes=size, **kw) in (ERR_DEVICE, ERR_CUDA)
    assert fwd(lib, saved_bytes=more + 256, **kw) == ERR_WORKSPACE
    assert fwd(lib, saved_bytes=less, final=at(12), **kw) == ERR_WORKSPACE
    assert fwd(lib, saved_bytes=more, final=at(12), **kw) in (ERR_DEVICE, ERR_CUDA)


@pytest.mark.parametrize("flags", [2, 3])
def test_alignment_and_extent_of_fp32_gate_gradients(lib, flags):  # noqa: F811
    import torch
    if torch.cuda.is_available():
        pytest.skip("these addresses exist nowhere: only where no device accepts the call")
    saved = lib.kda_chunk_saved_bytes(1, 64, 2, 0, 0, 0)
    work = lib.kda_chunk_bwd_workspace_bytes(1, 64, 2, 2, 0, 0, saved)

    def bwd(zero_rest, **ptr):
        p = {n: at(i) for i, n in enumerate(("q", "k", "gate", "beta", "do", "dq", "dk", "dv",
                                             "dgate", "dbeta"))}
        p.update(ptr)
        op = ChunkBwdOpts(saved=at(12), saved_bytes=saved, workspace=at(13), workspace_bytes=work,
                          zero_rest=zero_rest)
        return lib.kda_chunk_bwd(*p.values(), 1, 64, 2, 0, ctypes.addressof(op), 0)

    good = (ERR_DEVICE, ERR_CUDA)
    assert bwd(0, dbeta=at(9, 2)) in good and bwd(flags, dbeta=at(9, 2)) == ERR_ALIGN
    assert bwd(flags, dbeta=at(9, 4)) in good
    size = 64 * 2 * 128 * 2  # of dgate in 16 bits; as many bytes again in fp32
    assert bwd(flags & 1, dv=at(8, size)) in good and bwd(flags, dv=at(8, size)) == ERR_OVERLAP
    assert bwd(flags, dv=at(8, 2 * size)) in good
