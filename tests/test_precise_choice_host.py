"""The size of `saved` chooses the kernels of a BF16 call without a state (no call reaches CUDA)."""

import pytest

from tests.test_ops_abi_host import (ERR_CUDA, ERR_DEVICE, ERR_WORKSPACE, at, fwd,  # noqa: F401
                                     lib)


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
