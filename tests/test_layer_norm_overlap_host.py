"""Which rows of layer norm's tensors count as overlapping (no call here reaches CUDA, except that
those in order meet the check of the device)."""

import pytest

from tests.test_ops_abi_host import (ERR_CUDA, ERR_DEVICE, ERR_OVERLAP, at, lib,  # noqa: F401
                                     norm_bwd, norm_fwd)

IN_ORDER = (ERR_DEVICE, ERR_CUDA)


@pytest.fixture(autouse=True)
def no_device():
    import torch
    if torch.cuda.is_available():
        pytest.skip("these addresses exist nowhere: only where no device accepts the call")


@pytest.mark.parametrize("off,good", [(20, True), (30, True), (76, True), (-20, True), (-30, True),
                                      (-74, True), (18, False), (32, False), (42, False),
                                      (0, False), (2, False), (60, False), (-18, False),
                                      (-42, False), (-60, False)])
def test_rows_between_rows(lib, off, good):  # noqa: F811
    """x: four rows of 20 bytes, 50 from one to the next; y the same, `off` bytes on."""
    rc = norm_fwd(lib, xs=25, ys=25, x=at(0, 1000), y=at(0, 1000 + off))
    assert rc in IN_ORDER if good else rc == ERR_OVERLAP


def test_strides_that_differ_are_taken_whole(lib):  # noqa: F811
    assert norm_fwd(lib, xs=25, ys=30, x=at(0), y=at(0, 20)) == ERR_OVERLAP
    assert norm_fwd(lib, xs=25, ys=30, x=at(0), y=at(0, 1000)) in IN_ORDER


def test_the_backward(lib):  # noqa: F811
    p = dict(dy=at(0), x=at(0, 20), dx=at(0, 40))
    assert norm_bwd(lib, strides=(30, 30, 30), **p) in IN_ORDER
    assert norm_bwd(lib, strides=(29, 29, 29), **p) == ERR_OVERLAP
    assert norm_bwd(lib, strides=(30, 30, 25), **p) == ERR_OVERLAP
