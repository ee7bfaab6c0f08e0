"""CPU tests of what the entry points of include/gated_delta.h refuse, and under which name."""
import ctypes
import os

import pytest
import torch

import chunked_linear_scan_amd as cls

pytestmark = pytest.mark.skipif(not os.path.exists(cls.LIB_PATH),
                                reason="library not built (run __graft_entry__.build())")


def test_residual_norm_bwd_names_the_gradient():
    """The tensor that the others are held to is dy here, and what is wrong with it is said of dy."""
    r, rstd = torch.zeros(3, 8), torch.zeros(3)
    with pytest.raises(ValueError, match=r"^dy must be on a GPU"):
        cls.residual_norm_bwd(torch.zeros(3, 8), r, None, rstd)
    with pytest.raises(TypeError, match=r"^dy must be float32, bfloat16 or float16"):
        cls.residual_norm_bwd(torch.zeros(3, 8, dtype=torch.int32), r, None, rstd)
    with pytest.raises(ValueError, match=r"^dy must be \[\.\.\., dim\]"):
        cls.residual_norm_bwd(torch.zeros(()), r, None, rstd)
    with pytest.raises(ValueError, match=r"^x must be on a GPU"):
        cls.residual_norm(torch.zeros(3, 8))


def step_status(**sizes):
    """What gated_delta_step says of sizes; y is off its alignment, which is refused after them."""
    from test_delta_abi import AT, delta_in, library
    s = delta_in(**{**dict(seqlen=1, kheads=1, dtype=1), **sizes})
    return library().gated_delta_step(ctypes.byref(s), AT, AT + 1, None)


@pytest.mark.parametrize("dk,rows", [(32, 128), (64, 64), (128, 32), (256, 16), (100, 32), (1, 128)])
def test_step_refuses_what_its_own_launch_cannot_hold(dk, rows):
    """A workgroup of 256 threads takes `rows` rows of a state once there are many: below 2^24 workgroups are launched
    (the state of 2^14 sequences of 64 heads of 256 by 64 is 64 GiB, which the device holds)."""
    align, shape = -5, -2
    assert step_status(batch=1 << 14, heads=64, dk=dk, dv=256) == (align if 256 // rows << 20 < 1 << 24 else shape)
    assert step_status(batch=(1 << 18) - 1, heads=64, dk=dk, dv=rows) == align
    assert step_status(batch=1 << 18, heads=64, dk=dk, dv=rows) == shape
    assert step_status(batch=1 << 17, heads=64, dk=dk, dv=rows + 1) == shape
    assert step_status(batch=1 << 17, heads=64, dk=dk, dv=rows) == align
