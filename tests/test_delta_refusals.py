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
