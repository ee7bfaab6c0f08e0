"""CPU tests of the sizes that include/selective_scan.h names as its limits: those
just inside are accepted, those just outside refused.  Nothing is launched: an
accepted size is seen by the misaligned output that is refused after it."""
import ctypes
import os

import pytest

import chunked_linear_scan_amd as cls
from test_selective_abi import AT, ScanGrads, conv_in, library, scan_in

pytestmark = pytest.mark.skipif(not os.path.exists(cls.LIB_PATH),
                                reason="library not built (run __graft_entry__.build())")

SHAPE, ALIGN = -2, -5


# batch, seqlen, channels, states, groups
SCAN_SIZES = [((1024, 1, 16384, 16, 1), ALIGN), ((4096, 2, 5120, 16, 1), ALIGN), ((64, 1, 1024, 64, 1024), ALIGN),
              ((1024, 1, 5120, 64, 1), ALIGN),
              (((1 << 18) - 1, 1, 4096, 16, 1), ALIGN), ((1 << 18, 1, 4096, 16, 1), SHAPE),   # 2^32 threads
              (((1 << 20) - 1, 1, 1, 64, 1), ALIGN), (((1 << 22), 1, 1, 64, 1), SHAPE),
              ((1, 1, 16205264, 64, 1), ALIGN), ((1, 1, 16205265, 64, 1), SHAPE),           # dA's sums
              ((1, 1 << 30, 1024, 16, 1), ALIGN), ((1, 1 << 30, 1025, 16, 1), SHAPE),       # 2^40 values
              ((1, (1 << 30) + 1, 1, 16, 1), SHAPE), (((1 << 24) + 1, 1, 1, 1, 1), SHAPE),
              ((1, 1, (1 << 24) + 1, 1, 1), SHAPE)]


@pytest.mark.parametrize("size,status", SCAN_SIZES)
def test_scan_sizes(size, status):
    lib = library()
    s = scan_in(**dict(zip(("batch", "seqlen", "channels", "dstate", "ngroups"), size)))
    assert lib.selective_scan_fwd(ctypes.byref(s), AT + 1, AT, AT, AT, 1 << 60, None) == status
    g = ScanGrads(**{**{k: AT for k in ("dy", "checkpoints", "ddt", "dz", "dB", "dC", "dA")}, "du": AT + 1})
    assert lib.selective_scan_bwd(ctypes.byref(s), ctypes.byref(g), AT, 1 << 60, None) == status
    for f, args in ((lib.selective_scan_bwd_workspace_size, size), (lib.selective_scan_checkpoint_size, size[:4])):
        assert (f(*args) > 0) == (status == ALIGN)


# batch, channels, states, groups
STEP_SIZES = [((1024, 5120, 64, 1), ALIGN), ((64, 1024, 64, 1024), ALIGN), ((4096, 4096, 64, 4096), ALIGN),
              ((1 << 20, 1 << 12, 4, 1), SHAPE), (((1 << 20) - 1, 1 << 12, 4, 1), ALIGN),   # a sequence to a thread
              ((1 << 20, 1 << 12, 16, 1), SHAPE), (((1 << 20) - 4, 1 << 12, 16, 1), ALIGN),  # four
              ((1 << 18, 1 << 12, 64, 1), SHAPE), (((1 << 18) - 4, 1 << 12, 64, 1), ALIGN),
              ((1, (1 << 24) + 1, 4, 1), SHAPE), (((1 << 24) + 1, 1, 4, 1), SHAPE)]


@pytest.mark.parametrize("size,status", STEP_SIZES)
def test_step_sizes(size, status):
    lib = library()
    s = scan_in(**dict(zip(("batch", "channels", "dstate", "ngroups"), size)))
    assert lib.selective_scan_step(ctypes.byref(s), AT, AT + 1, None) == status


@pytest.mark.parametrize("n,at", [(16, AT + 4), (16, AT + 8), (3, AT + 2)])
def test_step_refuses_a_state_off_its_alignment(n, at):
    """16 bytes where rows are whole vectors, else that of an element."""
    s = scan_in(dstate=n)
    assert library().selective_scan_step(ctypes.byref(s), at, AT, None) == ALIGN


# batch, seqlen, channels
CONV_SIZES = [((1 << 24, 1 << 30, 1 << 24), SHAPE), ((1 << 20, 1 << 20, 1 << 20), SHAPE), ((64, 4096, 5120), ALIGN),
              (((1 << 24) - 4, 1, 64), ALIGN), ((1 << 24, 1, 64), SHAPE), ((1, (1 << 24) - 12, 960), ALIGN),
              ((1, (1 << 24) - 8, 960), SHAPE)]


@pytest.mark.parametrize("size,status", CONV_SIZES)
def test_conv_sizes(size, status):
    lib = library()
    s = conv_in(**dict(zip(("batch", "seqlen", "channels"), size)))
    assert lib.short_conv_fwd(ctypes.byref(s), AT + 1, AT, None) == status
    assert lib.short_conv_bwd(ctypes.byref(s), AT, 0, 0, None, AT + 1, AT, AT, AT, AT, 1 << 60, None) == status
    for width in (2, 4):
        assert (lib.short_conv_bwd_workspace_size(*size, width) > 0) == (status == ALIGN)
    assert lib.short_conv_bwd_workspace_size(*size, 1) == 0 and lib.short_conv_bwd_workspace_size(*size, 5) == 0


# batch, rows, states, slots
CACHE_SIZES = [((1, (1 << 26) - 257, 1, 1), ALIGN), ((1, (1 << 26) - 256, 1, 1), SHAPE),
               ((64, (1 << 20) - 257, 16, 64), ALIGN), ((64, (1 << 20) - 256, 16, 64), SHAPE),
               ((1, 1 << 15, 1, (1 << 31) - 1), ALIGN), ((1, 1 << 15, 1, 1 << 31), SHAPE),
               ((1, 1 << 16, 1, 1 << 30), ALIGN), ((1, (1 << 16) + 1, 1, 1 << 30), SHAPE)]


@pytest.mark.parametrize("size,status", CACHE_SIZES)
def test_cache_sizes(size, status):
    lib = library()
    assert lib.state_cache_write(AT + 2, AT, *size, 3, AT, AT, None) == status
    assert lib.state_cache_read(AT, AT + 2, AT, *size, 3, AT, None) == status


@pytest.mark.parametrize("status,words", [(SHAPE, ("channels", "stride")), (ALIGN, ("alignment",)), (-8, ("width", "state"))])
def test_error_texts_hold_for_every_call(status, words):
    text = cls.strerror(status)
    assert all(w in text for w in words) and "16" not in text
