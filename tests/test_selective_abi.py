"""CPU tests of include/selective_scan.h: declared functions are exported, bad
arguments are refused on the host before any launch, sizes add up, and the
binding refuses tensors that do not fit."""
import ctypes
import os
import re

import pytest
import torch

import chunked_linear_scan_amd as cls

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "selective_scan.h")

pytestmark = pytest.mark.skipif(not os.path.exists(cls.LIB_PATH),
                                reason="library not built (run __graft_entry__.build())")

AT = 0x10000  # 16-byte aligned, never dereferenced on error paths
I64, I32, VP, SZ = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t


class ScanInputs(ctypes.Structure):
    """``selective_scan_inputs``."""
    _fields_ = ([(n, I64) for n in ("batch", "seqlen", "channels", "dstate", "ngroups")]
                + [("dtype", I32), ("softplus", I32)]
                + [(n, VP) for n in ("u", "dt", "z", "B", "C", "A", "D", "dt_bias", "h0", "seqlens")]
                + [(n, I64) for n in ("u_batch", "u_token", "dt_batch", "dt_token", "z_batch", "z_token",
                                      "B_batch", "B_token", "B_group", "C_batch", "C_token", "C_group")])


class ScanGrads(ctypes.Structure):
    """``selective_scan_grads``."""
    _fields_ = ([("dy", VP), ("dy_batch", I64), ("dy_token", I64)]
                + [(n, VP) for n in ("dh_final", "checkpoints", "du", "ddt", "dz", "dB", "dC", "dA", "dD",
                                     "ddt_bias", "dh0")])


class ConvInputs(ctypes.Structure):
    """``short_conv_inputs``."""
    _fields_ = ([(n, I64) for n in ("batch", "seqlen", "channels", "width")]
                + [("dtype", I32), ("silu", I32), ("x", VP), ("x_batch", I64), ("x_token", I64)]
                + [(n, VP) for n in ("weight", "bias", "initial_state", "seqlens")])


def library():
    lib = ctypes.CDLL(cls.LIB_PATH)
    for name, args, res in (
            ("selective_scan_workspace_size", [I64] * 5, SZ),
            ("selective_scan_bwd_workspace_size", [I64] * 5, SZ),
            ("selective_scan_checkpoint_size", [I64] * 4, SZ),
            ("selective_scan_fwd", [VP] * 5 + [SZ, VP], ctypes.c_int),
            ("selective_scan_bwd", [VP] * 3 + [SZ, VP], ctypes.c_int),
            ("selective_scan_step", [VP] * 4, ctypes.c_int),
            ("short_conv_fwd", [VP] * 4, ctypes.c_int),
            ("short_conv_bwd_workspace_size", [I64] * 4, SZ),
            ("short_conv_bwd", [VP, VP, I64, I64] + [VP] * 6 + [SZ, VP], ctypes.c_int),
            ("short_conv_step", [VP] * 4, ctypes.c_int),
            ("state_cache_write", [VP, VP] + [I64] * 4 + [ctypes.c_int] + [VP] * 3, ctypes.c_int),
            ("state_cache_read", [VP] * 3 + [I64] * 4 + [ctypes.c_int, VP, VP], ctypes.c_int)):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, res
    return lib


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b([a-z_][a-z0-9_]*)\s*\(", text))
    assert names == {"selective_scan_workspace_size", "selective_scan_bwd_workspace_size",
                     "selective_scan_checkpoint_size", "selective_scan_fwd", "selective_scan_bwd",
                     "selective_scan_step", "short_conv_fwd", "short_conv_bwd_workspace_size", "short_conv_bwd",
                     "short_conv_step", "state_cache_write", "state_cache_read"}
    lib = ctypes.CDLL(cls.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n


def test_structures_have_the_header_s_fields():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    for name, struct in (("selective_scan_inputs", ScanInputs), ("selective_scan_grads", ScanGrads),
                         ("short_conv_inputs", ConvInputs)):
        body = re.search(r"typedef struct \{([^}]*)\} %s;" % name, text).group(1)
        fields = [re.sub(r"\W", "", f.split()[-1]) for d in body.split(";") for f in d.split(",") if f.strip()]
        assert fields == [f for f, _ in struct._fields_], name


def scan_in(**k):
    a = dict(batch=2, seqlen=200, channels=64, dstate=16, ngroups=1, dtype=1, softplus=1, u=AT, dt=AT, z=AT, B=AT, C=AT,
             A=AT, D=AT, dt_bias=AT, h0=AT, seqlens=AT)
    a.update(k)
    return ScanInputs(**a)


BAD_SCAN = [(dict(u=None), -1), (dict(A=None), -1), (dict(B=None), -1), (dict(C=None), -1), (dict(dt=None), -1),
            (dict(dtype=3), -3), (dict(dtype=-1), -3), (dict(batch=0), -2), (dict(channels=0), -2),
            (dict(dstate=0), -2), (dict(dstate=65), -8), (dict(ngroups=3), -2), (dict(ngroups=0), -2),
            (dict(u=AT + 1), -5), (dict(z=AT + 1), -5), (dict(A=AT + 2), -5), (dict(u_batch=-1), -2),
            (dict(batch=1 << 40), -2), (dict(channels=1 << 30), -2), (dict(batch=1 << 20, channels=1 << 20), -2)]
BAD_LENGTH = [(dict(seqlen=0), -2), (dict(seqlen=1 << 31), -2), (dict(seqlens=AT + 2), -5), (dict(h0=AT + 1), -5)]


@pytest.mark.parametrize("bad,status", BAD_SCAN + BAD_LENGTH)
def test_scan_refuses(bad, status):
    lib, s = library(), scan_in(**bad)
    assert lib.selective_scan_fwd(ctypes.byref(s), AT, AT, AT, AT, 1 << 50, None) == status
    g = ScanGrads(**{k: AT for k in ("dy", "checkpoints", "du", "ddt", "dz", "dB", "dC", "dA")})
    assert lib.selective_scan_bwd(ctypes.byref(s), ctypes.byref(g), AT, 1 << 50, None) == status


@pytest.mark.parametrize("bad,status", BAD_SCAN)
def test_step_refuses(bad, status):
    lib, s = library(), scan_in(**bad)
    assert lib.selective_scan_step(ctypes.byref(s), AT, AT, None) == status


def test_scan_refuses_other_pointers():
    lib, s = library(), scan_in()
    ref = ctypes.byref(s)
    big = 1 << 50
    assert lib.selective_scan_fwd(None, AT, AT, AT, AT, big, None) == -1
    assert lib.selective_scan_fwd(ref, None, AT, AT, AT, big, None) == -1
    assert lib.selective_scan_fwd(ref, AT + 1, AT, AT, AT, big, None) == -5
    assert lib.selective_scan_fwd(ref, AT, AT + 2, AT, AT, big, None) == -5
    assert lib.selective_scan_fwd(ref, AT, AT, AT + 4, AT, big, None) == -5
    need = lib.selective_scan_workspace_size(2, 200, 64, 16, 1)
    assert need > 0  # 2 x 64 channels are cut into segments
    assert lib.selective_scan_fwd(ref, AT, AT, AT, AT, need - 1, None) == -6
    assert lib.selective_scan_fwd(ref, AT, AT, AT, None, big, None) == -6
    assert lib.selective_scan_step(ref, None, AT, None) == -1
    assert lib.selective_scan_step(ref, AT, None, None) == -1
    assert lib.selective_scan_step(ref, AT + 8, AT, None) == -5
    full = {k: AT for k in ("dy", "checkpoints", "du", "ddt", "dz", "dB", "dC", "dA")}
    for k in full:
        g = ScanGrads(**{**full, k: None})
        assert lib.selective_scan_bwd(ref, ctypes.byref(g), AT, big, None) == -1, k
    g = ScanGrads(**full)
    need = lib.selective_scan_bwd_workspace_size(2, 200, 64, 16, 1)
    assert lib.selective_scan_bwd(ref, ctypes.byref(g), AT, need - 1, None) == -6
    assert lib.selective_scan_bwd(ref, ctypes.byref(g), None, big, None) == -1
    g = ScanGrads(**full, dy_token=-4)
    assert lib.selective_scan_bwd(ref, ctypes.byref(g), AT, big, None) == -2


def test_scan_sizes():
    lib = library()
    # the state before every 8th token
    assert lib.selective_scan_checkpoint_size(2, 33, 10, 16) == 2 * 5 * 10 * 16 * 4
    assert lib.selective_scan_checkpoint_size(2, 33, 10, 33) == 2 * 5 * 10 * 33 * 4
    assert lib.selective_scan_checkpoint_size(2, 33, 10, 65) == 0
    assert lib.selective_scan_workspace_size(64, 4096, 4096, 16, 1) == 0  # whole sequences fill the device
    assert lib.selective_scan_workspace_size(1, 0, 64, 16, 1) == 0


def conv_in(**k):
    a = dict(batch=2, seqlen=100, channels=64, width=4, dtype=1, silu=1, x=AT, x_batch=6400, x_token=64, weight=AT,
             bias=AT, initial_state=AT, seqlens=AT)
    a.update(k)
    return ConvInputs(**a)


@pytest.mark.parametrize("bad,status", [(dict(x=None), -1), (dict(weight=None), -1), (dict(dtype=4), -3),
                                        (dict(batch=0), -2), (dict(channels=-1), -2), (dict(width=1), -8),
                                        (dict(width=5), -8), (dict(x=AT + 1), -5), (dict(weight=AT + 2), -5),
                                        (dict(x_batch=-1), -2), (dict(batch=1 << 22, channels=1 << 22), -2)])
def test_conv_refuses(bad, status):
    lib, s = library(), conv_in(**bad)
    ref, big = ctypes.byref(s), 1 << 50
    assert lib.short_conv_fwd(ref, AT, AT, None) == status
    assert lib.short_conv_step(ref, AT, AT, None) == status
    assert lib.short_conv_bwd(ref, AT, 0, 0, None, AT, AT, AT, AT, AT, big, None) == status


def test_conv_refuses_other_pointers():
    lib, s = library(), conv_in()
    ref, big = ctypes.byref(s), 1 << 50
    assert lib.short_conv_fwd(ref, None, AT, None) == -1
    assert lib.short_conv_fwd(ref, AT, AT + 1, None) == -5
    assert lib.short_conv_step(ref, None, AT, None) == -1
    assert lib.short_conv_bwd(ref, None, 0, 0, None, AT, AT, AT, AT, AT, big, None) == -1
    assert lib.short_conv_bwd(ref, AT, 0, 0, None, None, AT, AT, AT, AT, big, None) == -1
    assert lib.short_conv_bwd(ref, AT, -1, 0, None, AT, AT, AT, AT, AT, big, None) == -2
    need = lib.short_conv_bwd_workspace_size(2, 100, 64, 4)
    assert lib.short_conv_bwd(ref, AT, 0, 0, None, AT, AT, AT, AT, AT, need - 1, None) == -6
    zero = conv_in(seqlen=0)
    assert lib.short_conv_fwd(ctypes.byref(zero), AT, AT, None) == -2


@pytest.mark.parametrize("args,status", [((2, 8, 16, 4, 3), 0), ((0, 8, 16, 4, 3), -2), ((2, 0, 16, 4, 3), -2),
                                         ((2, 8, 0, 4, 3), -2), ((2, 8, 257, 4, 3), -8), ((2, 8, 16, 0, 3), -2),
                                         ((2, 8, 16, 4, 1), -3), ((2, 1 << 33, 16, 4, 4), -2),
                                         ((1 << 20, 1 << 20, 16, 4, 4), -2)])
def test_cache_refuses(args, status):
    lib = library()
    if status == 0:  # the sizes are fine, the pointers are not
        for k in range(4):
            p = [AT] * 4
            p[k] = None
            assert lib.state_cache_write(p[0], p[1], *args, p[2], p[3], None) == -1
            assert lib.state_cache_read(p[2], p[3], p[1], *args, p[0], None) == -1
        assert lib.state_cache_write(AT + 2, AT, *args, AT, AT, None) == -5
        assert lib.state_cache_read(AT, AT + 1, AT, *args, AT, None) == -5
        return
    assert lib.state_cache_write(AT, AT, *args, AT, AT, None) == status
    assert lib.state_cache_read(AT, AT, AT, *args, AT, None) == status


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(2, 5, 8)
    A = torch.zeros(8, 4)
    B = torch.zeros(2, 5, 1, 4)
    with pytest.raises(ValueError, match="GPU"):
        cls.selective_scan(x, x, A, B, B)
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        cls.selective_scan(x.double(), x, A, B, B)
    with pytest.raises(ValueError, match="batch, seqlen, channels"):
        cls.selective_scan(x[0], x, A, B, B)
    with pytest.raises(ValueError, match="GPU"):
        cls.short_conv(x, torch.zeros(8, 4))
    with pytest.raises(TypeError, match="int8 or float8_e4m3fn"):
        cls.state_cache_write(x, x, x, x)
    with pytest.raises(ValueError, match="GPU"):
        cls.state_cache_read(torch.zeros(3, 8, 4, dtype=torch.int8), torch.zeros(3, 8), torch.zeros(2))
