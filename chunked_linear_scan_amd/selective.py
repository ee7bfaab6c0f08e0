"""Python binding of ``include/selective_scan.h``: the selective scan, the
short convolution in front of it, and the 8-bit cache of states.

Argument marshalling only, as in the rest of the package: tensors are checked
for device, dtype and shape, outputs and workspaces are allocated with torch,
and the library's kernels run on torch's current stream of the inputs' device.
Activations may be slices of wider rows (their last dimension adjacent);
parameters and states are contiguous.  Each call has a workspace of its own
from torch's allocator, so calls on several streams and captured graphs share
none.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

_i64, _i32, _vp, _sz = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t
_CODE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_CACHE_CODE = {torch.int8: 3, torch.float8_e4m3fn: 4}

# The header's structures, packed in one go: filling the ctypes fields one by
# one takes longer than the smallest kernels.
_PACK_SCAN = struct.Struct("5q2i10P12q")
_PACK_GRADS = struct.Struct("P2q11P")
_PACK_CONV = struct.Struct("4q2iP2q4P")


class _ScanInputs(ctypes.Structure):
    """``selective_scan_inputs``."""
    _fields_ = ([(n, _i64) for n in ("batch", "seqlen", "channels", "dstate", "ngroups")]
                + [("dtype", _i32), ("softplus", _i32)]
                + [(n, _vp) for n in ("u", "dt", "z", "B", "C", "A", "D", "dt_bias", "h0", "seqlens")]
                + [(n, _i64) for n in ("u_batch", "u_token", "dt_batch", "dt_token", "z_batch", "z_token",
                                       "B_batch", "B_token", "B_group", "C_batch", "C_token", "C_group")])


class _ScanGrads(ctypes.Structure):
    """``selective_scan_grads``."""
    _fields_ = ([("dy", _vp), ("dy_batch", _i64), ("dy_token", _i64)]
                + [(n, _vp) for n in ("dh_final", "checkpoints", "du", "ddt", "dz", "dB", "dC", "dA", "dD",
                                      "ddt_bias", "dh0")])


class _ConvInputs(ctypes.Structure):
    """``short_conv_inputs``."""
    _fields_ = ([(n, _i64) for n in ("batch", "seqlen", "channels", "width")]
                + [("dtype", _i32), ("silu", _i32), ("x", _vp), ("x_batch", _i64), ("x_token", _i64)]
                + [(n, _vp) for n in ("weight", "bias", "initial_state", "seqlens")])


def declare(lib: ctypes.CDLL) -> None:
    """Sets the argument types of this header's functions."""
    ps = pg = pc = _vp  # packed bytes, or a reference to the structure
    for name, args, res in (
            ("selective_scan_workspace_size", [_i64] * 5, _sz),
            ("selective_scan_bwd_workspace_size", [_i64] * 5, _sz),
            ("selective_scan_checkpoint_size", [_i64] * 4, _sz),
            ("selective_scan_fwd", [ps, _vp, _vp, _vp, _vp, _sz, _vp], ctypes.c_int),
            ("selective_scan_bwd", [ps, pg, _vp, _sz, _vp], ctypes.c_int),
            ("selective_scan_step", [ps, _vp, _vp, _vp], ctypes.c_int),
            ("short_conv_fwd", [pc, _vp, _vp, _vp], ctypes.c_int),
            ("short_conv_bwd_workspace_size", [_i64] * 4, _sz),
            ("short_conv_bwd", [pc, _vp, _i64, _i64] + [_vp] * 6 + [_sz, _vp], ctypes.c_int),
            ("short_conv_step", [pc, _vp, _vp, _vp], ctypes.c_int),
            ("state_cache_write", [_vp, _vp] + [_i64] * 4 + [ctypes.c_int, _vp, _vp, _vp], ctypes.c_int),
            ("state_cache_read", [_vp, _vp, _vp] + [_i64] * 4 + [ctypes.c_int, _vp, _vp], ctypes.c_int)):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, res


_library = None


def _lib():
    global _library
    if _library is None:
        from . import load_library
        _library = load_library()
    return _library


def _at(t) -> int:
    return 0 if t is None else t.data_ptr()


def _run(what, device, f, *args) -> None:
    """Calls f on the device's current stream, with the device current."""
    at = device.index
    stream = torch._C._cuda_getCurrentRawStream(at)
    if at == torch._C._cuda_getDevice():
        status = f(*args, stream)
    else:
        with torch.cuda.device(device):
            status = f(*args, stream)
    if status != 0:
        from . import SSDError
        raise SSDError(status, what)


# Outputs: the forms of torch.empty that take the least time to call.
_DENSE = torch.contiguous_format


def _like(t):
    return torch.empty_like(t, memory_format=_DENSE)


def _check(name, t, at, dtype, shape, strided=False):
    """t is on GPU number `at` with this dtype and shape, contiguous or (strided) its last dimension adjacent."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == at and (
                t.is_contiguous() or (strided and (t.stride(-1) == 1 or t.shape[-1] == 1))):
            return
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    if t.get_device() != at:
        raise ValueError(f"{name} must be on one GPU with the other tensors (got {t.device})")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    raise ValueError(f"{name}'s last dimension must be adjacent in memory" if strided else f"{name} must be contiguous")


def _activation(name, t, dims):
    """The GPU's number, the dtype and the shape of the tensor that the others are held to."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    kind, shape = t.dtype, t.shape
    if kind not in _CODE:
        raise TypeError(f"{name} must be float32, bfloat16 or float16")
    if len(shape) != len(dims):
        raise ValueError(f"{name} must be [{', '.join(dims)}]")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU (got {t.device})")
    if not (t.is_contiguous() or t.stride(-1) == 1 or shape[-1] == 1):
        raise ValueError(f"{name}'s last dimension must be adjacent in memory")
    return t.get_device(), kind, shape


def _last_dim(name, t, dims):
    if not isinstance(t, torch.Tensor) or t.dim() != len(dims):
        raise ValueError(f"{name} must be [{', '.join(dims)}]")
    return t.shape[-1]


def _seqlens(t, at, batch):
    if t is not None:
        _check("seqlens", t, at, torch.int32, (batch,))


# ---------------------------------------------------------------------------
# selective scan
# ---------------------------------------------------------------------------
_SEQ, _ONE = ("batch", "seqlen", "channels"), ("batch", "channels")


def _scan_inputs(u, dt, A, B, C, D, z, dt_bias, h0, seqlens, dt_softplus, step=False):
    """(the packed structure, its sizes)"""
    at, kind, shape = _activation("u", u, _ONE if step else _SEQ)
    n, ch = shape[0], shape[-1]
    _check("dt", dt, at, kind, shape, True)
    if z is not None:
        _check("z", z, at, kind, shape, True)
    N = _last_dim("A", A, ("channels", "dstate"))
    _check("A", A, at, torch.float32, (ch, N))
    _last_dim("B", B, ("batch", "ngroups", "dstate") if step else ("batch", "seqlen", "ngroups", "dstate"))
    G = B.shape[-2]
    bc = (n, G, N) if step else (n, shape[1], G, N)
    _check("B", B, at, kind, bc, True)
    _check("C", C, at, kind, bc, True)
    if D is not None:
        _check("D", D, at, torch.float32, (ch,))
    if dt_bias is not None:
        _check("dt_bias", dt_bias, at, torch.float32, (ch,))
    if h0 is not None:
        _check("h0", h0, at, torch.float32, (n, ch, N))
    _seqlens(seqlens, at, n)
    L = 1 if step else shape[1]
    us, ds, bs, cs = u.stride(), dt.stride(), B.stride(), C.stride()
    zs = us if z is None else z.stride()
    if step:
        strides = (us[0], 0, ds[0], 0, zs[0], 0, bs[0], 0, bs[1], cs[0], 0, cs[1])
    else:
        strides = (us[0], us[1], ds[0], ds[1], zs[0], zs[1], bs[0], bs[1], bs[2], cs[0], cs[1], cs[2])
    return _PACK_SCAN.pack(n, L, ch, N, G, _CODE[kind], 1 if dt_softplus else 0, u.data_ptr(), dt.data_ptr(), _at(z),
                           B.data_ptr(), C.data_ptr(), A.data_ptr(), _at(D), _at(dt_bias), _at(h0), _at(seqlens),
                           *strides), (n, L, ch, N, G)


def _checkpoint_shape(lib, sizes):
    n, L, ch, N, _ = sizes
    return (n, lib.selective_scan_checkpoint_size(n, L, ch, N) // max(4 * n * ch * N, 1), N, ch)


def selective_scan(u, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, seqlens=None, dt_softplus: bool = True,
                   want_final_state: bool = True, want_checkpoints: bool = False, out: torch.Tensor | None = None):
    """Selective scan over whole sequences.  With dt' = softplus(dt + dt_bias):

        h_t = exp(dt'_t A) h_{t-1} + dt'_t B_t u_t,   y_t = (C_t . h_t + D u_t) silu(z_t)

    for each channel, with a decay for each of its states.  u, dt and z
    (optional) [Bt, L, channels] and B, C [Bt, L, groups, N] in fp32, bf16 or
    fp16 (one dtype; slices of wider rows are fine); A [channels, N], D and
    dt_bias [channels] and h0 [Bt, channels, N] in fp32 (the last three
    optional); N is at most 64.  seqlens (int32 [Bt], on the GPU): tokens at
    or past a sequence's length are padding; their y is zero.

    Returns (y, h_final or None), and with want_checkpoints
    (y, h_final or None, checkpoints), where checkpoints is what
    ``selective_scan_bwd`` takes."""
    lib = _lib()
    s, sizes = _scan_inputs(u, dt, A, B, C, D, z, dt_bias, h0, seqlens, dt_softplus)
    n, _, ch, N, _ = sizes
    dev, f32 = u.device, torch.float32
    if out is None:
        y = _like(u)
    else:
        y = out
        _check("out", y, dev.index, u.dtype, u.shape)
    hf = torch.empty(n, ch, N, dtype=f32, device=dev) if want_final_state else None
    kept = torch.empty(*_checkpoint_shape(lib, sizes), dtype=f32, device=dev) if want_checkpoints else None
    need = lib.selective_scan_workspace_size(*sizes)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _run("selective_scan", dev, lib.selective_scan_fwd, s, y.data_ptr(), _at(hf), _at(kept), _at(ws), need)
    return (y, hf, kept) if want_checkpoints else (y, hf)


def selective_scan_bwd(dy, u, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, seqlens=None,
                       dt_softplus: bool = True, checkpoints: torch.Tensor | None = None, dh_final=None) -> dict:
    """Gradients of ``selective_scan``'s inputs from the gradient dy of its y
    (and dh_final of its h_final), with the checkpoints of the forward pass
    over the same inputs.  Returns a dict of "du", "ddt", "dB", "dC" (and
    "dz") in u's dtype and "dA" (and "dD", "ddt_bias", "dh0") in fp32; those
    in parentheses where the input was given.  dB and dC are summed over the
    channels of a group.  Padding has zero gradients."""
    lib = _lib()
    s, sizes = _scan_inputs(u, dt, A, B, C, D, z, dt_bias, h0, seqlens, dt_softplus)
    n, _, ch, N, _ = sizes
    dev, f32 = u.device, torch.float32
    _check("dy", dy, dev.index, u.dtype, u.shape, True)
    if checkpoints is None:
        raise ValueError("checkpoints: run selective_scan with want_checkpoints=True")
    _check("checkpoints", checkpoints, dev.index, f32, _checkpoint_shape(lib, sizes))
    if dh_final is not None:
        _check("dh_final", dh_final, dev.index, f32, (n, ch, N))
    got = {"du": _like(u), "ddt": _like(u), "dA": _like(A), "dB": _like(B), "dC": _like(C)}
    if D is not None:
        got["dD"] = _like(D)
    if z is not None:
        got["dz"] = _like(u)
    if dt_bias is not None:
        got["ddt_bias"] = _like(dt_bias)
    if h0 is not None:
        got["dh0"] = _like(h0)
    g = _PACK_GRADS.pack(dy.data_ptr(), dy.stride(0), dy.stride(1), _at(dh_final), checkpoints.data_ptr(),
                         *(_at(got.get(k)) for k in ("du", "ddt", "dz", "dB", "dC", "dA", "dD", "ddt_bias", "dh0")))
    need = max(lib.selective_scan_bwd_workspace_size(*sizes), 16)
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    _run("selective_scan_bwd", dev, lib.selective_scan_bwd, s, g, ws.data_ptr(), need)
    return got


def selective_scan_step(h, u, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus: bool = True,
                        out: torch.Tensor | None = None):
    """One token of ``selective_scan`` for every sequence: updates the state h
    [Bt, channels, N] (fp32) in place and returns y [Bt, channels].  u, dt and
    z [Bt, channels], B and C [Bt, groups, N]; the rest as there."""
    lib = _lib()
    s, (n, _, ch, N, _) = _scan_inputs(u, dt, A, B, C, D, z, dt_bias, None, None, dt_softplus, True)
    dev = u.device
    _check("h", h, dev.index, torch.float32, (n, ch, N))
    if out is None:
        y = _like(u)
    else:
        y = out
        _check("out", y, dev.index, u.dtype, u.shape)
    _run("selective_scan_step", dev, lib.selective_scan_step, s, h.data_ptr(), y.data_ptr())
    return y


# ---------------------------------------------------------------------------
# short convolution
# ---------------------------------------------------------------------------
def _conv_inputs(x, weight, bias, initial_state, seqlens, silu, step=False):
    """(the packed structure, its sizes)"""
    at, kind, shape = _activation("x", x, _ONE if step else _SEQ)
    n, ch = shape[0], shape[-1]
    W = _last_dim("weight", weight, ("channels", "width"))
    _check("weight", weight, at, torch.float32, (ch, W))
    if bias is not None:
        _check("bias", bias, at, torch.float32, (ch,))
    if initial_state is not None:
        _check("initial_state", initial_state, at, kind, (n, W - 1, ch))
    _seqlens(seqlens, at, n)
    L, xs = (1, x.stride()) if step else (shape[1], x.stride())
    return _PACK_CONV.pack(n, L, ch, W, _CODE[kind], 1 if silu else 0, x.data_ptr(), xs[0], 0 if step else xs[1],
                           weight.data_ptr(), _at(bias), _at(initial_state), _at(seqlens)), (n, L, ch, W)


def short_conv(x, weight, bias=None, initial_state=None, seqlens=None, silu: bool = True,
               want_final_state: bool = True, out: torch.Tensor | None = None):
    """Causal convolution of each channel over its last `width` tokens, with
    the activation silu (or none): x [Bt, L, channels] in fp32, bf16 or fp16
    (slices of wider rows are fine), weight [channels, width] with width 2 to
    4 and bias [channels] in fp32.  initial_state [Bt, width - 1, channels]
    holds the inputs before the first token (oldest first; zeros without), and
    the final state the last ones.  seqlens as in ``selective_scan``.  Returns
    (y, final_state or None)."""
    lib = _lib()
    s, (n, _, ch, W) = _conv_inputs(x, weight, bias, initial_state, seqlens, silu)
    dev = x.device
    if out is None:
        y = _like(x)
    else:
        y = out
        _check("out", y, dev.index, x.dtype, x.shape)
    last = torch.empty(n, W - 1, ch, dtype=x.dtype, device=dev) if want_final_state else None
    _run("short_conv", dev, lib.short_conv_fwd, s, y.data_ptr(), _at(last))
    return y, last


def short_conv_bwd(dy, x, weight, bias=None, initial_state=None, seqlens=None, silu: bool = True,
                   dfinal_state=None) -> dict:
    """Gradients of ``short_conv``'s inputs from the gradient dy of its y (and
    dfinal_state of its final state): a dict of "dx" in x's dtype, "dweight"
    in fp32, and "dbias" (fp32) and "dinitial_state" where those were given."""
    lib = _lib()
    s, sizes = _conv_inputs(x, weight, bias, initial_state, seqlens, silu)
    n, _, ch, W = sizes
    dev = x.device
    _check("dy", dy, dev.index, x.dtype, x.shape, True)
    if dfinal_state is not None:
        _check("dfinal_state", dfinal_state, dev.index, x.dtype, (n, W - 1, ch))
    got = {"dx": _like(x), "dweight": _like(weight)}
    if bias is not None:
        got["dbias"] = _like(bias)
    if initial_state is not None:
        got["dinitial_state"] = _like(initial_state)
    need = max(lib.short_conv_bwd_workspace_size(*sizes), 16)
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    _run("short_conv_bwd", dev, lib.short_conv_bwd, s, dy.data_ptr(), dy.stride(0), dy.stride(1), _at(dfinal_state),
         got["dx"].data_ptr(), got["dweight"].data_ptr(), _at(got.get("dbias")), _at(got.get("dinitial_state")),
         ws.data_ptr(), need)
    return got


def short_conv_step(state, x, weight, bias=None, silu: bool = True, out: torch.Tensor | None = None):
    """One token of ``short_conv`` for every sequence: state
    [Bt, width - 1, channels] (x's dtype) takes x [Bt, channels] in and drops
    its oldest row, in place; returns y [Bt, channels]."""
    lib = _lib()
    s, (n, _, ch, W) = _conv_inputs(x, weight, bias, None, None, silu, True)
    dev = x.device
    _check("state", state, dev.index, x.dtype, (n, W - 1, ch))
    if out is None:
        y = _like(x)
    else:
        y = out
        _check("out", y, dev.index, x.dtype, x.shape)
    _run("short_conv_step", dev, lib.short_conv_step, s, state.data_ptr(), y.data_ptr())
    return y


# ---------------------------------------------------------------------------
# 8-bit cache of states
# ---------------------------------------------------------------------------
def _cache_args(cache, scales, slots):
    if not isinstance(cache, torch.Tensor) or cache.dtype not in _CACHE_CODE:
        raise TypeError("cache must be int8 or float8_e4m3fn")
    shape = cache.shape
    if len(shape) < 2:
        raise ValueError("cache must be [slots, ..., dstate]")
    if not cache.is_cuda:
        raise ValueError(f"cache must be on a GPU (got {cache.device})")
    dev = cache.device
    at = dev.index
    _check("cache", cache, at, cache.dtype, shape)
    _check("scales", scales, at, torch.float32, shape[:-1])
    n = _last_dim("slots", slots, ("batch",))
    _check("slots", slots, at, torch.int32, (n,))
    return dev, (n, *shape[1:]), (n, math.prod(shape[1:-1]), shape[-1], shape[0], _CACHE_CODE[cache.dtype])


def state_cache_write(h, cache, scales, slots) -> None:
    """Keeps the states h [Bt, ..., dstate] (fp32: a final state of
    ``ssd_fwd`` or ``selective_scan``, or the state of a step) in 8 bits, state
    i in slot slots[i] (int32 [Bt], on the GPU) of cache [slots, ..., dstate]
    (int8 or float8_e4m3fn), with a scale for each row of dstate values in
    scales [slots, ...] (fp32).  A state whose slot is out of range is not
    written; of several that name one slot the last is."""
    dev, shape, sizes = _cache_args(cache, scales, slots)
    _check("h", h, dev.index, torch.float32, shape)
    _run("state_cache_write", dev, _lib().state_cache_write, h.data_ptr(), slots.data_ptr(), *sizes, cache.data_ptr(),
         scales.data_ptr())


def state_cache_read(cache, scales, slots, out: torch.Tensor | None = None):
    """The states in the given slots of a cache that ``state_cache_write``
    filled, as fp32 [Bt, ..., dstate]: the h0 of ``ssd_fwd`` or
    ``selective_scan``, or the state of a step.  A slot out of range gives a
    state of zeros."""
    dev, shape, sizes = _cache_args(cache, scales, slots)
    if out is None:
        h = torch.empty(*shape, dtype=torch.float32, device=dev)
    else:
        h = out
        _check("out", h, dev.index, torch.float32, shape)
    _run("state_cache_read", dev, _lib().state_cache_read, cache.data_ptr(), scales.data_ptr(), slots.data_ptr(), *sizes,
         h.data_ptr())
    return h


__all__ = ["selective_scan", "selective_scan_bwd", "selective_scan_step", "short_conv", "short_conv_bwd",
           "short_conv_step", "state_cache_write", "state_cache_read"]
