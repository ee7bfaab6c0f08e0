"""Python functions of ``include/selective_scan.h``: the selective scan, the
short convolution in front of it, and the 8-bit cache of states.

Argument marshalling only, as in the rest of the package, and done by the
native module ``_selective_binding`` (``binding/selective_binding.cpp``):
tensors are checked for device, dtype and shape, outputs and workspaces are
allocated with torch, and the library's kernels run on torch's current stream
of the inputs' device.  Activations may be slices of wider rows (their last
dimension adjacent); parameters and states are contiguous; outputs given as
`out` must not overlap inputs.  Each call has a
workspace of its own from torch's allocator, so calls on several streams and
captured graphs share none.

Nothing is recorded for autograd: gradients come from ``selective_scan_bwd`` and
``short_conv_bwd``.  Where a tensor that requires a gradient is passed while
autograd records, a backward pass through the outputs raises (a state updated in
place carries no such mark).
"""
from __future__ import annotations

import torch

_module = None


def _native():
    """The native binding, loaded once; raises if it or the library is missing."""
    global _module
    if _module is None:
        from . import load_library
        load_library()
        try:
            from . import _selective_binding
        except ImportError as e:
            raise RuntimeError("the native binding is missing or does not load: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`") from e
        _module = _selective_binding
    return _module


class _Unrecorded(torch.autograd.Function):
    """Outputs as they are, marked so that a backward pass through them raises.  The mark hangs on a tensor of its own:
    it keeps no graph of the caller's alive."""

    @staticmethod
    def forward(ctx, what, mark, *outputs):
        ctx.what = what
        ctx.mark_dirty(*outputs)
        return outputs

    @staticmethod
    def backward(ctx, *grads):
        call = ctx.what.removesuffix("_step") + "_bwd"
        raise RuntimeError(f"{ctx.what} records no gradient: take those of its inputs from {call}, over whole sequences, "
                           "or pass tensors that require none")


def _unrecorded(what, outputs):
    """Called by the binding where autograd follows one of a call's inputs."""
    return list(_Unrecorded.apply(what, torch.empty(0, requires_grad=True), *(t.detach() for t in outputs)))


# ---------------------------------------------------------------------------
# selective scan
# ---------------------------------------------------------------------------
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
    y, h, kept = _native().selective_scan(u, dt, A, B, C, D, z, dt_bias, h0, seqlens, dt_softplus, want_final_state,
                                          want_checkpoints, out)
    return (y, h, kept) if want_checkpoints else (y, h)


def selective_scan_bwd(dy, u, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, seqlens=None,
                       dt_softplus: bool = True, checkpoints: torch.Tensor | None = None, dh_final=None) -> dict:
    """Gradients of ``selective_scan``'s inputs from the gradient dy of its y
    (and dh_final of its h_final), with the checkpoints of the forward pass
    over the same inputs.  Returns a dict of "du", "ddt", "dB", "dC" (and
    "dz") in u's dtype and "dA" (and "dD", "ddt_bias", "dh0") in fp32; those
    in parentheses where the input was given.  dB and dC are summed over the
    channels of a group.  Padding has zero gradients."""
    return _native().selective_scan_bwd(dy, u, dt, A, B, C, D, z, dt_bias, h0, seqlens, dt_softplus, checkpoints,
                                        dh_final)


def selective_scan_step(h, u, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus: bool = True,
                        out: torch.Tensor | None = None):
    """One token of ``selective_scan`` for every sequence: updates the state h
    [Bt, channels, N] (fp32; on 16 bytes where N is a multiple of 4, as torch
    allocates and slices it) in place and returns y [Bt, channels].  u, dt and
    z [Bt, channels], B and C [Bt, groups, N]; the rest as there."""
    return _native().selective_scan_step(h, u, dt, A, B, C, D, z, dt_bias, dt_softplus, out)


# ---------------------------------------------------------------------------
# short convolution
# ---------------------------------------------------------------------------
def short_conv(x, weight, bias=None, initial_state=None, seqlens=None, silu: bool = True,
               want_final_state: bool = True, out: torch.Tensor | None = None):
    """Causal convolution of each channel over its last `width` tokens, with
    the activation silu (or none): x [Bt, L, channels] in fp32, bf16 or fp16
    (slices of wider rows are fine), weight [channels, width] with width 2 to
    4 and bias [channels] in fp32.  initial_state [Bt, width - 1, channels]
    holds the inputs before the first token (oldest first; zeros without), and
    the final state the last ones.  seqlens as in ``selective_scan``.  Returns
    (y, final_state or None)."""
    return _native().short_conv(x, weight, bias, initial_state, seqlens, silu, want_final_state, out)


def short_conv_bwd(dy, x, weight, bias=None, initial_state=None, seqlens=None, silu: bool = True,
                   dfinal_state=None) -> dict:
    """Gradients of ``short_conv``'s inputs from the gradient dy of its y (and
    dfinal_state of its final state): a dict of "dx" in x's dtype, "dweight"
    in fp32, and "dbias" (fp32) and "dinitial_state" where those were given."""
    return _native().short_conv_bwd(dy, x, weight, bias, initial_state, seqlens, silu, dfinal_state)


def short_conv_step(state, x, weight, bias=None, silu: bool = True, out: torch.Tensor | None = None):
    """One token of ``short_conv`` for every sequence: state
    [Bt, width - 1, channels] (x's dtype) takes x [Bt, channels] in and drops
    its oldest row, in place; returns y [Bt, channels]."""
    return _native().short_conv_step(state, x, weight, bias, silu, out)


# ---------------------------------------------------------------------------
# 8-bit cache of states
# ---------------------------------------------------------------------------
def state_cache_write(h, cache, scales, slots) -> None:
    """Keeps the states h [Bt, ..., dstate] (fp32: a final state of
    ``ssd_fwd`` or ``selective_scan``, or the state of a step) in 8 bits, state
    i in slot slots[i] (int32 [Bt], on the GPU) of cache [slots, ..., dstate]
    (int8 or float8_e4m3fn), with a scale for each row of dstate values in
    scales [slots, ...] (fp32).  A state whose slot is out of range is not
    written; of several that name one slot the last is."""
    _native().state_cache_write(h, cache, scales, slots)


def state_cache_read(cache, scales, slots, out: torch.Tensor | None = None):
    """The states in the given slots of a cache that ``state_cache_write``
    filled, as fp32 [Bt, ..., dstate]: the h0 of ``ssd_fwd`` or
    ``selective_scan``, or the state of a step.  A slot out of range gives a
    state of zeros."""
    return _native().state_cache_read(cache, scales, slots, out)


__all__ = ["selective_scan", "selective_scan_bwd", "selective_scan_step", "short_conv", "short_conv_bwd",
           "short_conv_step", "state_cache_write", "state_cache_read"]
