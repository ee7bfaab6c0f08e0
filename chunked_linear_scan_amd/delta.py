"""Python functions of ``include/gated_delta.h``: the gated delta rule, and the
norms around the block of a layer with this or another recurrence.

Argument marshalling only, by the same native module and to the same rules as
in ``selective``: activations may be slices of wider rows (their last
dimension adjacent), states are contiguous, every call has a workspace of its
own from torch's allocator, and nothing is recorded for autograd: gradients come from
the functions that end in ``_bwd``.
"""
from __future__ import annotations

import torch

from .selective import _native


# ---------------------------------------------------------------------------
# gated delta rule
# ---------------------------------------------------------------------------
def gated_delta(q, k, v, g, beta, h0=None, seqlens=None, scale: float | None = None, want_final_state: bool = True,
                want_checkpoints: bool = False, out: torch.Tensor | None = None):
    """Gated delta rule over whole sequences, for each head:

        S_t = e^{g_t} S_{t-1} + beta_t (v_t - e^{g_t} S_{t-1} k_t) k_t^T,   y_t = scale S_t q_t

    q and k [Bt, L, key heads, dk] and v [Bt, L, heads, dv] in fp32, bf16 or
    fp16 (one dtype; slices of wider rows are fine), heads a multiple of the
    key heads, which adjacent heads share; g (a logarithm, usually at most 0)
    and beta [Bt, L, heads] and the state h0 [Bt, heads, dv, dk] (optional) in
    fp32.  dk is at most 256.  The rule expects keys of length one
    (``gated_norm`` with a weight of dk**-0.5 makes them) and beta in 0 to 2;
    scale is dk**-0.5 unless given.  seqlens (int32 [Bt], on the GPU): tokens
    at or past a sequence's length are padding; their y is zero.  With 16-bit
    elements products take what was computed before them in two numbers of that
    type: h_final is within some 2^-18 of fp32's in bf16, and in fp16 as near as
    fp32 where v and h0 are of the size of 1 (of 2^-n, some 2^(n - 25)).

    Returns (y, h_final or None), and with want_checkpoints
    (y, h_final or None, checkpoints), where checkpoints is what
    ``gated_delta_bwd`` takes."""
    y, h, kept = _native().gated_delta(q, k, v, g, beta, h0, seqlens, scale, want_final_state, want_checkpoints, out)
    return (y, h, kept) if want_checkpoints else (y, h)


def gated_delta_bwd(dy, q, k, v, g, beta, h0=None, seqlens=None, scale: float | None = None,
                    checkpoints: torch.Tensor | None = None, dh_final=None) -> dict:
    """Gradients of ``gated_delta``'s inputs from the gradient dy of its y (and
    dh_final of its h_final), with the checkpoints of the forward pass over the
    same inputs.  Returns a dict of "dq", "dk", "dv" in v's dtype, "dg",
    "dbeta" in fp32, and "dh0" where h0 was given.  dq and dk are summed over
    the heads that share a key head.  Padding has zero gradients.  fp16
    gradients lose nothing to the size of dy and dh_final."""
    return _native().gated_delta_bwd(dy, q, k, v, g, beta, h0, seqlens, scale, checkpoints, dh_final)


def gated_delta_step(h, q, k, v, g, beta, scale: float | None = None, out: torch.Tensor | None = None):
    """One token of ``gated_delta`` for every sequence: updates the state h
    [Bt, heads, dv, dk] (fp32; on 16 bytes where dk is a multiple of 4, as
    torch allocates and slices it) in place and returns y [Bt, heads, dv].  q
    and k [Bt, key heads, dk], v [Bt, heads, dv], g and beta [Bt, heads]."""
    return _native().gated_delta_step(h, q, k, v, g, beta, scale, out)


# ---------------------------------------------------------------------------
# norms
# ---------------------------------------------------------------------------
def gated_norm(x, weight=None, z=None, eps: float = 1e-6, gate_first: bool = False, want_rstd: bool = False,
               out: torch.Tensor | None = None):
    """Norm of each row by its root mean square, with a gate: the output norm of
    a recurrence.  x and z (optional) [..., heads, dim] in fp32, bf16 or fp16
    (slices of wider rows are fine), weight (optional) [dim] in fp32:

        y = (x / rms(x)) weight silu(z),   or with gate_first   y = (u / rms(u)) weight,  u = x silu(z)

    where rms(x) = sqrt(mean(x^2) + eps) over the last dimension (at most
    16384).  Returns y, and with want_rstd (y, rstd), where rstd
    [..., heads] is what ``gated_norm_bwd`` takes."""
    y, rstd = _native().gated_norm(x, weight, z, eps, gate_first, want_rstd, out)
    return (y, rstd) if want_rstd else y


def gated_norm_bwd(dy, x, weight=None, z=None, rstd: torch.Tensor | None = None, gate_first: bool = False) -> dict:
    """Gradients of ``gated_norm``'s inputs from the gradient dy of its y and the
    forward pass's rstd: a dict of "dx" and, where they were given, "dz" in
    x's dtype and "dweight" in fp32."""
    return _native().gated_norm_bwd(dy, x, weight, z, rstd, gate_first)


def residual_norm(x, residual=None, weight=None, scale=None, eps: float = 1e-6, want_rstd: bool = False):
    """The residual stream past a block and the norm in front of the next:

        r = residual + scale x,   y = (r / rms(r)) weight

    x [..., dim] in fp32, bf16 or fp16, residual (optional, zeros without) in
    fp32 or x's dtype, weight and scale (optional, ones without) [dim] in fp32.
    Returns (y, r), y in x's dtype and r in residual's (x's without); the norm
    is that of r as it is returned.  With want_rstd (y, r, rstd), where rstd
    [...] is what ``residual_norm_bwd`` takes."""
    y, r, rstd = _native().residual_norm(x, residual, weight, scale, eps, want_rstd)
    return (y, r, rstd) if want_rstd else (y, r)


def residual_norm_bwd(dy, r, weight, rstd, dr=None, x=None, scale=None) -> dict:
    """Gradients of ``residual_norm``'s inputs from the gradients dy of its y and
    dr (optional, zeros without) of its r, with the forward pass's r and rstd:
    a dict of "dresidual" in r's dtype, "dx" in dy's, and where they were given
    "dweight" and "dscale" (which needs x) in fp32."""
    return _native().residual_norm_bwd(dy, r, weight, rstd, dr, x, scale)


__all__ = ["gated_delta", "gated_delta_bwd", "gated_delta_step", "gated_norm", "gated_norm_bwd", "residual_norm",
           "residual_norm_bwd"]
