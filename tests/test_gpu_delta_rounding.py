"""GPU tests of what 16-bit operands may cost the gated delta rule: outputs in
16 bits are off by their own rounding, and fp16 gradients are as near at any size of dy.

Tolerances as in test_gpu_delta.py, with the oracle's bounds, in which every
computed operand is two numbers of its type.
"""
import math

import numpy as np
import pytest
import torch

import chunked_linear_scan_amd as cls
from oracle import delta as od
from test_gpu_delta import KEYS, check, delta_case, oracle_args, run
from test_gpu_selective import U, close, f64, on_gpu

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1, 1, 1, 8, 8), (2, 130, 2, 4, 96, 72), (1, 200, 1, 2, 256, 40), (2, 65, 10, 10, 128, 200)]


def off_by_rounding(got, ref, label):
    """The 2-norm of the error is that of one rounding, and 2 % more for values that another rounding takes to the
    other side: operands of 16 bits at least in all leave 2^-16 and sums of some terms a few times that, against a
    rounding's 2^-9 / sqrt(3) (bf16)."""
    one = np.linalg.norm(f64(torch.from_numpy(ref).to(got.dtype)) - ref)
    off = np.linalg.norm(f64(got) - ref)
    assert off <= 1.02 * one, (label, off, one)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_y_is_off_by_its_rounding(shape, kind):
    c = delta_case(300 + SHAPES.index(shape), *shape, kind=kind)
    a = oracle_args(c)
    y, _ = cls.gated_delta(*(on_gpu(c)[k] for k in KEYS))
    ry, _ = od.delta(**a)
    _, err = od.delta_bounds(kind, 64, **a)
    close(y, ry, err["y"] / U, str(shape))
    off_by_rounding(y, ry, str(shape))


def test_fp16_y_of_a_small_scale():
    """The scale multiplies sums in fp32 and no operand: with 2^-9 y is what it is with 1, to the output's rounding."""
    c = on_gpu(delta_case(310, 1, 100, 1, 2, 64, 32, kind="f16"))
    c["v"], c["h0"] = c["v"] * 8, c["h0"] * 8
    y, _ = cls.gated_delta(*(c[k] for k in KEYS), scale=1.0)
    small, _ = cls.gated_delta(*(c[k] for k in KEYS), scale=2.0 ** -9)
    fits = y.abs() >= 2.0 ** -4  # a normal number of the type in both
    assert fits.any() and torch.equal((small * 512)[fits], y[fits])


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES[1:])
def test_gradients_of_16_bits_are_off_by_their_rounding(shape, kind):
    c = delta_case(320 + SHAPES.index(shape), *shape, kind=kind, start=False)
    got = check(c, kind, label=str(shape), dh=False)
    want = od.delta_grads(f64(c["dy"]), **oracle_args(c))
    for n in ("dq", "dk", "dv"):
        off_by_rounding(got[n], want[n], f"{shape} {n}")
