"""GPU tests of the gated delta rule's fp16 gradients at small and large dy and dh_final.

Gradients are linear in dy and dh_final together.  Multiplied by a power of two, both have the
same numbers in front of the exponent, and so have the fp32 gradients, bit for bit, as long as the
kernels' operands do not depend on the gradients' size.  (dq, dk and dv are fp16: small ones have fewer bits.)
"""
import numpy as np
import pytest
import torch

import chunked_linear_scan_amd as cls
from oracle import delta as od
from test_gpu_delta import KEYS, check, delta_case, oracle_args, run
from test_gpu_selective import U, close, f64, on_gpu

pytestmark = pytest.mark.gpu


def exact_case(seed, *shape, **more):
    """dy in whole multiples of 2^-4 up to 4: 2^-14 of it still is a number of the type."""
    c = delta_case(seed, *shape, kind="f16", **more)
    g = torch.Generator().manual_seed(seed)
    c["dy"] = (torch.randint(-64, 65, c["dy"].shape, generator=g) / 16).half()
    c["dh"] = torch.randint(-64, 65, c["dh"].shape, generator=g) / 64
    return c


# heads taken apart in 64, 1, .. parts; values of one vector and of more than a workgroup has lanes
SHAPES = [(2, 130, 2, 4, 96, 72), (1, 200, 1, 2, 256, 40), (1, 70, 2, 2, 32, 200), (2, 9, 1, 1, 8, 8), (700, 3, 1, 3, 16, 8),
          (1, 40, 1, 1, 16, 2100), (1, 1, 1, 1, 1, 1), (100, 65, 1, 1, 20, 13)]


@pytest.mark.parametrize("power", [-14, -10, 13])
@pytest.mark.parametrize("shape", SHAPES)
def test_gradients_of_any_size_alike(shape, power):
    c = on_gpu(exact_case(400 + SHAPES.index(shape), *shape, ragged=shape[0] > 1))
    want = run(c)
    got = run({**c, "dy": c["dy"] * 2.0 ** power, "dh": c["dh"] * 2.0 ** power})
    for n in ("dg", "dbeta", "dh0"):
        assert want[n].any() and torch.equal(got[n], want[n] * 2.0 ** power), (n, power)


@pytest.mark.parametrize("size", [1e-3, 1e-5])
@pytest.mark.parametrize("dh", [False, True])
def test_small_gradients(size, dh):
    c = delta_case(410, 2, 150, 2, 4, 64, 48, kind="f16")
    c["dy"], c["dh"] = (c["dy"].float() * size).half(), c["dh"] * size
    got = check(c, "f16", label=str(size), dh=dh)
    want = od.delta_grads(f64(c["dy"]), **oracle_args(c), dh=f64(c["dh"]) if dh else None)
    for n in ("dg", "dbeta", "dh0"):  # two fp16 numbers to an operand: 2^-22 = 2.4e-7, some of them in a row
        assert np.linalg.norm(f64(got[n]) - want[n]) <= 2e-6 * np.linalg.norm(want[n]), n


def test_gradients_past_the_type():
    """dh_final past 65504 and a small dy: finite, and as near as others."""
    c = delta_case(411, 1, 90, 1, 2, 64, 48, kind="f16")
    c["dh"] = c["dh"] * 1e6
    got = run(on_gpu(c))
    a = oracle_args(c)
    _, err = od.delta_bounds("f16", 64, **a, dy=f64(c["dy"]), dh=f64(c["dh"]))
    want = od.delta_grads(f64(c["dy"]), **a, dh=f64(c["dh"]))
    for n in ("dg", "dbeta", "dh0"):
        close(got[n], want[n], err[n] / U, n)


def test_pairs_past_the_type():
    """Products of dy with the corrections past 65504 that a small scale brings back."""
    c = delta_case(412, 1, 90, 1, 2, 64, 128, kind="f16", start=False)
    c["v"], c["dy"] = c["v"] * 1000, c["dy"] * 30
    check(c, "f16", scale=2.0 ** -10, label="pairs", dh=False)


def test_one_head_s_size_is_its_own():
    """A head with large gradients beside one with small ones, and lengths of zero: each as on its own."""
    c = exact_case(413, 3, 100, 2, 2, 64, 32)
    c["dy"][:, :, 1] *= 2.0 ** -12
    c["dh"][:, 1] *= 2.0 ** -12
    c["seqlens"] = torch.tensor([100, 0, 64], dtype=torch.int32)
    d = on_gpu(c)
    got = run(d)
    one = {k: v[:, :, 1:].contiguous() if k in ("q", "k", "v", "g", "beta", "dy") else
           v[:, 1:].contiguous() if k in ("h0", "dh") else v for k, v in d.items()}
    one["dy"], one["dh"] = one["dy"] * 4096, one["dh"] * 4096
    want = run(one)
    for n, head in (("dg", 2), ("dbeta", 2), ("dh0", 1)):
        assert torch.equal(got[n].narrow(head, 1, 1) * 4096, want[n]), n
    assert not got["dg"][1].any() and torch.equal(got["dh0"][1], d["dh"][1])


def test_sizes_in_a_graph():
    """Captured once and replayed with gradients of other sizes."""
    c = on_gpu(exact_case(415, 2, 130, 1, 2, 64, 48))
    want = {n: v.clone() for n, v in run(c).items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run(c)
    for power in (-9, 4, 3):
        c["dy"].mul_(2.0 ** power)
        c["dh"].mul_(2.0 ** power)
        for n in want:
            want[n] = want[n] * 2.0 ** (power if n != "y" and n != "h" else 0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for n in ("y", "h", "dg", "dbeta", "dh0"):
            assert torch.equal(got[n], want[n]), (n, power)


def test_values_that_are_not_finite_do_not_set_the_size():
    """A NaN or an infinity in one token's dy leaves the later chunks' gradients what they were."""
    c = on_gpu(exact_case(414, 1, 200, 1, 1, 64, 32))
    want = run(c)
    for bad in (float("nan"), float("inf"), float("-inf")):
        dy = c["dy"].clone()
        dy[0, 10, 0, 3] = bad
        got = run({**c, "dy": dy})
        for n in ("dg", "dbeta", "dv"):
            assert torch.equal(got[n][:, 64:], want[n][:, 64:]), (bad, n)
            assert torch.isfinite(want[n]).all() and not torch.isfinite(got[n][:, :64]).all()
