"""GPU tests of gated_norm and residual_norm against the float64 oracle.

Tolerance as in test_gpu_selective.py: 2 * 2^-24 * scale + eps/2 |ref|, with the
oracle's count of fp32 roundings for the scale.  The norm's inputs are what the
kernels were given: for residual_norm the stream as it was returned.
"""
import math

import numpy as np
import pytest
import torch

import chunked_linear_scan_amd as cls
from oracle import delta as od
from test_gpu_selective import KINDS, close, f64, on_gpu

pytestmark = pytest.mark.gpu

# lanes of a row and runs of 8 values to a lane: every kernel, with rows that fill it, one short and barely started
DIMS = [1, 7, 8, 63, 64, 65, 72, 127, 128, 129, 500, 512, 513, 1000, 1024, 1025, 2047, 2048, 2056, 4096, 4100, 8192, 8200,
        16383, 16384]


def gated_case(seed, rows, H, dim, kind, gate=True, weight=True, odd=0):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t = KINDS[kind]
    z = rn(rows, (H + 1) * dim + odd).to(t)[:, dim + odd:].unflatten(-1, (H, dim))
    return dict(x=(rn(rows, H, dim) * torch.exp(rn(rows, H, 1))).to(t), z=z if gate else None,
                weight=rn(dim) if weight else None, dy=rn(rows, H, dim + odd).to(t)[..., odd:])


def check_gated(c, gate_first, label, eps=1e-6):
    d = on_gpu(c)
    y, rstd = cls.gated_norm(d["x"], d["weight"], d["z"], eps=eps, gate_first=gate_first, want_rstd=True)
    assert torch.equal(y, cls.gated_norm(d["x"], d["weight"], d["z"], eps=eps, gate_first=gate_first))
    G = cls.gated_norm_bwd(d["dy"], d["x"], d["weight"], d["z"], rstd, gate_first)
    a = [f64(c[k]) for k in ("x", "weight", "z")]
    ry, rr, sy, sr = od.gated_norm(*a, eps=eps, gate_first=gate_first)
    close(y, ry, sy, label + " y")
    close(rstd, rr, sr, label + " rstd")
    want, sc = od.gated_norm_grads(f64(c["dy"]), *a, eps=eps, gate_first=gate_first)
    if c["weight"] is None:
        want.pop("dweight")
    assert set(G) == set(want)
    for n in want:
        close(G[n], want[n], sc[n], f"{label} {n}")


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dim", DIMS)
def test_gated_norm(dim, kind):
    rows, H = (5, 3) if dim <= 1024 else (3, 1)
    check_gated(gated_case(dim, rows, H, dim, kind), dim % 2 == 0, f"{dim}")
    check_gated(gated_case(dim + 1, rows, H, dim, kind, odd=1), dim % 2 == 1, f"{dim} off vectors")


@pytest.mark.parametrize("gate_first", [False, True])
@pytest.mark.parametrize("gate,weight", [(False, True), (True, False), (False, False)])
def test_gated_norm_options(gate, weight, gate_first):
    check_gated(gated_case(3, 6, 2, 100, "bf16", gate, weight), gate_first, "options", eps=1e-3)


def test_gated_norm_of_many_rows():
    """More rows than the gradients' launch has lanes for: its workgroups walk several, and sum all."""
    check_gated(gated_case(4, 20000, 2, 24, "f32"), False, "many short")
    check_gated(gated_case(5, 3000, 1, 1100, "bf16"), True, "many long")


@pytest.mark.parametrize("dim,rows", [(700, 2500), (2500, 700), (5000, 600), (9000, 300)])
def test_norms_of_many_wide_rows(dim, rows):
    """A row over 128 to 1024 lanes, and more rows than workgroups: the waves' sums of one row and the next do not meet."""
    check_gated(gated_case(6 + dim, rows, 1, dim, "bf16"), False, "wide")
    check_residual(residual_case(7 + dim, rows, dim, "bf16", "f32"), "wide")


def test_gated_norm_row_of_zeros_and_large_values():
    """A zero row has the norm of eps alone; squares stay finite up to 2^63 (fp32), and gates saturate."""
    c = gated_case(6, 4, 2, 64, "f32")
    c["x"][0] = 0
    c["x"][1] *= 2.0 ** 50
    c["z"] = c["z"].clone()
    c["z"][2, 0], c["z"][2, 1] = 200.0, -200.0
    check_gated(c, False, "extremes")


def test_gated_norm_nan_stays_in_its_row():
    c = on_gpu(gated_case(7, 9, 3, 40, "bf16"))
    y = cls.gated_norm(c["x"], c["weight"], c["z"])
    x = c["x"].clone()
    x[4, 1, 7], x[5, 2, 0] = math.nan, math.inf
    y2 = cls.gated_norm(x, c["weight"], c["z"])
    bad = torch.zeros(9, 3, dtype=torch.bool, device="cuda")
    bad[4, 1] = bad[5, 2] = True
    assert torch.equal(y2[~bad], y[~bad]) and torch.isnan(y2[4, 1]).all() and torch.isnan(y2[5, 2, 0])


def test_norms_of_more_dimensions_and_slices():
    """[batch, seqlen, heads, dim] slices of wider rows are one run of rows; others are refused."""
    g = torch.Generator().manual_seed(8)
    wide = torch.randn(3, 7, 5 * 32, generator=g).cuda()
    x = wide[..., 32:96].unflatten(-1, (2, 32))
    y = cls.gated_norm(x)
    assert torch.equal(y, cls.gated_norm(x.contiguous())) and y.shape == x.shape
    assert torch.equal(cls.residual_norm(wide[..., :40])[0], cls.residual_norm(wide[..., :40].contiguous())[0])
    assert torch.equal(cls.gated_norm(x[:, :1]), cls.gated_norm(x[:, :1].contiguous()))
    one = wide[:1, :1].expand(4, 6, 160)[..., :64].unflatten(-1, (2, 32))
    assert torch.equal(cls.gated_norm(one), cls.gated_norm(one.contiguous()))
    for bad in (wide[:, :5, :64].unflatten(-1, (2, 32)), wide[:, :1].expand(3, 7, 160)[..., :64].unflatten(-1, (2, 32))):
        with pytest.raises(ValueError, match="one distance"):
            cls.gated_norm(bad)
    with pytest.raises(ValueError, match="adjacent"):
        cls.gated_norm(x.transpose(-1, -2))


def residual_case(seed, rows, dim, kind, stream, residual=True, scale=True, weight=True, odd=0):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t, st = KINDS[kind], KINDS[stream]
    cut = lambda v: v[:, odd:]  # noqa: E731
    return dict(x=cut(rn(rows, dim + odd).to(t)), residual=cut((3 * rn(rows, dim + odd)).to(st)) if residual else None,
                scale=rn(dim) if scale else None, weight=rn(dim) if weight else None,
                dy=cut(rn(rows, dim + odd).to(t)), dr=cut(rn(rows, dim + odd).to(st)))


def check_residual(c, label, dr=True):
    d = on_gpu(c)
    y, r, rstd = cls.residual_norm(d["x"], d["residual"], d["weight"], d["scale"], want_rstd=True)
    a = {k: f64(v) for k, v in c.items()}
    close(r, *od.residual_stream(a["x"], a["residual"], a["scale"]), label + " r")
    kept = f64(r)
    ry, rr, sy, sr = od.gated_norm(kept[:, None], a["weight"])
    close(y, ry[:, 0], sy[:, 0], label + " y")
    close(rstd, rr[:, 0], sr[:, 0], label + " rstd")
    G = cls.residual_norm_bwd(d["dy"], r, d["weight"], rstd, dr=d["dr"] if dr else None, x=d["x"], scale=d["scale"])
    want, sc = od.residual_norm_grads(a["dy"], kept, a["weight"], dr=a["dr"] if dr else None, x=a["x"], scale=a["scale"])
    if c["weight"] is None:
        want.pop("dweight")
    assert set(G) == set(want)
    for n in want:
        close(G[n], want[n], sc[n], f"{label} {n}")


@pytest.mark.parametrize("kind,stream", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("dim", DIMS)
def test_residual_norm(dim, kind, stream):
    rows = 7 if dim <= 1024 else 3
    check_residual(residual_case(dim, rows, dim, kind, stream), f"{dim}")
    check_residual(residual_case(dim + 1, rows, dim, kind, stream, odd=1), f"{dim} off vectors")


@pytest.mark.parametrize("off", ["residual", "scale", "weight", "dr", "all", "none"])
def test_residual_norm_options(off):
    on = {k: off not in (k, "all") for k in ("residual", "scale", "weight")}
    check_residual(residual_case(20, 9, 100, "bf16", "bf16" if off in ("residual", "all") else "f32", **on), off,
                   dr=off not in ("dr", "all"))


def test_residual_norm_of_many_rows():
    check_residual(residual_case(21, 40000, 16, "f32", "f32"), "many short")
    check_residual(residual_case(22, 2500, 1200, "bf16", "f32"), "many long")


def test_norms_same_bits_every_run_and_in_a_graph():
    c, e = on_gpu(gated_case(23, 3000, 2, 128, "bf16")), on_gpu(residual_case(24, 1500, 256, "bf16", "f32"))

    def step():
        y, k = cls.gated_norm(c["x"], c["weight"], c["z"], want_rstd=True)
        y2, r, k2 = cls.residual_norm(e["x"], e["residual"], e["weight"], e["scale"], want_rstd=True)
        return [y, y2, r, *cls.gated_norm_bwd(c["dy"], c["x"], c["weight"], c["z"], k).values(),
                *cls.residual_norm_bwd(e["dy"], r, e["weight"], k2, dr=e["dr"], x=e["x"], scale=e["scale"]).values()]

    want = [v.clone() for v in step()]
    assert all(torch.equal(a, b) for a, b in zip(step(), want))
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        r1 = step()
    with torch.cuda.graph(g2):
        r2 = step()
    for k in range(3):
        c["x"].mul_(-1.5)
        e["residual"].mul_(0.5)
        want = [v.clone() for v in step()]
        torch.cuda.synchronize()
        for g in (g1, g2):
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for r in (r1, r2):
            assert all(torch.equal(a, b) for a, b in zip(r, want)), k


def test_norm_offsets_past_32_bits():
    base = torch.zeros((1 << 31) + 4096, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(base, (3, 64), (1 << 30, 1))
    x.copy_(torch.randn(3, 64))
    assert torch.equal(cls.residual_norm(x)[0], cls.residual_norm(x.contiguous())[0])
    assert torch.equal(cls.gated_norm(x[:, None]), cls.gated_norm(x[:, None].contiguous()))


def test_ssd_output_norm():
    """Behind an SSD layer the gate comes first, and the norm is over all heads' outputs."""
    g = torch.Generator().manual_seed(25)
    nb, L, H, P, S = 2, 64, 4, 64, 64
    x = torch.randn(nb, L, H, P, generator=g).bfloat16().cuda()
    B, C = (torch.randn(nb, L, 1, S, generator=g).bfloat16().cuda() for _ in range(2))
    dt = torch.nn.functional.softplus(torch.randn(nb, L, H, generator=g) - 2).cuda()
    A = -torch.exp(torch.rand(H, generator=g)).cuda()
    y, _ = cls.ssd_fwd(x, dt, A, B, C, chunk=64)
    z = torch.randn(nb, L, H * P, generator=g).bfloat16().cuda()
    w = torch.randn(H * P, generator=g).cuda()
    o = cls.gated_norm(y.flatten(2)[:, :, None], w, z[:, :, None], eps=1e-5, gate_first=True)
    ry, _, sy, _ = od.gated_norm(f64(y).reshape(nb * L, 1, H * P), f64(w), f64(z).reshape(nb * L, 1, H * P), 1e-5, True)
    close(o, ry.reshape(o.shape), sy.reshape(o.shape), "ssd norm")


def test_binding_refuses_bad_tensors():
    c, e = on_gpu(gated_case(26, 4, 2, 16, "bf16")), on_gpu(residual_case(27, 4, 16, "bf16", "f32"))
    for bad in (dict(weight=c["weight"][:8]), dict(weight=c["weight"].half()), dict(z=c["z"].float()), dict(z=c["z"][:2]),
                dict(z=c["z"].cpu()), dict(out=torch.empty(4, 2, 8, dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            cls.gated_norm(**{**dict(x=c["x"], weight=c["weight"], z=c["z"]), **bad})
    with pytest.raises(ValueError, match="want_rstd"):
        cls.gated_norm_bwd(c["dy"], c["x"])
    with pytest.raises(ValueError, match="rstd"):
        cls.gated_norm_bwd(c["dy"], c["x"], rstd=torch.ones(8, device="cuda"))
    with pytest.raises(TypeError, match="residual"):
        cls.residual_norm(e["x"], e["residual"].half())
    with pytest.raises(TypeError, match="residual"):
        cls.residual_norm(e["x"], e["residual"].double())
    with pytest.raises(ValueError, match="scale"):
        cls.residual_norm(e["x"], e["residual"], scale=e["scale"][:4])
    y, r, k = cls.residual_norm(e["x"], e["residual"], want_rstd=True)
    with pytest.raises(ValueError, match="x"):
        cls.residual_norm_bwd(e["dy"], r, None, k, scale=e["scale"])
    with pytest.raises(TypeError, match="dr"):
        cls.residual_norm_bwd(e["dy"], r, None, k, dr=e["dr"].half())
    with pytest.raises(cls.SSDError):
        cls.residual_norm(torch.zeros(2, 16385, device="cuda"))
    with pytest.raises(cls.SSDError):
        cls.gated_norm(torch.zeros(0, 2, 8, device="cuda"))
