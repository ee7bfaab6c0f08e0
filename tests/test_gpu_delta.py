"""GPU tests of the gated delta rule against the float64 oracle.

Tolerance, element by element: |got - ref| <= 2 bound + eps/2 |ref|, plus half
the smallest subnormal of an fp16 output.  ``bound`` is the oracle's sum of
what the roundings of the kernels' operands and fp32 sums can do to the element
(its docstring says which), to first order, doubled here for the rest;
eps/2 |ref| is the one rounding to the output's type, half a step.
"""
import math
import threading

import numpy as np
import pytest
import torch

import chunked_linear_scan_amd as cls
from oracle import delta as od, selective as osel
from test_gpu_selective import KINDS, U, close, f64, on_gpu

pytestmark = pytest.mark.gpu

KEYS = ("q", "k", "v", "g", "beta", "h0", "seqlens")


def delta_case(seed, nb, L, Hk, H, dk, dv, kind="bf16", start=True, ragged=False, strong=False, off=0):
    """Inputs as a layer has them: q, k and v column ranges of one row per token (`off` elements from its start)."""
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t = KINDS[kind]
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    nk = Hk * dk
    row = torch.empty(nb, L, off + 2 * nk + H * dv)
    row[..., off:off + nk] = unit(rn(nb, L, Hk, dk) + 0.3).flatten(-2)
    row[..., off + nk:off + 2 * nk] = unit(rn(nb, L, Hk, dk) + 0.3).flatten(-2)
    row[..., off + 2 * nk:] = rn(nb, L, H * dv)
    row = row.to(t)
    c = dict(q=row[..., off:off + nk].unflatten(-1, (Hk, dk)), k=row[..., off + nk:off + 2 * nk].unflatten(-1, (Hk, dk)),
             v=row[..., off + 2 * nk:].unflatten(-1, (H, dv)))
    gb = torch.cat([-(rn(nb, L, H).abs() * (4.0 if strong else 0.1)), torch.sigmoid(rn(nb, L, H))], -1)
    c["g"], c["beta"] = gb[..., :H], gb[..., H:]
    c["h0"] = 0.5 * rn(nb, H, dv, dk) if start else None
    c["seqlens"] = torch.randint(0, L + 1, (nb,), generator=g).to(torch.int32) if ragged else None
    c["dy"] = rn(nb, L, H, dv + 3).to(t)[..., :dv]
    c["dh"] = rn(nb, H, dv, dk)
    return c


def oracle_args(c):
    a = {k: f64(c[k]) for k in KEYS[:-1]}
    a["seqlens"] = None if c["seqlens"] is None else c["seqlens"].numpy()
    return a


def run(d, scale=None, dh=True, **more):
    y, h, kept = cls.gated_delta(*(d[k] for k in KEYS), scale=scale, want_checkpoints=True, **more)
    grads = cls.gated_delta_bwd(d["dy"], *(d[k] for k in KEYS), scale=scale, checkpoints=kept,
                                dh_final=d["dh"] if dh else None)
    return {"y": y, "h": h, **grads}


def check(c, kind, scale=None, label="", dh=True):
    got = run(on_gpu(c), scale, dh)
    torch.cuda.synchronize()
    a = oracle_args(c)
    _, err = od.delta_bounds(kind, 32 if kind == "f32" else 64, **a, scale=scale, dy=f64(c["dy"]),
                             dh=f64(c["dh"]) if dh else None)
    y, h = od.delta(**a, scale=scale)
    want = {"y": y, "h": h, **od.delta_grads(f64(c["dy"]), **a, scale=scale, dh=f64(c["dh"]) if dh else None)}
    assert set(got) == set(want) - (set() if c["h0"] is not None else {"dh0"})
    for n in sorted(got):
        assert got[n].is_contiguous()
        close(got[n], want[n], err[n] / U, f"{label} {n}")  # close() doubles, and adds the output's rounding
    return got


# batch, length, key heads, heads, dk, dv
SHAPES = [(1, 1, 1, 1, 1, 1), (2, 2, 1, 2, 8, 8), (1, 31, 1, 1, 64, 64), (2, 32, 2, 2, 16, 24), (1, 33, 1, 3, 65, 17),
          (1, 63, 2, 2, 128, 128), (1, 64, 1, 1, 128, 16), (2, 65, 1, 2, 40, 100), (1, 130, 2, 4, 96, 72),
          (1, 100, 1, 1, 256, 64), (1, 70, 1, 2, 200, 130), (1, 200, 1, 1, 33, 5), (3, 129, 1, 1, 128, 64)]


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_delta_and_gradients(shape, kind):
    seed = 100 + SHAPES.index(shape)
    check(delta_case(seed, *shape, kind=kind, start=seed % 2 == 0, ragged=seed % 3 == 0, strong=seed % 5 == 0), kind,
          label=str(shape))


# more than 256 tiles of 16 columns, so workgroups of two; the last one of a head with one, or part of one
MANY = [(3, 64, 2, 6, 64, 250), (2, 65, 10, 10, 128, 200), (1, 190, 3, 9, 24, 500), (3, 330, 1, 3, 72, 450),
        (2, 129, 2, 6, 256, 360)]


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", MANY)
def test_delta_many_columns(shape, kind):
    seed = 200 + MANY.index(shape)
    check(delta_case(seed, *shape, kind=kind, start=seed % 2 == 0, ragged=seed % 2 == 1), kind, label=str(shape))


def test_delta_of_a_head_does_not_depend_on_the_others():
    """Workgroups of one and of two tiles of columns: the same sums in the same order."""
    c = on_gpu(delta_case(210, 2, 200, 9, 9, 64, 250, start=True))
    want = run(c)
    few = {k: v[:, :, :4] if k in ("q", "k", "v", "g", "beta", "dy") else v[:, :4].contiguous() if k in ("h0", "dh") else v
           for k, v in c.items()}
    got = run(few)
    for n in got:
        head = 1 if n in ("h", "dh0") else 2
        assert torch.equal(got[n], want[n].narrow(head, 0, 4)), n


@pytest.mark.parametrize("off", ["start", "dh", "ragged", "strong", "scale", "negative scale", "none"])
def test_delta_options(off):
    c = delta_case(7, 2, 90, 2, 4, 64, 40, start=off != "start", ragged=off == "ragged", strong=off == "strong")
    check(c, "bf16", scale={"scale": 0.7, "negative scale": -0.3}.get(off), dh=off != "dh", label=off)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("off", [1, 2, 4, 8])
def test_delta_rows_off_whole_vectors(off, kind):
    check(delta_case(8, 2, 70, 1, 2, 64, 32, kind=kind, off=off), kind, label=f"off {off}")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("lens", [[0, 0, 0], [1, 0, 150], [64, 65, 63], [32, 33, 31], [-3, 900, 128]])
def test_delta_lengths_and_what_the_padding_holds(lens, kind):
    """Any length, and NaN and infinities wherever a token is padding: outputs and gradients there are zeros."""
    c = delta_case(9, 3, 150, 1, 2, 48, 40, kind=kind)
    c["seqlens"] = torch.tensor(lens, dtype=torch.int32)
    clean = check(c, kind, label=str(lens))
    stuffed = dict(c)
    for k in ("q", "k", "v", "g", "beta", "dy"):
        v = c[k].clone()
        for b, n in enumerate(lens):
            v[b, min(max(n, 0), 150):] = math.nan if b % 2 else math.inf
        stuffed[k] = v
    got = run(on_gpu(stuffed))
    for n, w in clean.items():
        assert torch.equal(got[n], w), n
        if n not in ("h", "dh0"):
            for b, m in enumerate(lens):
                assert not got[n][b, min(max(m, 0), 150):].any(), n


def test_delta_forgets_at_minus_infinity():
    """g = -infinity starts a new sequence at its token: what came before has no effect and no gradient."""
    for kind in ("f32", "bf16"):
        c = delta_case(10, 2, 140, 1, 2, 64, 32, kind=kind)
        g = c["g"].clone()
        at = (0, 5, 6, 31, 32, 64, 100)
        for t in at:
            g[:, t] = -math.inf
        c["g"] = g
        got = check(c, kind, label="resets")
        assert not got["dh0"].any() and not got["dg"][:, list(at)].any()


def test_delta_of_growing_states():
    """Positive logarithms are evaluated as they are."""
    c = delta_case(11, 1, 70, 1, 2, 32, 16, kind="f32")
    c["g"] = -c["g"]
    check(c, "f32", label="growth")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_delta_alike_keys(kind):
    """One key over and over with beta up to 1 (the triangle's worst case of this rule), and zero beta and keys."""
    c = delta_case(12, 1, 130, 1, 4, 64, 32, kind=kind)
    c["k"] = c["k"][:, :1].expand_as(c["k"]).contiguous()
    beta = c["beta"].clone()
    beta[..., 0], beta[..., 1] = 1.0, 0.0
    beta[..., 2] = (torch.arange(130) % 2).float()
    c["beta"] = beta
    check(c, kind, label="alike")
    c["k"] = torch.zeros_like(c["k"])
    check(c, kind, label="zero keys")


def test_delta_beta_past_one():
    """beta in 1..2 reflects: still no growth."""
    c = delta_case(13, 1, 150, 1, 2, 64, 32, kind="bf16")
    c["beta"] = c["beta"] + 1
    check(c, "bf16", label="reflecting")


def test_delta_nan_stays_in_its_head_and_chunk():
    c = on_gpu(delta_case(14, 2, 200, 2, 4, 64, 64))
    y, _ = cls.gated_delta(*(c[k] for k in KEYS))
    v = c["v"].clone()
    v[1, 70, 2] = math.nan
    y2, h2 = cls.gated_delta(*(v if k == "v" else c[k] for k in KEYS))
    same = torch.ones(2, 200, 4, dtype=torch.bool, device="cuda")
    same[1, 64:, 2] = False
    assert torch.equal(y2[same], y[same])
    assert torch.isnan(y2[1, 70:, 2]).all() and torch.isnan(h2[1, 2]).all() and torch.isfinite(h2[0]).all()


def test_delta_fp16_states_of_any_small_size():
    """fp16 operands of small states keep their relative accuracy down to the type's subnormals: 2^-25 of each value."""
    c = delta_case(15, 1, 100, 1, 2, 64, 32, kind="f16", start=False)
    c["v"] = (c["v"].float() / 64).half()
    a = oracle_args(c)
    y, h = cls.gated_delta(*(on_gpu(c)[k] for k in KEYS))
    ry, rh = od.delta(**a)
    _, err = od.delta_bounds("f16", 64, **a)
    # N's small parts are whole multiples of 2^-24: up to 100 tokens' are off by half of one, times keys of length one
    close(h, rh, err["h"] / U + 100 * 2.0 ** -25 / U, "h")


def test_delta_shared_inputs_and_far_rows():
    """One sequence's q, k and g for all (strides of zero), and tokens 2^20 elements apart."""
    c = delta_case(16, 3, 70, 1, 2, 32, 24)
    for k in ("q", "k", "g", "beta"):
        c[k] = c[k][:1].expand(3, *c[k].shape[1:])
    d = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in c.items()}
    for k in ("q", "k", "g", "beta"):
        d[k] = c[k][:1].cuda().expand(3, *c[k].shape[1:])
        assert d[k].stride(0) == 0
    far = torch.zeros(70, 1 << 20, dtype=torch.bfloat16, device="cuda")
    far[:, 5:5 + 48] = d["v"][0].flatten(1)
    d["v"] = far[:, 5:5 + 48].unflatten(1, (2, 24))[None].expand(3, 70, 2, 24)
    c["v"] = c["v"][:1].expand(3, 70, 2, 24)
    got = run(d)
    a = oracle_args(c)
    _, err = od.delta_bounds("bf16", 64, **a, dy=f64(c["dy"]), dh=f64(c["dh"]))
    y, h = od.delta(**a)
    want = {"y": y, "h": h, **od.delta_grads(f64(c["dy"]), **a, dh=f64(c["dh"]))}
    for n in got:
        close(got[n], want[n], err[n] / U, n)


def test_delta_offsets_past_32_bits():
    """Sequences 2^31 and more elements from the first: the same bits as on their own."""
    L, H, dv = 40, 1, 16
    base = torch.zeros((1 << 31) + 4096, dtype=torch.bfloat16, device="cuda")
    c = on_gpu(delta_case(17, 2, L, 1, H, 32, dv))
    v = torch.as_strided(base, (2, L, H, dv), (1 << 31, dv, dv, 1))
    v.copy_(c["v"])
    want, got = run(c), run({**c, "v": v})
    for n in want:
        assert torch.equal(got[n], want[n]), n


def test_delta_long_sequence():
    """Many chunks, one head: the state's errors do not add up."""
    c = delta_case(18, 1, 2500, 1, 1, 32, 16, kind="bf16")
    check(c, "bf16", label="long")


def test_delta_same_bits_every_run_and_stale_memory():
    c = on_gpu(delta_case(19, 2, 200, 2, 4, 64, 48, ragged=True))
    want = run(c)
    for fill in (math.nan, 1e30):
        junk = [torch.full((1 << 22,), fill, device="cuda") for _ in range(8)]
        del junk  # the allocator hands this memory out next
        got = run(c)
        for n in want:
            assert torch.equal(got[n], want[n]), n


def test_delta_on_a_side_stream_and_in_graphs():
    c = on_gpu(delta_case(20, 2, 150, 1, 2, 64, 64))
    want = {n: v.clone() for n, v in run(c).items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run(c)
    side.synchronize()
    assert all(torch.equal(got[n], want[n]) for n in want)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        r1 = run(c)
    with torch.cuda.graph(g2):
        r2 = run(c)
    for k in range(3):
        c["v"].mul_(-0.5)  # new inputs, then both graphs at once on streams of their own
        want = {n: v.clone() for n, v in run(c).items()}
        torch.cuda.synchronize()
        for g in (g1, g2):
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for r in (r1, r2):
            assert all(torch.equal(r[n], want[n]) for n in want), k


def test_delta_from_two_threads_at_once():
    c = on_gpu(delta_case(21, 2, 300, 1, 2, 128, 64))
    want = run(c)
    torch.cuda.synchronize()
    bad = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(10):
                got = run(c)
                s.synchronize()
                bad.extend(n for n in want if not torch.equal(got[n], want[n]))

    threads = [threading.Thread(target=work) for _ in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not bad


# ---------------------------------------------------------------------------
# one token
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("nb,Hk,H,dk,dv", [(1, 1, 1, 1, 1), (3, 1, 2, 8, 5), (2, 2, 2, 64, 64), (2, 1, 4, 33, 7),
                                           (1, 2, 4, 128, 128), (2, 1, 1, 256, 100), (5, 1, 3, 100, 36),
                                           (70, 4, 8, 128, 128), (40, 4, 8, 30, 200)])
def test_delta_step(nb, Hk, H, dk, dv, kind):
    c = delta_case(30, nb, 1, Hk, H, dk, dv, kind=kind, off=3)
    d = {k: v[:, 0] if k in ("q", "k", "v", "g", "beta") else v for k, v in on_gpu(c).items()}
    h = d["h0"].clone()
    y = cls.gated_delta_step(h, d["q"], d["k"], d["v"], d["g"], d["beta"])
    a = oracle_args(c)
    ry, rh = od.delta_step(a["h0"], *(a[k][:, 0] for k in ("q", "k", "v", "g", "beta")))
    kn, qn = (np.repeat(np.linalg.norm(a[x][:, 0], axis=-1), H // Hk, 1)[..., None] for x in "kq")  # [nb, H, 1]
    S = np.exp(a["g"][:, 0])[..., None] * np.linalg.norm(a["h0"], axis=-1)  # the faded state's rows
    # fp32 throughout: a row's dots carry 32 units of its norm's, a factor few more
    delta = np.abs(a["beta"][:, 0])[..., None] * (kn * S + np.abs(a["v"][:, 0]))
    ak = np.repeat(np.abs(a["k"][:, 0]), H // Hk, 1)[:, :, None]
    close(h, rh, 8 * np.abs(a["h0"]) + 40 * delta[..., None] * ak, "h")
    close(y, ry, 64 * dk ** -0.5 * qn * (S + delta * kn), "y")


def test_delta_steps_are_the_prompt():
    """Token by token from a prompt's final state: what the whole sequence gives."""
    nb, L, more = 2, 70, 9
    c = delta_case(31, nb, L + more, 1, 2, 64, 48, kind="f32")
    d = on_gpu(c)
    names = ("q", "k", "v", "g", "beta")
    _, h = cls.gated_delta(*(d[k][:, :L] for k in names), h0=d["h0"])
    ys = [cls.gated_delta_step(h, *(d[k][:, t] for k in names)) for t in range(L, L + more)]
    a = oracle_args(c)
    _, err = od.delta_bounds("f32", 32, **a)
    y, rh = od.delta(**a)
    # a step's own roundings are of the kind that a chunk's bound counts
    close(torch.stack(ys, 1), y[:, L:], 2 * err["y"][:, L:] / U, "y")
    close(h, rh, 2 * err["h"] / U, "h")


def test_delta_step_on_states_past_32_bits_and_in_a_graph():
    nb, H, dk, dv = 5, 4, 256, 256
    cache = torch.zeros(1 << 13, H, dv, dk, device="cuda")  # 2^31 values
    d = on_gpu(delta_case(32, nb, 1, 2, H, dk, dv))
    args = [d[k][:, 0] for k in ("q", "k", "v", "g", "beta")]
    h = cache[-nb:]
    h.copy_(d["h0"])
    want_h = d["h0"].clone()
    want = cls.gated_delta_step(want_h, *args)
    assert torch.equal(cls.gated_delta_step(h, *args), want) and torch.equal(h, want_h)
    assert not cache[:-nb].any()
    h.copy_(d["h0"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = cls.gated_delta_step(h, *args)
    for _ in range(3):
        want_h.copy_(h)
        want = cls.gated_delta_step(want_h, *args)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(h, want_h)


def test_delta_states_through_the_cache():
    """A prompt's state kept in 8 bits, read back, and continued."""
    d = on_gpu(delta_case(33, 2, 64, 1, 2, 64, 32))
    _, h = cls.gated_delta(*(d[k] for k in KEYS))
    cache = torch.zeros(4, 2, 32, 64, dtype=torch.int8, device="cuda")
    scales = torch.zeros(4, 2, 32, device="cuda")
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    cls.state_cache_write(h, cache, scales, slots)
    back = cls.state_cache_read(cache, scales, slots)
    # half a step of the row's scale, and the scale's own rounding
    assert ((back - h).abs() <= h.abs().amax(-1, keepdim=True) / 127 * (0.5 + 2.0 ** -15)).all()
    y, _ = cls.gated_delta(*(d[k] for k in KEYS[:5]), h0=back)
    assert torch.isfinite(y).all()


# ---------------------------------------------------------------------------
# a layer
# ---------------------------------------------------------------------------
def test_a_layer_s_operators_together():
    """The stream and its norm, the convolution, keys of length one, the delta rule and its gated norm: forward and
    every gradient as a training step chains them, each against the oracle on what it was given."""
    nb, L, H, dk, dv, dim = 2, 75, 2, 32, 24, 64
    g = torch.Generator().manual_seed(40)
    rn = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    lens = torch.tensor([75, 41], dtype=torch.int32, device="cuda")
    x, res, w0, s0 = rn(nb, L, dim), rn(nb, L, dim), 1 + 0.1 * rn(dim), 0.5 + 0.1 * rn(dim)
    u, r, rstd0 = cls.residual_norm(x, res, w0, scale=s0, want_rstd=True)
    ch = 2 * H * dk + H * dv
    proj, wc = rn(dim, ch) * dim ** -0.5, rn(ch, 4) * 0.5
    z = rn(nb, L, H, dv)
    p = u @ proj
    conv, _ = cls.short_conv(p, wc, seqlens=lens, want_final_state=False)
    qk = conv[..., :2 * H * dk].unflatten(-1, (2 * H, dk))
    wk = torch.full((dk,), dk ** -0.5, device="cuda")
    unit, rstd1 = cls.gated_norm(qk, wk, want_rstd=True)
    q, k = unit[:, :, :H], unit[:, :, H:]
    v = conv[..., 2 * H * dk:].unflatten(-1, (H, dv))
    gl, beta = -0.2 * rn(nb, L, H).abs(), torch.sigmoid(rn(nb, L, H))
    y, _, kept = cls.gated_delta(q, k, v, gl, beta, seqlens=lens, want_checkpoints=True)
    w2, do = 1 + 0.1 * rn(dv), rn(nb, L, H, dv)
    o, rstd2 = cls.gated_norm(y, w2, z, want_rstd=True)
    # backward
    G2 = cls.gated_norm_bwd(do, y, w2, z, rstd2)
    Gd = cls.gated_delta_bwd(G2["dx"], q, k, v, gl, beta, seqlens=lens, checkpoints=kept)
    G1 = cls.gated_norm_bwd(torch.cat([Gd["dq"], Gd["dk"]], 2), qk, wk, rstd=rstd1)
    dconv = torch.cat([G1["dx"].flatten(2), Gd["dv"].flatten(2)], -1)
    Gc = cls.short_conv_bwd(dconv, p, wc, seqlens=lens)
    du, dr = Gc["dx"] @ proj.t().contiguous(), rn(nb, L, dim)
    G0 = cls.residual_norm_bwd(du, r, w0, rstd0, dr=dr, x=x, scale=s0)
    torch.cuda.synchronize()

    rows = lambda t, n: f64(t).reshape(-1, *t.shape[-n:])  # noqa: E731
    close(r, *osplit(od.residual_stream(f64(x), f64(res), f64(s0))), "stream")
    ry, rr, sy, sr = od.gated_norm(rows(r, 1)[:, None], f64(w0))
    close(u, ry.reshape(u.shape), sy.reshape(u.shape), "first norm")
    cy, _, cs = osel.conv(f64(p), f64(wc), seqlens=lens.cpu().numpy())
    close(conv, cy, cs, "convolution")
    ry, _, sy, _ = od.gated_norm(rows(qk, 2), f64(wk))
    close(unit, ry.reshape(unit.shape), sy.reshape(unit.shape), "keys")
    live = torch.arange(L, device="cuda") < lens[:, None]
    assert ((k.norm(dim=-1) - 1).abs()[live] < 1e-3).all()
    a = {"q": f64(q), "k": f64(k), "v": f64(v), "g": f64(gl), "beta": f64(beta), "seqlens": lens.cpu().numpy()}
    _, err = od.delta_bounds("f32", 32, **a, dy=f64(G2["dx"]))
    close(y, od.delta(**a)[0], err["y"] / U, "delta y")
    want = od.delta_grads(f64(G2["dx"]), **a)
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        close(Gd[n], want[n], err[n] / U, n)
    ry, _, sy, _ = od.gated_norm(rows(y, 2), f64(w2), rows(z, 2))
    close(o, ry.reshape(o.shape), sy.reshape(o.shape), "gated norm")
    want, sc = od.gated_norm_grads(rows(do, 2), rows(y, 2), f64(w2), rows(z, 2))
    for n in want:
        close(G2[n], want[n].reshape(G2[n].shape), sc[n].reshape(G2[n].shape), "gated norm " + n)
    want, sc = od.gated_norm_grads(np.concatenate([f64(Gd["dq"]), f64(Gd["dk"])], 2).reshape(-1, 2 * H, dk), rows(qk, 2),
                                   f64(wk))
    for n in want:
        close(G1[n], want[n].reshape(G1[n].shape), sc[n].reshape(G1[n].shape), "keys " + n)
    want, sc = od.residual_norm_grads(rows(du, 1), rows(r, 1), f64(w0), dr=rows(dr, 1), x=rows(x, 1), scale=f64(s0))
    for n in want:
        close(G0[n], want[n].reshape(G0[n].shape), sc[n].reshape(G0[n].shape), "first norm " + n)


def osplit(pair):
    return pair


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------
def test_delta_outputs_given_by_the_caller():
    c = on_gpu(delta_case(50, 2, 30, 1, 2, 32, 16))
    args = [c[k] for k in KEYS]
    y, _ = cls.gated_delta(*args)
    out = torch.empty_like(y)
    before = out._version
    got, h = cls.gated_delta(*args, out=out, want_final_state=False)
    assert h is None and got.data_ptr() == out.data_ptr() and torch.equal(out, y) and out._version == before + 1
    one = [c[k][:, 0] for k in KEYS[:5]]
    h = c["h0"].clone()
    want = cls.gated_delta_step(h, *one)
    h.copy_(c["h0"])
    before, out = h._version, torch.empty_like(want)
    assert cls.gated_delta_step(h, *one, out=out).data_ptr() == out.data_ptr() and torch.equal(out, want)
    assert h._version == before + 1
    for bad in (out[:, :1], out.float(), torch.empty(2, 2, 32, dtype=torch.bfloat16, device="cuda")[..., :16]):
        with pytest.raises((ValueError, TypeError)):
            cls.gated_delta_step(h, *one, out=bad)


def test_a_gradient_is_not_lost_in_silence():
    c = on_gpu(delta_case(51, 2, 9, 1, 2, 16, 8, kind="f32"))
    seq, one = [c[k] for k in KEYS[:6]], [c["h0"]] + [c[k][:, 0].contiguous() for k in KEYS[:5]]
    x, w = torch.randn(4, 2, 8, device="cuda"), torch.randn(8, device="cuda")
    calls = {"gated_delta": (lambda *t: cls.gated_delta(*t), seq),
             "gated_delta_step": (lambda h, *t: (cls.gated_delta_step(h.detach().clone() if False else h, *t),), one),
             "gated_norm": (lambda *t: (cls.gated_norm(*t),), [x, w, x.clone()]),
             "residual_norm": (lambda *t: cls.residual_norm(*t), [x, x.clone(), w, w.clone()])}
    for name, (call, tensors) in calls.items():
        state = [v.clone() for v in tensors]
        want = call(*state)
        assert not any(v.requires_grad for v in want)
        for i in range(len(tensors)):
            leaves = [v.clone().requires_grad_() if j == i else v.clone() for j, v in enumerate(tensors)]
            got = call(*leaves)
            for a, b in zip(got, want):
                assert a.requires_grad and torch.equal(a.detach(), b), (name, i)
                with pytest.raises(RuntimeError, match=f"{name} records no gradient.*{name.removesuffix('_step')}_bwd"):
                    a.sum().backward()
            with torch.no_grad():
                assert not any(v.requires_grad for v in call(*leaves))


def test_binding_refuses_bad_tensors():
    c = on_gpu(delta_case(52, 2, 9, 1, 2, 16, 8))
    args = {k: c[k] for k in KEYS}
    go = lambda **k: cls.gated_delta(**{**args, **k})  # noqa: E731
    for k, v, err in (("q", c["q"].float(), TypeError), ("q", c["q"][..., :8], ValueError), ("k", c["k"].cpu(), ValueError),
                      ("k", c["k"][:, :5], ValueError), ("v", c["v"].transpose(2, 3), ValueError),
                      ("v", c["v"].double(), TypeError), ("g", c["g"].bfloat16(), TypeError),
                      ("beta", c["beta"][..., :1], ValueError), ("beta", c["beta"].half(), TypeError),
                      ("h0", c["h0"].half(), TypeError), ("h0", c["h0"].transpose(2, 3), ValueError),
                      ("h0", c["h0"][:1], ValueError), ("seqlens", torch.zeros(2, dtype=torch.int64, device="cuda"), TypeError),
                      ("seqlens", torch.zeros(3, dtype=torch.int32, device="cuda"), ValueError),
                      ("out", torch.empty(2, 9, 2, 8, device="cuda"), TypeError)):
        with pytest.raises(err):
            go(**{k: v})
    with pytest.raises(cls.SSDError):  # three heads do not share two key heads
        cls.gated_delta(torch.zeros(2, 9, 2, 16, dtype=torch.bfloat16, device="cuda"),
                        torch.zeros(2, 9, 2, 16, dtype=torch.bfloat16, device="cuda"),
                        torch.zeros(2, 9, 3, 8, dtype=torch.bfloat16, device="cuda"),
                        torch.zeros(2, 9, 3, device="cuda"), torch.zeros(2, 9, 3, device="cuda"))
    wide = torch.zeros(2, 9, 1, 257, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(cls.SSDError):
        go(q=wide, k=wide, h0=None)
    with pytest.raises(cls.SSDError):
        cls.gated_delta(*(c[k][:, :0] for k in KEYS[:5]))
    with pytest.raises(ValueError, match="want_checkpoints"):
        cls.gated_delta_bwd(c["dy"], **args)
    with pytest.raises(ValueError, match="checkpoints"):
        cls.gated_delta_bwd(c["dy"], **args, checkpoints=torch.zeros(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="dy"):
        cls.gated_delta_bwd(c["dy"][:, :4], **args)
