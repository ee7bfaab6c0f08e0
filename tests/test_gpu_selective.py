"""GPU tests of the selective scan, the short convolution and the 8-bit cache
against the float64 oracle.

Tolerance, element by element: |got - ref| <= 2 * 2^-24 * scale + eps/2 |ref|,
plus half the smallest subnormal of an fp16 output.  ``scale`` is the oracle's
count of the fp32 roundings that reach the element (its docstring says which;
doubled here for second-order terms), and eps/2 |ref| is the one rounding to
the output's type, half a step.  What is held in 8 bits is compared byte by
byte.
"""
import math

import numpy as np
import pytest
import torch

import chunked_linear_scan_amd as cls
from oracle import selective as osel, ssd as ossd

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
KINDS = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def f64(t):
    return None if t is None else t.detach().to(torch.float64).cpu().numpy()


def close(got, ref, scale, label):
    kind = got.dtype
    g = f64(got)
    assert g.shape == ref.shape, (label, g.shape, ref.shape)
    half = torch.finfo(kind).eps / 2 if kind != torch.float32 else U
    bound = 2 * U * scale + half * np.abs(ref) + (2.0 ** -25 if kind == torch.float16 else 1e-37)
    bad = ~(np.abs(g - ref) <= bound)
    if bad.any():
        i = np.unravel_index(int(np.argmax(np.where(bad, np.abs(g - ref) / bound, 0))), bad.shape)
        raise AssertionError((label, int(bad.sum()), g.size, "worst", tuple(map(int, i)), g[i], ref[i], bound[i]))


def scan_case(seed, nb, L, ch, N, G, kind="bf16", gate=True, skip=True, bias=True, start=False, ragged=False,
              softplus=True):
    """Inputs as a layer has them: u adjacent, z and the convolution's input in one row, B and C behind dt's columns."""
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    dt_ = KINDS[kind]
    c = dict(u=rn(nb, L, ch).to(dt_), dt=(0.7 * rn(nb, L, ch)).to(dt_),
             A=-torch.exp(rn(ch, N)), D=rn(ch) if skip else None)
    if not softplus:
        c["dt"] = c["dt"].abs()
    xz = rn(nb, L, 2 * ch + 1).to(dt_)
    bc = rn(nb, L, 7 + 2 * G * N).to(dt_)
    c["z"] = xz[..., ch + 1:] if gate else None
    c["B"] = bc[..., 7:7 + G * N].unflatten(-1, (G, N))
    c["C"] = bc[..., 7 + G * N:].unflatten(-1, (G, N))
    c["dt_bias"] = (rn(ch) - 2 if softplus else rn(ch).abs()) if bias else None
    c["h0"] = rn(nb, ch, N) if start else None
    c["seqlens"] = torch.randint(0, L + 1, (nb,), generator=g).to(torch.int32) if ragged else None
    c["dy"] = rn(nb, L, ch + 3).to(dt_)[..., 2:2 + ch]
    c["dh"] = rn(nb, ch, N)
    return c


SCAN_KEYS = ("u", "dt", "A", "B", "C", "D", "z", "dt_bias", "h0", "seqlens")


def on_gpu(c):
    """The same tensors on the GPU, slices still slices of wider rows."""
    out = {}
    for k, v in c.items():
        if isinstance(v, torch.Tensor) and not v.is_contiguous():
            base = torch.empty_strided(v.shape, v.stride(), dtype=v.dtype, device="cuda")
            base.copy_(v)
            v = base
        out[k] = v.cuda() if isinstance(v, torch.Tensor) else v
    return out


def oracle_args(c):
    a = {k: f64(c[k]) for k in SCAN_KEYS[:-1]}
    a["seqlens"] = None if c["seqlens"] is None else c["seqlens"].numpy()
    return a


def check_scan(c, softplus=True, label=""):
    d = on_gpu(c)
    y, h, kept = cls.selective_scan(*(d[k] for k in SCAN_KEYS), dt_softplus=softplus, want_checkpoints=True)
    grads = cls.selective_scan_bwd(d["dy"], *(d[k] for k in SCAN_KEYS), dt_softplus=softplus, checkpoints=kept,
                                   dh_final=d["dh"])
    torch.cuda.synchronize()
    a = oracle_args(c)
    ry, rh, ys, hs = osel.scan(**a, softplus=softplus)
    close(y, ry, ys, label + " y")
    close(h, rh, hs, label + " h")
    G, S = osel.scan_grads(f64(c["dy"]), **a, softplus=softplus, dh=f64(c["dh"]))
    want = {"du", "ddt", "dA", "dB", "dC"} | {n for n, k in (("dD", "D"), ("dz", "z"), ("ddt_bias", "dt_bias"),
                                                           ("dh0", "h0")) if c[k] is not None}
    assert set(grads) == want
    for k in sorted(want):
        close(grads[k], G[k], S[k], f"{label} {k}")


# batch, length, channels, states, groups
SHAPES = [(1, 1, 1, 1, 1), (2, 15, 64, 16, 1), (1, 16, 65, 16, 1), (3, 17, 63, 4, 1), (2, 33, 130, 5, 2),
          (1, 100, 192, 16, 3), (2, 40, 24, 8, 4), (1, 50, 70, 20, 1), (2, 31, 66, 33, 2), (1, 24, 64, 64, 1),
          (2, 19, 6, 3, 6), (1, 300, 70, 16, 1)]


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_scan_and_gradients(shape, kind):
    print(f"[scan] {shape} {kind}", flush=True)
    check_scan(scan_case(1 + sum(shape), *shape, kind=kind, start=shape[0] > 1), label=f"{shape} {kind}")


@pytest.mark.parametrize("off", ["gate", "skip", "bias", "softplus", "start", "ragged", "all"])
def test_scan_options(off):
    print(f"[scan] without {off}", flush=True)
    o = dict(gate=True, skip=True, bias=True, softplus=True, start=True, ragged=True)
    for k in o if off == "all" else (off,):
        o[k] = k == "softplus" and off == "all"
    check_scan(scan_case(5, 3, 45, 72, 16, 2, kind="f32", **o), softplus=o["softplus"], label=off)


@pytest.mark.parametrize("N", [16, 40])
@pytest.mark.parametrize("lens", [[0, 0, 0], [1, 0, 700], [16, 17, 15], [64, 65, 700], [-3, 900, 128]])
def test_scan_lengths_and_nan_in_the_padding(lens, N):
    """Segments (few channels, many tokens) that lie before, across and past a sequence's end; what stands in the
    padding is never used; lengths are taken into 0..L."""
    print(f"[scan] lengths {lens} N={N}", flush=True)
    L = 700
    c = scan_case(9, 3, L, 40, N, 1, kind="f32", start=True)
    import ctypes
    lib = ctypes.CDLL(cls.LIB_PATH)
    lib.selective_scan_workspace_size.argtypes = [ctypes.c_int64] * 5
    lib.selective_scan_workspace_size.restype = ctypes.c_size_t
    assert lib.selective_scan_workspace_size(3, L, 40, N, 1) > 0
    c["seqlens"] = torch.tensor(lens, dtype=torch.int32)
    for i, n in enumerate(lens):
        for k in ("u", "dt", "z", "B", "C", "dy"):
            c[k][i, max(0, min(n, L)):] = math.nan
    check = dict(c)
    for k in ("u", "dt", "z", "B", "C", "dy"):
        check[k] = torch.nan_to_num(c[k], nan=0.0)
    d = on_gpu(c)
    y, h, kept = cls.selective_scan(*(d[k] for k in SCAN_KEYS), want_checkpoints=True)
    grads = cls.selective_scan_bwd(d["dy"], *(d[k] for k in SCAN_KEYS), checkpoints=kept, dh_final=d["dh"])
    a = oracle_args(check)
    ry, rh, ys, hs = osel.scan(**a)
    close(y, ry, ys, "y")
    close(h, rh, hs, "h")
    G, S = osel.scan_grads(f64(check["dy"]), **a, dh=f64(c["dh"]))
    for k, v in grads.items():
        close(v, G[k], S[k], k)
    for i, n in enumerate(lens):
        for v in (y, grads["du"], grads["ddt"], grads["dz"], grads["dB"], grads["dC"]):
            assert not v[i, max(0, min(n, L)):].any()


def test_scan_long_sequence_in_segments():
    """A sequence of several thousand tokens in many segments, against the oracle's token loop."""
    check_scan(scan_case(11, 1, 3001, 20, 16, 1, kind="f32", start=True), label="long")


def test_scan_extreme_steps():
    """Steps that forget everything at once, steps near zero, and dt far into both tails of softplus."""
    c = scan_case(12, 2, 60, 64, 16, 1, kind="f32", start=True)
    c["dt"][:, ::7] = 60.0
    c["dt"][:, 3::7] = -40.0
    c["dt"][:, 5::11] = 0.0
    check_scan(c, label="extreme")
    y, _ = cls.selective_scan(*(on_gpu(c)[k] for k in SCAN_KEYS))
    assert torch.isfinite(y).all()


def test_scan_nan_stays_in_its_channel():
    c = scan_case(13, 1, 40, 80, 16, 1, kind="f32")
    clean, _ = cls.selective_scan(*(on_gpu(c)[k] for k in SCAN_KEYS))
    c["u"][0, 20, 5] = math.nan
    y, h = cls.selective_scan(*(on_gpu(c)[k] for k in SCAN_KEYS))
    assert y[0, 20:, 5].isnan().all() and h[0, 5].isnan().all()
    keep = torch.ones(80, dtype=torch.bool, device="cuda")
    keep[5] = False
    assert torch.equal(y[:, :, keep], clean[:, :, keep]) and torch.equal(y[0, :20, 5], clean[0, :20, 5])


def test_scan_inputs_shared_by_all_sequences():
    """B and C of one sequence expanded over the batch (batch stride 0), and one B for both groups (group stride 0)."""
    c = scan_case(14, 3, 30, 66, 8, 2, kind="f32")
    for k in ("B", "C"):
        c[k] = c[k][:1, :, :1].contiguous()
    d = on_gpu(c)
    wide = {k: d[k].expand(3, 30, 2, 8) for k in ("B", "C")}
    full = {k: v.contiguous() for k, v in wide.items()}
    one = cls.selective_scan(*({**d, **wide}[k] for k in SCAN_KEYS))
    two = cls.selective_scan(*({**d, **full}[k] for k in SCAN_KEYS))
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])


def test_scan_rows_far_apart():
    """Sequences and tokens whose offsets pass 32 bits (in elements) within a large buffer."""
    c = scan_case(17, 2, 70, 64, 16, 1, kind="bf16")
    d = on_gpu(c)
    base = torch.empty((1 << 32) + 70 * (1 << 25), dtype=torch.bfloat16, device="cuda")

    def far(v, at):
        f = base[at:].as_strided(v.shape, ((1 << 32), 1 << 25, *v.stride()[2:])) if v.dim() == 3 else base[at:].as_strided(
            v.shape, (1 << 32, 1 << 25, 16, 1))
        f.copy_(v)
        return f

    wide = {k: far(d[k], i * 4096) for i, k in enumerate(("u", "dt", "z", "B", "C", "dy"))}
    runs = []
    for a in (d, {**d, **wide}):
        args = [a[k] for k in SCAN_KEYS]
        y, h, kept = cls.selective_scan(*args, want_checkpoints=True)
        runs.append([y, h, *cls.selective_scan_bwd(a["dy"], *args, checkpoints=kept).values()])
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_scan_same_bits_every_run_and_stale_memory():
    """Gradients, too: no atomics.  Workspaces and outputs come from memory that held something else."""
    c = on_gpu(scan_case(15, 2, 400, 100, 16, 1, kind="bf16", start=True, ragged=True))
    first = None
    for i in range(20):
        junk = torch.full((1 << 22,), math.nan, device="cuda")
        del junk
        y, h, kept = cls.selective_scan(*(c[k] for k in SCAN_KEYS), want_checkpoints=True)
        grads = cls.selective_scan_bwd(c["dy"], *(c[k] for k in SCAN_KEYS), checkpoints=kept)
        got = [y, h, *(grads[k] for k in sorted(grads))]
        assert not any(torch.isnan(v).any() for v in got)
        first = first or [v.clone() for v in got]
        assert all(torch.equal(a, b) for a, b in zip(got, first)), i


def test_scan_on_a_side_stream_and_in_a_graph():
    c = on_gpu(scan_case(16, 2, 333, 96, 16, 1, kind="bf16", start=True))
    args = [c[k] for k in SCAN_KEYS]

    def step():
        y, h, kept = cls.selective_scan(*args, want_checkpoints=True)
        return [y, h, *cls.selective_scan_bwd(c["dy"], *args, checkpoints=kept).values()]

    want = [v.clone() for v in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        r1 = step()
    with torch.cuda.graph(g2):
        r2 = step()
    for k in range(3):
        c["u"].mul_(-1.0)  # a new input, then both graphs at once on streams of their own
        want = [v.clone() for v in step()]
        torch.cuda.synchronize()
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        with torch.cuda.stream(s1):
            g1.replay()
        with torch.cuda.stream(s2):
            g2.replay()
        torch.cuda.synchronize()
        for got in (r1, r2):
            assert all(torch.equal(a, b) for a, b in zip(got, want)), k


def test_scan_from_two_threads_at_once():
    """Two host threads, a stream each, over the same inputs: every call has a workspace of its own."""
    import threading
    c = on_gpu(scan_case(18, 2, 500, 80, 16, 1, kind="bf16", start=True))
    args = [c[k] for k in SCAN_KEYS]

    def step():
        y, h, kept = cls.selective_scan(*args, want_checkpoints=True)
        return [y, h, *cls.selective_scan_bwd(c["dy"], *args, checkpoints=kept).values()]

    want = step()
    torch.cuda.synchronize()
    bad = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(10):
                got = step()
                s.synchronize()
                bad.extend(i for i, (a, b) in enumerate(zip(got, want)) if not torch.equal(a, b))

    threads = [threading.Thread(target=work) for _ in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not bad


def test_outputs_given_by_the_caller():
    """Every entry point with `out` writes there and returns it; another shape or type is refused."""
    c = on_gpu(scan_case(19, 2, 30, 64, 16, 1, kind="bf16"))
    args = [c[k] for k in SCAN_KEYS]
    y, _ = cls.selective_scan(*args)
    out = torch.empty_like(y)
    got, _ = cls.selective_scan(*args, out=out)
    assert got.data_ptr() == out.data_ptr() and torch.equal(out, y)
    w = torch.randn(64, 4, device="cuda")
    y, _ = cls.short_conv(c["u"], w)
    got, _ = cls.short_conv(c["u"], w, out=out)
    assert got.data_ptr() == out.data_ptr() and torch.equal(out, y)
    with pytest.raises(ValueError):
        cls.short_conv(c["u"], w, out=out[:, :5])
    with pytest.raises(ValueError):
        cls.short_conv(c["u"], w, out=torch.empty(2, 30, 128, dtype=torch.bfloat16, device="cuda")[..., :64])


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("nb,ch,N,G", [(1, 1, 1, 1), (3, 65, 16, 1), (2, 48, 5, 2), (5, 130, 20, 1), (2, 64, 64, 4),
                                       (70, 192, 16, 1), (2, 24, 3, 3),
                                       (87, 3001, 16, 1), (50, 2700, 18, 1)])
def test_scan_step(nb, ch, N, G, kind):
    print(f"[scan step] {nb} {ch} {N} {G} {kind}", flush=True)
    c = scan_case(20 + nb + N, nb, 1, ch, N, G, kind=kind, start=True)
    d = on_gpu(c)
    h = d["h0"].clone()
    one = lambda k: None if d[k] is None else d[k][:, 0]  # noqa: E731
    y = cls.selective_scan_step(h, one("u"), one("dt"), d["A"], one("B"), one("C"), d["D"], z=one("z"),
                                dt_bias=d["dt_bias"])
    ry, rh, ys, hs = osel.scan(**oracle_args(c))
    close(y[:, None], ry, ys, "y")
    close(h, rh, hs, "h")
    h = d["h0"].clone()
    y = cls.selective_scan_step(h, one("u"), one("dt").abs(), d["A"], one("B"), one("C"), dt_softplus=False)
    a = oracle_args(c)
    a.update(dt=np.abs(a["dt"]), D=None, z=None, dt_bias=None)
    ry, rh, ys, hs = osel.scan(**a, softplus=False)
    close(y[:, None], ry, ys, "plain y")
    close(h, rh, hs, "plain h")


# ---------------------------------------------------------------------------
# short convolution
# ---------------------------------------------------------------------------
def conv_case(seed, nb, L, ch, W, kind, bias=True, start=True, ragged=False, odd=False):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    dt_ = KINDS[kind]
    first = 1 if odd else 8  # an odd first channel leaves no row on 16 bytes
    return dict(x=rn(nb, L, ch + 16).to(dt_)[..., first:first + ch], weight=rn(ch, W), bias=rn(ch) if bias else None,
                initial_state=rn(nb, W - 1, ch).to(dt_) if start else None,
                seqlens=torch.randint(0, L + 1, (nb,), generator=g).to(torch.int32) if ragged else None,
                dy=rn(nb, L, ch + 8).to(dt_)[..., :ch], dfinal=rn(nb, W - 1, ch).to(dt_))


def check_conv(c, silu=True, label="", stuffed=None):
    d = on_gpu(stuffed or c)
    keys = ("x", "weight", "bias", "initial_state", "seqlens")
    y, last = cls.short_conv(*(d[k] for k in keys), silu=silu)
    grads = cls.short_conv_bwd(d["dy"], *(d[k] for k in keys), silu=silu, dfinal_state=d["dfinal"])
    a = {k: f64(c[k]) for k in keys[:4]}
    a["seqlens"] = None if c["seqlens"] is None else c["seqlens"].numpy()
    ry, rl, ys = osel.conv(**a, silu_on=silu)
    close(y, ry, ys, label + " y")
    assert np.array_equal(f64(last), rl), label
    G, S = osel.conv_grads(f64(c["dy"]), **a, silu_on=silu, dfinal=f64(c["dfinal"]))
    assert set(grads) == {"dx", "dweight"} | ({"dbias"} if c["bias"] is not None else set()) | (
        {"dinitial_state"} if c["initial_state"] is not None else set())
    for k, v in grads.items():
        close(v, G[k], S[k], f"{label} {k}")
    return y, grads


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("nb,L,ch,W", [(1, 1, 1, 4), (2, 2, 8, 4), (3, 7, 64, 3), (1, 33, 24, 2), (2, 100, 72, 4),
                                       (1, 65, 13, 4), (2, 9, 130, 2)])
def test_conv(nb, L, ch, W, kind):
    print(f"[conv] {nb} {L} {ch} {W} {kind}", flush=True)
    check_conv(conv_case(30 + L, nb, L, ch, W, kind), label=f"{nb} {L} {ch} {W} {kind}")


@pytest.mark.parametrize("nb,L,ch,W", [(4, 2050, 2048, 4), (1, 4097, 513, 3), (8, 2053, 2050, 4), (4, 2050, 1028, 2)])
def test_conv_in_longer_runs(nb, L, ch, W):
    """Enough work for runs of 8 and 16 tokens forward, in whole vectors and channel by channel."""
    print(f"[conv] {nb} {L} {ch} {W}", flush=True)
    check_conv(conv_case(35, nb, L, ch, W, "bf16", ragged=True), label=f"{nb} {L} {ch} {W}")


def test_conv_in_vectors_of_eight():
    """Enough 16-bit channels for vectors of 8: each token is that of its sequence alone, which runs in other vectors."""
    g = torch.Generator(device="cuda").manual_seed(37)
    nb, L, ch, W = 5, 8201, 1640, 4
    assert nb * (ch // 8) * ((L + 15) // 16) >= 1 << 19 > (ch // 8) * ((L + 15) // 16)
    x = torch.randn(nb, L, ch, generator=g, device="cuda").bfloat16()
    w, b = torch.randn(ch, W, generator=g, device="cuda"), torch.randn(ch, generator=g, device="cuda")
    start = torch.randn(nb, W - 1, ch, generator=g, device="cuda").bfloat16()
    lens = torch.tensor([L, 0, 17, 5000, L - 1], dtype=torch.int32, device="cuda")
    y, last = cls.short_conv(x, w, b, start, lens)
    for i in range(nb):
        y1, last1 = cls.short_conv(x[i:i + 1], w, b, start[i:i + 1], lens[i:i + 1])
        assert torch.equal(y[i:i + 1], y1) and torch.equal(last[i:i + 1], last1), i


def test_conv_gradients_in_long_runs():
    """Enough work for backward runs of 32 tokens, against float64 on whole tensors."""
    g = torch.Generator(device="cuda").manual_seed(36)
    nb, L, ch, W = 2, 4101, 4100, 4
    x, dy = (torch.randn(nb, L, ch, generator=g, device="cuda") for _ in range(2))
    w, b = torch.randn(ch, W, generator=g, device="cuda"), torch.randn(ch, generator=g, device="cuda")
    got = cls.short_conv_bwd(dy, x, w, b)
    pad = torch.zeros(nb, W - 1, ch, dtype=torch.float64, device="cuda")
    xp = torch.cat([pad, x.double()], 1)
    p = b.double() + sum(w[:, k].double() * xp[:, k:k + L] for k in range(W))
    s = torch.sigmoid(p)
    dp = dy.double() * s * (1 + p * (1 - s))
    dpp = torch.cat([dp, pad], 1)
    dx = sum(w[:, k].double() * dpp[:, W - 1 - k:W - 1 - k + L] for k in range(W))
    # dp: 16 u of its largest term, the W + 2 roundings of p through a slope below 1/2; then W products and sums
    big = sum(w[:, k].double().abs() * xp[:, k:k + L].abs() for k in range(W)) + b.double().abs()
    e = dy.double().abs() * (16 * s * (1 + p.abs()) + 0.5 * (W + 2) * big)
    ep, ap = (torch.cat([v, pad], 1) for v in (e, dp.abs()))
    bound = sum(w[:, k].double().abs() * (ep + 8 * ap)[:, W - 1 - k:W - 1 - k + L] for k in range(W))
    assert ((got["dx"].double() - dx).abs() <= 2 * U * bound + U * dx.abs()).all()
    for k in range(W):
        want, terms = (dp * xp[:, k:k + L]).sum((0, 1)), (dp * xp[:, k:k + L]).abs().sum((0, 1))
        err = (e * xp[:, k:k + L].abs()).sum((0, 1))
        # sums of 512 parts of 32 tokens: at most 640 additions deep
        assert ((got["dweight"][:, k].double() - want).abs() <= 2 * U * (err + 640 * terms)).all(), k
    assert ((got["dbias"].double() - dp.sum((0, 1))).abs() <= 2 * U * (e + 640 * dp.abs()).sum((0, 1))).all()


@pytest.mark.parametrize("off", ["bias", "start", "silu", "aligned", "none"])
def test_conv_options(off):
    print(f"[conv] without {off}", flush=True)
    c = conv_case(31, 4, 70, 40, 4, "bf16", bias=off != "bias", start=off != "start", ragged=True, odd=off == "aligned")
    check_conv(c, silu=off != "silu", label=off)


def test_conv_lengths_and_nan_in_the_padding():
    c = conv_case(32, 6, 70, 16, 4, "f32")
    c["seqlens"] = torch.tensor([0, 1, 2, 35, 70, 64], dtype=torch.int32)
    nan = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in c.items()}
    for i, n in enumerate(c["seqlens"].tolist()):
        nan["x"][i, n:] = math.nan
        nan["dy"][i, n:] = math.nan
    y, grads = check_conv(c, stuffed=nan, label="padding")
    for i, n in enumerate(c["seqlens"].tolist()):
        assert not y[i, n:].any() and not grads["dx"][i, n:].any()


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("nb,ch,W", [(1, 1, 2), (3, 72, 4), (5, 13, 3), (64, 200, 4)])
def test_conv_steps_are_the_prompt(nb, ch, W, kind):
    print(f"[conv step] {nb} {ch} {W} {kind}", flush=True)
    c = on_gpu(conv_case(33, nb, 6, ch, W, kind))
    y, last = cls.short_conv(c["x"], c["weight"], c["bias"], c["initial_state"])
    state = c["initial_state"].clone()
    steps = [cls.short_conv_step(state, c["x"][:, t], c["weight"], c["bias"]) for t in range(6)]
    assert torch.equal(torch.stack(steps, 1), y) and torch.equal(state, last)


def test_conv_same_bits_every_run_and_in_a_graph():
    c = on_gpu(conv_case(34, 3, 500, 96, 4, "bf16", ragged=True))
    args = (c["x"], c["weight"], c["bias"], c["initial_state"], c["seqlens"])
    step = lambda: [*cls.short_conv(*args), *cls.short_conv_bwd(c["dy"], *args).values()]  # noqa: E731
    want = [v.clone() for v in step()]
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(step(), want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for _ in range(3):
        c["dy"].mul_(-0.5)
        want = [v.clone() for v in step()]
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ---------------------------------------------------------------------------
# 8-bit cache
# ---------------------------------------------------------------------------
CACHE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (3, 5, 16), (2, 4, 64, 128), (2, 7, 3), (4, 33, 256), (2, 9, 100),
                                   (3, 70, 20), (1, 3, 250), (2, 64, 8), (2, 40, 64), (37, 1003, 100)])
def test_cache_bytes_and_scales(shape, kind):
    print(f"[cache] {shape} {kind}", flush=True)
    g = torch.Generator().manual_seed(40 + sum(shape))
    h = torch.randn(*shape, generator=g) * torch.exp(2 * torch.randn(*shape[:-1], 1, generator=g))
    h.view(-1, shape[-1])[0] = 0.0
    if shape[1] > 3:
        h[0, 1], h[0, 2] = h[0, 1] * 1e-33, h[0, 2] * 1e30
    nslots = shape[0] + 3
    cache = torch.randint(-100, 100, (nslots, *shape[1:]), generator=g).to(torch.int8).cuda().view(CACHE[kind])
    scales = torch.full((nslots, *shape[1:-1]), 7.0, device="cuda")
    before = cache.view(torch.int8).clone()
    slots = torch.randperm(nslots, generator=g)[:shape[0]].to(torch.int32)
    cls.state_cache_write(h.cuda(), cache, scales, slots.cuda())
    q, s = osel.cache_rows(h.numpy(), kind)
    at = slots.numpy()
    assert np.array_equal(scales.cpu().numpy()[at], s)
    assert np.array_equal(cache.float().cpu().numpy()[at], q.astype(np.float32))
    rest = [i for i in range(nslots) if i not in at.tolist()]
    assert torch.equal(cache.view(torch.int8)[rest], before[rest]) and (scales[rest] == 7.0).all()
    back = cls.state_cache_read(cache, scales, slots.cuda())
    want = (q.astype(np.float32) * s[..., None]).astype(np.float32)
    assert np.array_equal(back.cpu().numpy(), want)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_cache_slots_out_of_range_and_named_twice(kind):
    h = torch.randn(6, 300, 16, generator=torch.Generator().manual_seed(41)).cuda()
    cache = torch.zeros(3, 300, 16, dtype=CACHE[kind], device="cuda")
    scales = torch.zeros(3, 300, device="cuda")
    slots = torch.tensor([2, -1, 2, 0, 3, 2], dtype=torch.int32, device="cuda")
    cls.state_cache_write(h, cache, scales, slots)
    one, ones = torch.zeros_like(cache), torch.zeros_like(scales)
    cls.state_cache_write(h[[3, 5]], one, ones, torch.tensor([0, 2], dtype=torch.int32, device="cuda"))
    assert torch.equal(cache.view(torch.int8), one.view(torch.int8)) and torch.equal(scales, ones)
    back = cls.state_cache_read(cache, scales, torch.tensor([2, -1, 3, 2, 1], dtype=torch.int32, device="cuda"))
    assert torch.equal(back[0], back[3]) and back[0].any() and not back[1].any() and not back[2].any()
    assert not back[4].any()


def test_cache_past_32_bits():
    """Slots whose bytes lie beyond 4 GiB."""
    nslots, rows, S = 70000, 4096, 16
    cache = torch.empty(nslots, rows, S, dtype=torch.int8, device="cuda")
    scales = torch.empty(nslots, rows, device="cuda")
    h = torch.randn(2, rows, S, generator=torch.Generator().manual_seed(43)).cuda()
    slots = torch.tensor([nslots - 1, 0], dtype=torch.int32, device="cuda")
    cls.state_cache_write(h, cache, scales, slots)
    small, smalls = torch.zeros(2, rows, S, dtype=torch.int8, device="cuda"), torch.zeros(2, rows, device="cuda")
    cls.state_cache_write(h, small, smalls, torch.tensor([0, 1], dtype=torch.int32, device="cuda"))
    assert torch.equal(cache[nslots - 1], small[0]) and torch.equal(cache[0], small[1])
    back = cls.state_cache_read(cache, scales, slots)
    assert torch.equal(back, cls.state_cache_read(small, smalls, torch.tensor([0, 1], dtype=torch.int32, device="cuda")))


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_cache_rows_that_are_not_finite(kind, bad):
    h = torch.randn(1, 4, 16, generator=torch.Generator().manual_seed(42))
    h[0, 1, 3] = bad
    cache, scales = torch.zeros(1, 4, 16, dtype=CACHE[kind], device="cuda"), torch.zeros(1, 4, device="cuda")
    slots = torch.zeros(1, dtype=torch.int32, device="cuda")
    cls.state_cache_write(h.cuda(), cache, scales, slots)
    back = cls.state_cache_read(cache, scales, slots)
    assert back[0, 1].isnan().all() and torch.isfinite(back[0, [0, 2, 3]]).all()


# ---------------------------------------------------------------------------
# together, and refusals
# ---------------------------------------------------------------------------
def test_a_layer_s_prompt_snapshot_and_decoding():
    """Convolution and scan over a padded batch of prompts, the states kept in the cache and read back, then decoding
    token by token from them: the whole equals the oracle's over each sequence, with the states rounded to 8 bits
    in between."""
    nb, L, more, ch, N = 3, 50, 5, 72, 16
    lens = torch.tensor([50, 13, 1], dtype=torch.int32)
    c = scan_case(50, nb, L + more, ch, N, 1, kind="f32")
    w = conv_case(51, nb, L + more, ch, 4, "f32")
    d, e = on_gpu(c), on_gpu(w)
    cut = lambda v: v[:, :L]  # noqa: E731
    x, cs = cls.short_conv(cut(e["x"]), e["weight"], e["bias"], seqlens=lens.cuda())
    y, h = cls.selective_scan(x, cut(d["dt"]), d["A"], cut(d["B"]), cut(d["C"]), d["D"], z=cut(d["z"]),
                              dt_bias=d["dt_bias"], seqlens=lens.cuda())
    cache = torch.zeros(5, ch, N, dtype=torch.int8, device="cuda")
    scales = torch.zeros(5, ch, device="cuda")
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    cls.state_cache_write(h, cache, scales, slots)
    hd = cls.state_cache_read(cache, scales, slots)
    a, cw = oracle_args(c), {k: f64(w[k]) for k in ("x", "weight", "bias")}
    rx, rc, _ = osel.conv(cw["x"][:, :L], cw["weight"], cw["bias"], seqlens=lens.numpy())
    assert np.array_equal(f64(cs), rc)
    pa = {**a, "u": f64(x), "seqlens": lens.numpy(), **{k: a[k][:, :L] for k in ("dt", "z", "B", "C")}}
    ry, rh, ys, hs = osel.scan(**pa)
    close(y, ry, ys, "prompt y")
    close(h, rh, hs, "prompt h")
    q, s = osel.cache_rows(h.cpu().numpy(), "int8")
    assert np.array_equal(hd.cpu().numpy(), (q.astype(np.float32) * s[..., None]))
    start = f64(hd)
    xs, ys_, us = [], [], []
    for t in range(L, L + more):
        xt = cls.short_conv_step(cs, e["x"][:, t], e["weight"], e["bias"])
        yt = cls.selective_scan_step(hd, xt, d["dt"][:, t], d["A"], d["B"][:, t], d["C"][:, t], d["D"], z=d["z"][:, t],
                                     dt_bias=d["dt_bias"])
        us.append(f64(xt))
        ys_.append(yt)
    ta = {**a, "u": np.stack(us, 1), "h0": start, **{k: a[k][:, L:] for k in ("dt", "z", "B", "C")}}
    ry, rh, sy, sh = osel.scan(**ta)
    close(torch.stack(ys_, 1), ry, sy, "decoded y")
    close(hd, rh, sh, "decoded h")


def test_ssd_states_through_the_cache():
    """A prefix's SSD state kept in 8 bits and read back as the rest's h0."""
    g = torch.Generator().manual_seed(52)
    nb, L, H, P, S = 2, 128, 4, 64, 128
    x = torch.randn(nb, 2 * L, H, P, generator=g).to(torch.bfloat16).cuda()
    B, C = (torch.randn(nb, 2 * L, 1, S, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    dt = torch.nn.functional.softplus(torch.randn(nb, 2 * L, H, generator=g) - 2).cuda()
    A = -torch.exp(torch.rand(H, generator=g)).cuda()
    part = lambda v, k: v[:, k * L:(k + 1) * L].contiguous()  # noqa: E731
    _, h = cls.ssd_fwd(part(x, 0), part(dt, 0), A, part(B, 0), part(C, 0), chunk=128)
    cache = torch.zeros(4, H, P, S, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.zeros(4, H, P, device="cuda")
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    cls.state_cache_write(h, cache, scales, slots)
    h0 = cls.state_cache_read(cache, scales, slots)
    bound = torch.maximum(h.abs() * 2.0 ** -4, h.abs().amax(-1, keepdim=True) / 448 * 2.0 ** -10)
    assert ((h0 - h).abs() <= bound * (1 + 1e-6)).all()
    y, _ = cls.ssd_fwd(part(x, 1), part(dt, 1), A, part(B, 1), part(C, 1), None, h0, chunk=128)
    ry, _ = ossd.ssd_loop(*(f64(v) for v in (part(x, 1), part(dt, 1), A, part(B, 1), part(C, 1))), None, f64(h0))
    assert np.linalg.norm(f64(y) - ry) <= 2e-2 * np.linalg.norm(ry)


def test_binding_refuses_bad_tensors():
    c = on_gpu(scan_case(60, 2, 9, 16, 4, 2, kind="bf16", start=True))
    args = {k: c[k] for k in SCAN_KEYS}
    run = lambda **k: cls.selective_scan(**{**args, **k})  # noqa: E731
    for k, v, err in (("dt", c["dt"].float(), TypeError), ("z", c["z"][:, :8], ValueError),
                      ("B", c["B"][..., :3], ValueError), ("C", c["C"].cpu(), ValueError),
                      ("A", c["A"].double(), TypeError), ("A", c["A"].t(), ValueError),
                      ("D", c["D"][:8], ValueError), ("h0", c["h0"].half(), TypeError),
                      ("h0", c["h0"].transpose(1, 2), ValueError), ("u", c["u"].transpose(1, 2), ValueError),
                      ("seqlens", torch.zeros(2, dtype=torch.int64, device="cuda"), TypeError),
                      ("seqlens", torch.zeros(3, dtype=torch.int32, device="cuda"), ValueError),
                      ("out", torch.empty(2, 9, 16, device="cuda"), TypeError)):
        with pytest.raises(err):
            run(**{k: v})
    with pytest.raises(ValueError, match="checkpoints"):
        cls.selective_scan_bwd(c["dy"], **args)
    with pytest.raises(ValueError, match="checkpoints"):
        cls.selective_scan_bwd(c["dy"], **args, checkpoints=torch.zeros(2, 3, 4, 16, device="cuda"))
    with pytest.raises(cls.SSDError):
        big = torch.zeros(2, 9, 1, 65, dtype=torch.bfloat16, device="cuda")
        cls.selective_scan(c["u"], c["dt"], torch.zeros(16, 65, device="cuda"), big, big)
    with pytest.raises(cls.SSDError):
        cls.short_conv(c["u"], torch.zeros(16, 5, device="cuda"))
    with pytest.raises(cls.SSDError):
        cls.short_conv(c["u"][:, :0], torch.zeros(16, 4, device="cuda"))
    h = torch.zeros(2, 16, 4, device="cuda")
    cache, scales = torch.zeros(3, 16, 4, dtype=torch.int8, device="cuda"), torch.zeros(3, 16, device="cuda")
    slots = torch.zeros(2, dtype=torch.int32, device="cuda")
    for bad in ((h[:1], cache, scales, slots), (h, cache.float(), scales, slots), (h, cache, scales[:2], slots),
                (h, cache, scales, slots.long()), (h.half(), cache, scales, slots), (h, cache, scales, slots[:0])):
        with pytest.raises((ValueError, TypeError, cls.SSDError)):
            cls.state_cache_write(*bad)
