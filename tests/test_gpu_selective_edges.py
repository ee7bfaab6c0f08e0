"""GPU tests of the selective operators where the calls of test_gpu_selective.py do
not go: decays above 1, sizes beyond the usual, rows on and off whole vectors, and
how the functions stand beside autograd.  Oracle and tolerances are those of that
file."""
import numpy as np
import pytest
import torch

import chunked_linear_scan_amd as cls
from oracle import selective as osel
from test_gpu_selective import (SCAN_KEYS, check_scan, close, conv_case, f64, on_gpu, oracle_args, scan_case)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# decays above 1
# ---------------------------------------------------------------------------
def scan_both_ways(c, label):
    """Forward and backward of steps given as they are, without a gradient of the final state."""
    d = on_gpu(c)
    args = [d[k] for k in SCAN_KEYS]
    y, h, kept = cls.selective_scan(*args, dt_softplus=False, want_checkpoints=True)
    grads = cls.selective_scan_bwd(d["dy"], *args, dt_softplus=False, checkpoints=kept)
    a = oracle_args(c)
    ry, rh, ys, hs = osel.scan(**a, softplus=False)
    close(y, ry, ys, label + " y")
    close(h, rh, hs, label + " h")
    G, S = osel.scan_grads(f64(c["dy"]), **a, softplus=False)
    for k, v in grads.items():
        close(v, G[k], S[k], f"{label} {k}")


def growing_case(seed, L, N, sign):
    """Decays exp(dt A) with A > 0 (sign 1), or with A < 0 and negative steps (sign -1)."""
    c = scan_case(seed, 1, L, 8, N, 1, kind="f32", gate=False, bias=False, softplus=False)
    c["A"] = sign * (0.5 + 0.5 * torch.rand(8, N, generator=torch.Generator().manual_seed(seed)))
    c["dt"] = torch.full((1, L, 8), 0.01 * sign)
    c["dy"] = c["dy"].contiguous()
    return c


@pytest.mark.parametrize("N", [4, 16])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("L", [120, 1024])  # in one piece, and in segments of some 40 tokens
def test_scan_growth_of_a_zero_state(L, sign, N):
    """A hundred steps whose decays multiply to infinity in 32 bits, over a state (or, backward, a gradient) that is
    zero and stays it.  Even channels: at the start, where no input has come yet; odd ones: at the end, where no
    gradient has."""
    print(f"[scan] zero state, {L} tokens, sign {sign}, N={N}", flush=True)
    c = growing_case(70, L, N, sign)
    c["dt"][:, :100, ::2] = 6.0 * sign
    c["u"][:, :100, ::2] = 0.0
    c["dy"][:, :, ::2] = 0.0
    c["dt"][:, L - 100:, 1::2] = 6.0 * sign
    c["u"][:, :, 1::2] = 0.0
    c["dy"][:, L - 100:, 1::2] = 0.0
    scan_both_ways(c, f"zero state {L} {sign}")


@pytest.mark.parametrize("N", [4, 16])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("L", [120, 1024])
def test_scan_growth_of_a_tiny_state(L, sign, N):
    """States of 1e-30 that grow by more than 32 bits hold, to values that they hold; gradients likewise."""
    print(f"[scan] tiny state, {L} tokens, sign {sign}, N={N}", flush=True)
    c = growing_case(71, L, N, sign)
    g = torch.Generator().manual_seed(72)
    c["A"] = torch.full((8, N), 1.0 * sign) + 0.02 * torch.rand(8, N, generator=g) * sign
    c["h0"] = 1e-30 * torch.randn(1, 8, N, generator=g)
    c["u"].zero_()
    c["dt"].zero_()
    grow = slice(0, 100) if L == 120 else slice(42, 78)  # within one segment of 40 to 79
    c["dt"][:, grow] = (104.0 + torch.rand(1, 1, 8, generator=g)) / (grow.stop - grow.start) * sign
    c["dy"] *= 1e-30
    scan_both_ways(c, f"tiny state {L} {sign}")


# ---------------------------------------------------------------------------
# large sizes
# ---------------------------------------------------------------------------
def test_scan_of_many_sequences():
    """More sequences and channels than any cut of them; those picked equal the oracle."""
    nb, ch, N = 4096, 5120, 16
    some = [0, 1, 2047, 4095]
    c = scan_case(73, len(some), 2, ch, N, 1, kind="bf16", start=True)
    d = on_gpu(c)
    full = {k: d[k] if d[k] is None or k in ("A", "D", "dt_bias") else
            torch.zeros(nb, *d[k].shape[1:], dtype=d[k].dtype, device="cuda") for k in SCAN_KEYS}
    for k, v in full.items():
        if v is not None and v is not d[k]:
            v[some] = d[k]
    y, h = cls.selective_scan(*(full[k] for k in SCAN_KEYS))
    ry, rh, ys, hs = osel.scan(**oracle_args(c))
    close(y[some], ry, ys, "y")
    close(h[some], rh, hs, "h")
    y[some], h[some] = 0, 0
    assert not y.any() and not h.any()


def test_step_of_many_sequences():
    """1024 sequences of 5120 channels and 64 states, 1.3 GB of them; those picked equal the oracle."""
    nb, ch, N = 1024, 5120, 64
    some = [0, 1, 511, 1023]
    c = scan_case(74, len(some), 1, ch, N, 1, kind="bf16", start=True)
    d = on_gpu(c)
    spread = lambda v: torch.zeros(nb, *v.shape[1:], dtype=v.dtype, device="cuda").index_copy_(  # noqa: E731
        0, torch.tensor(some, device="cuda"), v)
    h = spread(d["h0"])
    u, dt, z, B, C = (spread(d[k][:, 0]) for k in ("u", "dt", "z", "B", "C"))
    y = cls.selective_scan_step(h, u, dt, d["A"], B, C, d["D"], z=z, dt_bias=d["dt_bias"])
    ry, rh, ys, hs = osel.scan(**oracle_args(c))
    close(y[some][:, None], ry, ys, "y")
    close(h[some], rh, hs, "h")
    y[some], h[some] = 0, 0
    assert not y.any() and not h.any()


def test_step_on_states_sliced_from_more():
    """States of sequences past the first, which with an odd number of values to a sequence start between vectors."""
    c = scan_case(75, 4, 1, 5, 3, 1, kind="f32", start=True)
    d = on_gpu(c)
    h = d["h0"].clone()
    part = h[1:]
    assert part.is_contiguous() and part.data_ptr() % 16 != 0
    one = lambda k: d[k][1:, 0]  # noqa: E731
    y = cls.selective_scan_step(part, one("u"), one("dt"), d["A"], one("B"), one("C"), d["D"], z=one("z"),
                                dt_bias=d["dt_bias"])
    ry, rh, ys, hs = osel.scan(**oracle_args(c))
    close(y[:, None], ry[1:], ys[1:], "y")
    close(part, rh[1:], hs[1:], "h")
    assert torch.equal(h[0], d["h0"][0])
    off = torch.zeros(1 + 4 * 16, device="cuda")[1:].view(1, 4, 16)
    z4, z16 = torch.zeros(1, 4, device="cuda"), torch.zeros(1, 1, 16, device="cuda")
    with pytest.raises(cls.SSDError):  # rows of whole vectors, off them
        cls.selective_scan_step(off, z4, z4, torch.zeros(4, 16, device="cuda"), z16, z16)


# ---------------------------------------------------------------------------
# beside autograd
# ---------------------------------------------------------------------------
def layer_calls():
    """name: (call, the tensors it takes) of every function with floating-point outputs of its own."""
    c = on_gpu(scan_case(76, 2, 9, 16, 4, 1, kind="f32", start=True))
    A, D, w, b = c["A"], c["D"], torch.randn(16, 4, device="cuda"), torch.randn(16, device="cuda")
    state = torch.randn(2, 3, 16, device="cuda")
    t = {k: c[k][:, 0].contiguous() for k in ("u", "dt", "z", "B", "C")}
    return {
        "selective_scan": (lambda u, dt, A, B, C, D, z, bias, h0: cls.selective_scan(
            u, dt, A, B, C, D, z=z, dt_bias=bias, h0=h0),
            [c["u"], c["dt"], A, c["B"], c["C"], D, c["z"], c["dt_bias"], c["h0"]]),
        "selective_scan_step": (lambda u, dt, A, B, C, D, z, bias: (cls.selective_scan_step(
            c["h0"].clone(), u, dt, A, B, C, D, z=z, dt_bias=bias),),
            [t["u"], t["dt"], A, t["B"], t["C"], D, t["z"], c["dt_bias"]]),
        "short_conv": (lambda x, w, b, s: cls.short_conv(x, w, b, s), [c["u"], w, b, state]),
        "short_conv_step": (lambda x, w, b: (cls.short_conv_step(state.clone(), x, w, b),), [t["u"], w, b]),
    }


@pytest.mark.parametrize("name", ["selective_scan", "selective_scan_step", "short_conv", "short_conv_step"])
def test_a_gradient_is_not_lost_in_silence(name):
    """No function records a gradient: a backward pass that would need one raises, and says what to call."""
    call, tensors = layer_calls()[name]
    want = call(*tensors)
    assert not any(v.requires_grad for v in want)
    for i in range(len(tensors)):
        leaves = [v.clone().requires_grad_() if j == i else v for j, v in enumerate(tensors)]
        got = call(*leaves)
        for g, w in zip(got, want):
            assert g.requires_grad and torch.equal(g.detach(), w), (name, i)
            with pytest.raises(RuntimeError, match=f"{name} records no gradient"):
                g.sum().backward()
        with torch.no_grad():
            assert not any(v.requires_grad for v in call(*leaves))
    # the gradient functions take what requires gradients, and give plain tensors
    if name == "short_conv":
        leaves = [v.clone().requires_grad_() for v in tensors]
        grads = cls.short_conv_bwd(tensors[0], *leaves)
        assert not any(v.requires_grad for v in grads.values())


def test_writes_in_place_are_seen_by_autograd():
    """States, caches and given outputs are written in place: a backward pass that still needs what they held raises."""
    c = on_gpu(scan_case(77, 2, 9, 16, 4, 1, kind="f32", start=True))
    t = {k: c[k][:, 0].contiguous() for k in ("u", "dt", "z", "B", "C")}
    w, state = torch.randn(16, 4, device="cuda"), torch.randn(2, 3, 16, device="cuda")
    cache, scales = torch.zeros(3, 16, 4, dtype=torch.int8, device="cuda"), torch.zeros(3, 16, device="cuda")
    slots = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    h, out, out1 = c["h0"].clone(), torch.empty(2, 9, 16, device="cuda"), torch.empty(2, 16, device="cuda")
    back = torch.empty(2, 16, 4, device="cuda")
    scan = [c[k] for k in ("u", "dt", "A", "B", "C")]
    step = [t["u"], t["dt"], c["A"], t["B"], t["C"]]
    for call, written in ((lambda: cls.selective_scan_step(h, *step, out=out1), (h, out1)),
                          (lambda: cls.short_conv_step(state, t["u"], w, out=out1), (state, out1)),
                          (lambda: cls.selective_scan(*scan, out=out), (out,)),
                          (lambda: cls.short_conv(c["u"], w, out=out), (out,)),
                          (lambda: cls.state_cache_write(h, cache, scales, slots), (cache, scales)),
                          (lambda: cls.state_cache_read(cache, scales, slots, out=back), (back,))):
        before = [v._version for v in written]
        call()
        assert [v._version for v in written] == [v + 1 for v in before]
    x = torch.randn(2, 16, 4, device="cuda", requires_grad=True)
    loss = (x * h).sum()
    cls.selective_scan_step(h, *step)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():  # such tensors count no versions
        inner = torch.zeros(2, 16, 4, device="cuda")
    cls.selective_scan_step(inner, *step)
    assert inner.any()


def test_memory_that_runs_out_is_torch_s_error():
    """An output larger than the device (inputs expanded over the batch), as torch reports it for its own."""
    x = torch.zeros(1, 1 << 10, 1 << 10, device="cuda").expand(1 << 17, 1 << 10, 1 << 10)
    B = torch.zeros(1, 1, 1, 4, device="cuda").expand(1 << 17, 1 << 10, 1, 4)
    assert x.numel() * 4 > torch.cuda.get_device_properties(0).total_memory
    with pytest.raises(torch.OutOfMemoryError):
        cls.selective_scan(x, x, torch.zeros(1 << 10, 4, device="cuda"), B, B)
    with pytest.raises(torch.OutOfMemoryError):
        cls.short_conv(x, torch.zeros(1 << 10, 4, device="cuda"))


# ---------------------------------------------------------------------------
# rows on and off whole vectors
# ---------------------------------------------------------------------------
def step_case(seed, nb, ch, N, G, kind, first):
    """One token whose B and C stand in one row behind `first` columns, as in a layer's projection."""
    c = scan_case(seed, nb, 1, ch, N, G, kind=kind, start=True)
    bc = torch.randn(nb, 1, first + 2 * G * N, generator=torch.Generator().manual_seed(seed)).to(c["u"].dtype)
    c["B"] = bc[..., first:first + G * N].unflatten(-1, (G, N))
    c["C"] = bc[..., first + G * N:].unflatten(-1, (G, N))
    return c, bc


# one and four sequences to a thread (1024 workgroups), whole and partial groups of four
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("nb,ch,N,G", [(2, 70, 4, 1), (3, 64, 8, 2), (1, 1536, 16, 1), (6, 33, 20, 3), (5, 24, 32, 1),
                                       (3, 48, 64, 2), (301, 1200, 12, 1), (130, 2400, 16, 2), (99, 1504, 20, 1),
                                       (67, 1928, 32, 4), (50, 1280, 64, 1), (29, 2320, 52, 1)])
def test_step_in_whole_vectors(nb, ch, N, G, kind):
    print(f"[scan step] {nb} {ch} {N} {G} {kind}", flush=True)
    for first in (0, 48):
        c, bc = step_case(80 + nb, nb, ch, N, G, kind, first)
        d = on_gpu(c)
        wide = bc.cuda()
        d["B"] = wide[..., first:first + G * N].unflatten(-1, (G, N))
        d["C"] = wide[..., first + G * N:].unflatten(-1, (G, N))
        h = d["h0"].clone()
        one = lambda k: d[k][:, 0]  # noqa: E731
        size = 4 * d["B"].element_size()  # bytes of four states
        for v in (one("B"), one("C")):
            assert v.data_ptr() % size == 0 and all(s * v.element_size() % size == 0 for s in v.stride()[:2])
        assert N % 4 == 0 and d["A"].data_ptr() % 16 == 0 and h.data_ptr() % 16 == 0
        y = cls.selective_scan_step(h, one("u"), one("dt"), d["A"], one("B"), one("C"), d["D"], z=one("z"),
                                    dt_bias=d["dt_bias"])
        ry, rh, ys, hs = osel.scan(**oracle_args(c))
        close(y[:, None], ry, ys, f"y {first}")
        close(h, rh, hs, f"h {first}")


def off_vectors(v):
    """The same tensor one element past a whole vector, its strides unchanged."""
    need = 1 + sum((n - 1) * s for n, s in zip(v.shape, v.stride()))
    base = torch.empty(need + 1, dtype=v.dtype, device=v.device)
    assert base.data_ptr() % 16 == 0
    moved = base[1:].as_strided(v.shape, v.stride())
    moved.copy_(v)
    assert moved.data_ptr() % 8 == v.element_size()
    return moved


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("name", ["x", "dy", "initial_state", "dfinal", "weight", "bias", "out", "none"])
def test_conv_with_one_tensor_off_whole_vectors(name, kind):
    """Strides that keep every row on a vector, from a first element that is not on one."""
    print(f"[conv] {name} off {kind}", flush=True)
    c = conv_case(81, 3, 70, 48, 4, kind)
    c["x"], c["dy"] = c["x"].contiguous(), c["dy"].contiguous()
    c["seqlens"] = torch.tensor([70, 0, 31], dtype=torch.int32)
    d = on_gpu(c)
    out = torch.empty_like(d["x"])
    if name == "out":
        out = off_vectors(out)
    elif name != "none":
        d[name] = off_vectors(d[name])
    args = [d[k] for k in ("x", "weight", "bias", "initial_state", "seqlens")]
    y, last = cls.short_conv(*args, out=out)
    grads = cls.short_conv_bwd(d["dy"], *args, dfinal_state=d["dfinal"])
    a = {k: f64(c[k]) for k in ("x", "weight", "bias", "initial_state")}
    a["seqlens"] = c["seqlens"].numpy()
    ry, rl, ys = osel.conv(**a)
    close(y, ry, ys, "y")
    assert np.array_equal(f64(last), rl)
    G, S = osel.conv_grads(f64(c["dy"]), **a, dfinal=f64(c["dfinal"]))
    for k, v in grads.items():
        close(v, G[k], S[k], k)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("name", ["x", "state", "weight", "bias", "out", "none"])
def test_conv_step_with_one_tensor_off_whole_vectors(name, kind):
    print(f"[conv step] {name} off {kind}", flush=True)
    c = conv_case(85, 3, 1, 48, 4, kind)
    d = on_gpu(c)
    t = dict(x=d["x"][:, 0].contiguous(), weight=d["weight"], bias=d["bias"], state=d["initial_state"].clone())
    t["out"] = torch.empty_like(t["x"])
    if name != "none":
        t[name] = off_vectors(t[name])
    y = cls.short_conv_step(t["state"], t["x"], t["weight"], t["bias"], out=t["out"])
    ry, rl, ys = osel.conv(*(f64(c[k]) for k in ("x", "weight", "bias", "initial_state")))
    close(y[:, None], ry, ys, "y")
    assert np.array_equal(f64(t["state"]), rl)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_scan_with_every_tensor_off_whole_vectors(kind):
    c = scan_case(82, 2, 70, 48, 16, 2, kind=kind, start=True)
    d = on_gpu(c)
    moved = {k: off_vectors(v) if torch.is_tensor(v) and v.is_floating_point() else v for k, v in d.items()}
    runs = []
    for a in (d, moved):
        args = [a[k] for k in SCAN_KEYS]
        y, h, kept = cls.selective_scan(*args, want_checkpoints=True)
        runs.append([y, h, *cls.selective_scan_bwd(a["dy"], *args, checkpoints=kept, dh_final=a["dh"]).values()])
    assert all(torch.equal(a, b) for a, b in zip(*runs))


# ---------------------------------------------------------------------------
# segments
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("N,G", [(3, 1), (4, 2), (7, 3), (8, 1), (16, 2), (24, 2), (32, 1), (64, 2)])
def test_scan_in_segments(N, G, softplus):
    """Every number of waves to a workgroup, in segments, with groups and steps given as they are."""
    print(f"[scan] segments N={N} G={G} softplus={softplus}", flush=True)
    c = scan_case(83, 2, 333, 12, N, G, kind="f32", start=True, ragged=True, softplus=softplus)
    c["seqlens"][0] = 333
    check_scan(c, softplus=softplus, label=f"{N} {G} {softplus}")


def test_scan_in_the_most_segments():
    """8192 tokens of few channels: as many segments as there can be, and one sequence that ends in the first."""
    c = scan_case(84, 2, 8192, 3, 4, 1, kind="f32", start=True)
    c["seqlens"] = torch.tensor([8192, 5], dtype=torch.int32)
    check_scan(c, label="most segments")
