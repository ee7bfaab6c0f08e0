"""Pins of the selective scan's, the convolution's and the cache's oracle:
closed forms, the SSD oracle on shared decays, and finite differences of the
gradients in float64."""
import numpy as np
import pytest

from oracle import selective as osel, ssd as ossd


def case(seed, nb=2, L=7, ch=6, n=3, g=2):
    r = np.random.default_rng(seed)
    return dict(u=r.normal(size=(nb, L, ch)), dt=r.normal(size=(nb, L, ch)), A=-np.exp(r.normal(size=(ch, n))),
                B=r.normal(size=(nb, L, g, n)), C=r.normal(size=(nb, L, g, n)), D=r.normal(size=ch),
                z=r.normal(size=(nb, L, ch)), dt_bias=r.normal(size=ch), h0=r.normal(size=(nb, ch, n)))


def test_one_decay_per_channel_is_the_ssd_recurrence():
    """With A the same for all states and positive steps given as they are,
    each channel is an SSD head of dim 1."""
    c = case(0, n=4)
    dt = np.abs(c["dt"])
    A = np.repeat(c["A"][:, :1], 4, 1)
    y, h, _, _ = osel.scan(c["u"], dt, A, c["B"], c["C"], c["D"], h0=c["h0"], softplus=False)
    ry, rh = ossd.ssd_loop(c["u"][..., None], dt, A[:, 0], c["B"], c["C"], c["D"], c["h0"][:, :, None])
    assert np.allclose(y, ry[..., 0], rtol=1e-12, atol=1e-12) and np.allclose(h, rh[:, :, 0], rtol=1e-12, atol=1e-12)


def test_no_decay_is_a_running_sum():
    c = case(1, g=1)
    one = np.ones_like(c["B"])
    y, h, _, _ = osel.scan(c["u"], np.ones_like(c["dt"]), np.zeros_like(c["A"]), one, one, softplus=False)
    assert np.allclose(y, 3 * np.cumsum(c["u"], 1))
    assert np.allclose(h, np.cumsum(c["u"], 1)[:, -1][..., None])


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("seqlens", [None, [0, 5]])
def test_scan_gradients_against_differences(softplus, seqlens):
    c = case(2)
    r = np.random.default_rng(3)
    dy, dh = r.normal(size=c["u"].shape), r.normal(size=c["h0"].shape)

    def loss(**k):
        y, h, _, _ = osel.scan(**{**c, **k}, seqlens=seqlens, softplus=softplus)
        return (y * dy).sum() + (h * dh).sum()

    # Negative steps without softplus grow the states, and the difference of two large losses cancels: each loss is
    # off by at most 2^-53 of its terms' error scales and of the sum's own roundings, the quotient by that over e.
    y, h, ys, hs = osel.scan(**c, seqlens=seqlens, softplus=softplus)
    terms = np.abs(y * dy).sum() + np.abs(h * dh).sum()
    noise = 2.0 ** -53 * ((ys * np.abs(dy)).sum() + (hs * np.abs(dh)).sum() + (y.size + h.size) * terms) / 1e-6

    G, _ = osel.scan_grads(dy, **c, seqlens=seqlens, softplus=softplus, dh=dh)
    names = {"u": "du", "dt": "ddt", "A": "dA", "B": "dB", "C": "dC", "D": "dD", "z": "dz", "dt_bias": "ddt_bias",
             "h0": "dh0"}
    for k, name in names.items():
        v = r.normal(size=c[k].shape)
        e = 1e-6
        diff = (loss(**{k: c[k] + e * v}) - loss(**{k: c[k] - e * v})) / (2 * e)
        assert abs(diff - (G[name] * v).sum()) <= 1e-6 * (1 + abs(diff)) + noise, (name, noise)


@pytest.mark.parametrize("name,key", [("du", "u"), ("ddt", "dt"), ("dA", "A"), ("dB", "B"), ("dC", "C"), ("dD", "D"),
                                      ("dz", "z"), ("ddt_bias", "dt_bias"), ("dh0", "h0")])
def test_gradients_of_steps_given_as_they_are(name, key):
    """softplus off with positive steps (decays below 1), where differences do not cancel."""
    c = case(8)
    c["dt"], c["dt_bias"] = np.abs(c["dt"]) + 0.1, np.abs(c["dt_bias"])
    r = np.random.default_rng(9)
    dy, v, e = r.normal(size=c["u"].shape), r.normal(size=c[key].shape), 1e-6
    loss = lambda x: (osel.scan(**{**c, key: x}, softplus=False)[0] * dy).sum()  # noqa: E731
    G, _ = osel.scan_grads(dy, **c, softplus=False)
    diff = (loss(c[key] + e * v) - loss(c[key] - e * v)) / (2 * e)
    assert abs(diff - (G[name] * v).sum()) <= 1e-6 * (1 + abs(diff))


@pytest.mark.parametrize("silu_on", [True, False])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_gradients_against_differences(W, silu_on):
    r = np.random.default_rng(4)
    c = dict(x=r.normal(size=(3, 6, 5)), weight=r.normal(size=(5, W)), bias=r.normal(size=5),
             initial_state=r.normal(size=(3, W - 1, 5)))
    seqlens = [6, 0, 2]
    dy, df = r.normal(size=c["x"].shape), r.normal(size=c["initial_state"].shape)

    def loss(**k):
        y, last, _ = osel.conv(**{**c, **k}, seqlens=seqlens, silu_on=silu_on)
        return (y * dy).sum() + (last * df).sum()

    G, _ = osel.conv_grads(dy, **c, seqlens=seqlens, silu_on=silu_on, dfinal=df)
    for k, name in {"x": "dx", "weight": "dweight", "bias": "dbias", "initial_state": "dinitial_state"}.items():
        v = r.normal(size=c[k].shape)
        e = 1e-6
        diff = (loss(**{k: c[k] + e * v}) - loss(**{k: c[k] - e * v})) / (2 * e)
        assert abs(diff - (G[name] * v).sum()) <= 1e-6 * (1 + abs(diff)), name


def test_conv_of_pieces_is_the_conv_of_the_whole():
    r = np.random.default_rng(5)
    x, w, b = r.normal(size=(2, 9, 4)), r.normal(size=(4, 4)), r.normal(size=4)
    y, last, _ = osel.conv(x, w, b)
    y1, s1, _ = osel.conv(x[:, :2], w, b)
    y2, s2, _ = osel.conv(x[:, 2:], w, b, s1)
    assert np.allclose(np.concatenate([y1, y2], 1), y) and np.allclose(s2, last)


def test_e4m3_table_and_rounding():
    v = osel.e4m3_values()
    assert v[0x7e] == 448 and v[1] == 2.0 ** -9 and v[0x38] == 1 and np.isnan(v[0x7f])
    import torch
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(np.nan_to_num(t, nan=7e7), np.nan_to_num(v, nan=7e7).astype(np.float32))
    r = np.random.default_rng(6)
    h = (r.normal(size=(64, 40)) * np.exp(r.normal(size=(64, 1)))).astype(np.float32)
    q, s = osel.cache_rows(h, "e4m3")
    inv = np.float32(448) / np.abs(h).max(-1, keepdims=True)
    want = torch.from_numpy(h * inv).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(q.astype(np.float32), want)


@pytest.mark.parametrize("kind,step", [("int8", 0.5 / 127), ("e4m3", 2.0 ** -4)])
def test_cache_rows_stay_within_half_a_step(kind, step):
    r = np.random.default_rng(7)
    h = r.normal(size=(50, 16)).astype(np.float32)
    q, s = osel.cache_rows(h, kind)
    m = np.abs(h).max(-1, keepdims=True)
    back = q * s[..., None]
    bound = step * m if kind == "int8" else np.maximum(step * np.abs(h), m / 448 * 2.0 ** -10)
    assert (np.abs(back - h) <= bound * (1 + 1e-5)).all()
