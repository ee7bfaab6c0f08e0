"""CPU pins of oracle/delta.py: closed forms, differences, and the chunk algebra
against the token loops."""
import numpy as np
import pytest

from oracle import delta as od


def case(seed, nb=2, L=23, Hk=1, H=2, dk=6, dv=5, start=True, ragged=False, strong=False):
    g = np.random.default_rng(seed)
    rn = g.standard_normal
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)  # noqa: E731
    c = dict(q=unit(rn((nb, L, Hk, dk))), k=unit(rn((nb, L, Hk, dk))), v=rn((nb, L, H, dv)),
             g=-np.abs(rn((nb, L, H))) * (5 if strong else 0.3), beta=1 / (1 + np.exp(-rn((nb, L, H)))),
             h0=rn((nb, H, dv, dk)) if start else None,
             seqlens=g.integers(0, L + 1, nb) if ragged else None)
    return c, rn((nb, L, H, dv)), rn((nb, H, dv, dk))


def test_orthogonal_keys_are_recalled():
    """Written with beta 1 and never faded, a value is read back by its key, times the scale."""
    n = 6
    k = np.eye(n)[None, :, None]
    v = np.random.default_rng(0).standard_normal((1, n, 1, 4))
    z, o = np.zeros((1, n, 1)), np.ones((1, n, 1))
    y, h = od.delta(k, k, v, z, o)
    assert np.allclose(y, v * n ** -0.5) and np.allclose(h[0, 0], v[0, :, 0].T)
    # the same key again: the value is replaced, not added to
    y, h = od.delta(np.repeat(k[:, :1], n, 1), np.repeat(k[:, :1], n, 1), v, z, o, scale=1.0)
    assert np.allclose(y, v) and np.allclose(h[0, 0][:, 0], v[0, -1, 0])


def test_beta_zero_only_fades_and_minus_infinity_forgets():
    c, _, _ = case(1)
    c["beta"][:] = 0
    _, h = od.delta(**c)
    assert np.allclose(h, c["h0"] * np.exp(c["g"].sum(1))[..., None, None])
    c, _, _ = case(2)
    c["g"][:, 9] = -np.inf
    y, h = od.delta(**c)
    cut = {k: (v[:, 9:] if k not in ("h0", "seqlens") else None) for k, v in c.items()}
    cut["g"] = cut["g"].copy()
    cut["g"][:, 0] = 0
    y2, h2 = od.delta(**cut)
    assert np.allclose(y[:, 9:], y2) and np.allclose(h, h2)


def test_additive_limit():
    """With orthogonal keys each written once the rule is a plain sum of outer products: linear attention."""
    c, _, _ = case(3, L=6, dk=6, start=False)
    c["k"][:] = np.eye(6)[None, :, None]
    y, _ = od.delta(**c)
    for b in range(2):
        for n in range(2):
            for t in range(6):
                s = sum(np.exp(c["g"][b, j + 1:t + 1, n].sum()) * c["beta"][b, j, n] * (c["k"][b, j, 0] @ c["q"][b, t, 0])
                        * c["v"][b, j, n] for j in range(t + 1))
                assert np.allclose(y[b, t, n], s * 6 ** -0.5)


@pytest.mark.parametrize("ragged", [False, True])
def test_gradients_against_differences(ragged):
    c, dy, dh = case(4, L=7, ragged=ragged)
    G = od.delta_grads(dy, **c, dh=dh)
    loss = lambda a: float(sum((o * d).sum() for o, d in zip(od.delta(**a), (dy, dh))))  # noqa: E731
    r = np.random.default_rng(5)
    for name in ("q", "k", "v", "g", "beta", "h0"):
        d = r.standard_normal(c[name].shape)
        step = 1e-6
        num = (loss({**c, name: c[name] + step * d}) - loss({**c, name: c[name] - step * d})) / (2 * step)
        got = float((G["d" + name] * d).sum())
        assert abs(num - got) <= 1e-7 * (1 + np.abs(G["d" + name] * d).sum()), (name, num, got)


@pytest.mark.parametrize("kind,C", [("bf16", 8), ("f32", 4), ("f16", 64)])
@pytest.mark.parametrize("ragged,strong", [(False, False), (True, True)])
def test_chunk_algebra_is_the_token_loop(kind, C, ragged, strong):
    c, dy, dh = case(6, Hk=2, H=4, ragged=ragged, strong=strong)
    val, err = od.delta_bounds(kind, C, **c, dy=dy, dh=dh)
    y, h = od.delta(**c)
    want = {"y": y, "h": h, **od.delta_grads(dy, **c, dh=dh)}
    assert set(val) == set(want)
    for n, w in want.items():
        assert np.allclose(val[n], w, atol=1e-12, rtol=1e-10), n
        assert (err[n] >= 0).all() and np.isfinite(err[n]).all()
        # a bound of use: far below the values themselves
        assert np.linalg.norm(err[n]) <= 60 * od.U1[kind] * np.linalg.norm(w) + 3e-3 * np.linalg.norm(w), n


def test_chunk_algebra_with_resets():
    c, dy, dh = case(7)
    c["g"][:, [0, 9, 10]] = -np.inf
    val, err = od.delta_bounds("f32", 8, **c, dy=dy, dh=dh)
    G = od.delta_grads(dy, **c, dh=dh)
    for n in G:
        assert np.allclose(val[n], G[n], atol=1e-12), n
        assert np.isfinite(err[n]).all()


@pytest.mark.parametrize("gate_first", [False, True])
@pytest.mark.parametrize("gate", [False, True])
def test_norm_gradients_against_differences(gate_first, gate):
    r = np.random.default_rng(8)
    x, z, w, dy = r.standard_normal((3, 2, 7)), r.standard_normal((3, 2, 7)), r.standard_normal(7), r.standard_normal((3, 2, 7))
    z = z if gate else None
    G, S = od.gated_norm_grads(dy, x, w, z, gate_first=gate_first)
    f = lambda **k: float((od.gated_norm(**{**dict(x=x, weight=w, z=z, gate_first=gate_first), **k})[0] * dy).sum())  # noqa: E731
    for name, v, key in (("x", x, "dx"), ("weight", w, "dweight")) + ((("z", z, "dz"),) if gate else ()):
        d = r.standard_normal(v.shape)
        num = (f(**{name: v + 1e-6 * d}) - f(**{name: v - 1e-6 * d})) / 2e-6
        assert abs(num - (G[key] * d).sum()) <= 1e-7, key
        assert (S[key] >= np.abs(G[key]) * (1 - 1e-12)).all()


def test_norm_rows_have_length_one_with_the_key_weight():
    x = np.random.default_rng(9).standard_normal((4, 2, 16))
    y, *_ = od.gated_norm(x, np.full(16, 16 ** -0.5), eps=0.0)
    assert np.allclose(np.linalg.norm(y, axis=-1), 1)


def test_residual_gradients_against_differences():
    r = np.random.default_rng(10)
    x, res, w, s, dy, dr = (r.standard_normal(n) for n in ((5, 6), (5, 6), 6, 6, (5, 6), (5, 6)))

    def f(x=x, res=res, w=w, s=s):
        stream, _ = od.residual_stream(x, res, s)
        return float((od.gated_norm(stream[:, None], w)[0][:, 0] * dy).sum() + (stream * dr).sum())

    stream, _ = od.residual_stream(x, res, s)
    G, _ = od.residual_norm_grads(dy, stream, w, dr=dr, x=x, scale=s)
    for name, v, key in (("x", x, "dx"), ("res", res, "dresidual"), ("w", w, "dweight"), ("s", s, "dscale")):
        d = r.standard_normal(v.shape)
        num = (f(**{name: v + 1e-6 * d}) - f(**{name: v - 1e-6 * d})) / 2e-6
        assert abs(num - (G[key] * d).sum()) <= 1e-7, key
