"""Selective scan, short convolution and 8-bit state cache as plain float64
token loops, with error scales.  Test infrastructure only.

Every ``*_scale`` result bounds, to first order and in units of the fp32 unit
roundoff u = 2^-24, what rounding can do to the fp32 evaluation of the same
quantity: each elementary step contributes its own roundings and carries on
those of its factors.  The counts are those of the kernels' formulas, taken
generously: a step dt' = softplus(.) is within 8 u (exp2, log2, reciprocal of
1 ulp each, their products; the exponent's rounding, up to 1.5 |dt + dt_bias| u
of a step in the tail, is left to the tests' factor of two, which holds it down
to -8), a decay exp(dt' A) within (4 + 12 |dt' A|) u (the exponent carries dt's
error, its own two products and A's conversion), a factor silu or its derivative
within 16 u of its largest term.
"""
from __future__ import annotations

import numpy as np


def sigmoid(x):
    return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))


def silu(x):
    return x * sigmoid(x)


def dsilu(x):
    s = sigmoid(x)
    return s * (1 + x * (1 - s))


def _steps(dt, dt_bias, softplus):
    x = dt + (0.0 if dt_bias is None else dt_bias)
    return x, (np.logaddexp(0.0, x) if softplus else x)


def _groups(v, ch):
    """[batch, groups, n] -> [batch, channels, n]"""
    return np.repeat(v, ch // v.shape[1], axis=1)


def _ends(seqlens, batch, L):
    return np.full(batch, L) if seqlens is None else np.clip(np.asarray(seqlens), 0, L)


def scan(u, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, seqlens=None, softplus=True):
    """Returns (y, h_final, y_scale, h_scale); u, dt, z [b, L, ch], B, C [b, L, g, n]."""
    nb, L, ch = u.shape
    n = A.shape[1]
    ends = _ends(seqlens, nb, L)
    h = np.zeros((nb, ch, n)) if h0 is None else h0.copy()
    H, E = np.abs(h), np.zeros_like(h)
    y, ys = np.zeros_like(u), np.zeros_like(u)
    for t in range(L):
        on = (t < ends)[:, None]
        _, d = _steps(np.where(on, dt[:, t], 0.0), dt_bias, softplus)
        ut = np.where(on, u[:, t], 0.0)
        on3 = on[..., None]
        Bt, Ct = (np.where(on3, _groups(v[:, t], ch), 0.0) for v in (B, C))
        x = d[..., None] * A
        a = np.exp(x)
        b = (d * ut)[..., None] * Bt
        E = np.where(on3, a * E + (4 + 12 * np.abs(x)) * a * H + 12 * np.abs(b) + a * H + np.abs(b), E)
        h = np.where(on3, a * h + b, h)
        H = np.where(on3, a * H + np.abs(b), H)
        yt, st = (Ct * h).sum(-1), (np.abs(Ct) * (E + (n + 4) * H)).sum(-1)
        if D is not None:
            yt, st = yt + D * ut, st + 4 * np.abs(D * ut)
        if z is not None:
            f = silu(np.where(on, z[:, t], 0.0))
            st = (st + 16 * ((np.abs(Ct) * H).sum(-1) + (0 if D is None else np.abs(D * ut)))) * np.abs(f)
            yt = yt * f
        y[:, t], ys[:, t] = np.where(on, yt, 0.0), np.where(on, st, 0.0)
    return y, h, ys, E + H


def scan_grads(dy, u, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, seqlens=None, softplus=True, dh=None):
    """Gradients of sum(y dy) + sum(h_final dh): ({name: value}, {name: scale})."""
    nb, L, ch = u.shape
    g, n = B.shape[2], A.shape[1]
    ends = _ends(seqlens, nb, L)
    h = np.zeros((nb, ch, n)) if h0 is None else h0.copy()
    H, E = np.abs(h), np.zeros_like(h)
    kept = []
    for t in range(L):  # the states before each token, their magnitudes and errors
        kept.append((h, H, E))
        on3 = (t < ends)[:, None, None]
        _, d = _steps(np.where(on3[..., 0], dt[:, t], 0.0), dt_bias, softplus)
        ut = np.where(on3[..., 0], u[:, t], 0.0)
        Bt = np.where(on3, _groups(B[:, t], ch), 0.0)
        x = d[..., None] * A
        a, b = np.exp(x), (d * ut)[..., None] * Bt
        E = np.where(on3, a * E + (5 + 12 * np.abs(x)) * a * H + 13 * np.abs(b), E)
        h, H = np.where(on3, a * h + b, h), np.where(on3, a * H + np.abs(b), H)
    zero = lambda *s: np.zeros(s)  # noqa: E731
    names = {"du": u.shape, "ddt": u.shape, "dz": u.shape, "dA": A.shape, "dB": B.shape, "dC": C.shape, "dD": (ch,),
             "ddt_bias": (ch,)}
    G = {k: zero(*s) for k, s in names.items()}
    S = {k: zero(*s) for k, s in names.items()}
    back = zero(nb, ch, n) if dh is None else dh.copy()   # dL/dh after the token, its magnitude and error
    Bk, Ek = np.abs(back), np.zeros_like(back)
    group = np.arange(ch) // (ch // g)
    tokens = nb * L + 16
    for t in reversed(range(L)):
        on = (t < ends)[:, None]
        on3 = on[..., None]
        h, H, E = kept[t]
        x_in, d = _steps(np.where(on, dt[:, t], 0.0), dt_bias, softplus)
        ut = np.where(on, u[:, t], 0.0)
        Bt, Ct = (np.where(on3, _groups(v[:, t], ch), 0.0) for v in (B, C))
        x = d[..., None] * A
        a, b = np.exp(x), (d * ut)[..., None] * Bt
        da = 5 + 12 * np.abs(x)                            # a's relative error, and a rounding
        hn, Hn, En = a * h + b, a * H + np.abs(b), a * E + da * a * H + 13 * np.abs(b)
        o = np.where(on, dy[:, t], 0.0)
        gy, gs = o, np.zeros_like(o)
        if z is not None:
            zt = np.where(on, z[:, t], 0.0)
            gy = o * silu(zt)
            gs = 16 * np.abs(gy)
            yv = (Ct * hn).sum(-1) + (0 if D is None else D * ut)
            ya = (np.abs(Ct) * Hn).sum(-1) + (0 if D is None else np.abs(D * ut))
            yE = (np.abs(Ct) * (En + (n + 4) * Hn)).sum(-1) + (0 if D is None else 4 * np.abs(D * ut))
            # the two terms of silu' can cancel: their magnitudes count
            big = np.abs(sigmoid(zt)) * (1 + np.abs(zt))
            G["dz"][:, t] = np.where(on, o * yv * dsilu(zt), 0.0)
            S["dz"][:, t] = np.where(on, np.abs(o) * (yE * np.abs(dsilu(zt)) + 16 * ya * big), 0.0)
        q = back + gy[..., None] * Ct
        Q = Bk + np.abs(gy)[..., None] * np.abs(Ct)
        Eq = Ek + gs[..., None] * np.abs(Ct) + 2 * Q
        on_q = lambda v: np.where(on3, v, 0.0)  # noqa: E731
        qa, Qa, Eqa = on_q(q * a), on_q(Q * a), on_q(a * (Eq + da * Q))
        qah, Qah = qa * h, Qa * H
        Eqah = Eqa * H + Qa * E + 2 * Qah
        sig, Sig, Esig = (on_q(q) * Bt).sum(-1), (on_q(Q) * np.abs(Bt)).sum(-1), (on_q(Eq) * np.abs(Bt)).sum(-1)
        Esig = Esig + (n + 2) * Sig
        G["du"][:, t] = d * sig + (0 if D is None else D * gy)
        S["du"][:, t] = np.abs(d) * (Esig + 12 * Sig) + (0 if D is None else np.abs(D) * (gs + 4 * np.abs(gy)))
        v = (qah * A).sum(-1) + ut * sig
        V = (Qah * np.abs(A)).sum(-1) + np.abs(ut) * Sig
        Ev = (Eqah * np.abs(A)).sum(-1) + np.abs(ut) * Esig + (n + 8) * V
        if softplus:
            f = sigmoid(x_in)
            v, V, Ev = v * f, V * f, (Ev + 12 * V) * f
        v, Ev, V = np.where(on, v, 0.0), np.where(on, Ev, 0.0), np.where(on, V, 0.0)
        G["ddt"][:, t], S["ddt"][:, t] = v, Ev
        G["ddt_bias"] += v.sum(0)
        S["ddt_bias"] += (Ev + tokens * V).sum(0)
        G["dA"] += (qah * d[..., None]).sum(0)
        S["dA"] += ((Eqah + (12 + tokens) * Qah) * np.abs(d)[..., None]).sum(0)
        G["dD"] += (gy * ut).sum(0)
        S["dD"] += ((gs + tokens * np.abs(gy)) * np.abs(ut)).sum(0)
        w = (d * ut)[..., None]
        for name, val, err in (("dB", on_q(q) * w, np.abs(w) * (on_q(Eq) + (12 + ch) * on_q(Q))),
                               ("dC", gy[..., None] * hn,
                                np.abs(gy)[..., None] * (En + ch * Hn) + gs[..., None] * Hn)):
            for k in range(g):
                G[name][:, t, k] += val[:, group == k].sum(1)
                S[name][:, t, k] += err[:, group == k].sum(1)
        back, Bk, Ek = np.where(on3, qa, back), np.where(on3, Qa, Bk), np.where(on3, Eqa + Qa, Ek)
    G["dh0"], S["dh0"] = back, Ek + Bk
    return G, S


def conv(x, weight, bias=None, initial_state=None, seqlens=None, silu_on=True):
    """Returns (y, final_state, y_scale)."""
    nb, L, ch = x.shape
    W = weight.shape[1]
    ends = _ends(seqlens, nb, L)
    y, ys = np.zeros_like(x), np.zeros_like(x)
    last = np.zeros((nb, W - 1, ch))
    for i in range(nb):
        first = np.zeros((W - 1, ch)) if initial_state is None else initial_state[i]
        seq = np.concatenate([first, x[i, :ends[i]]], 0)
        last[i] = seq[len(seq) - (W - 1):]
        for t in range(ends[i]):
            win = seq[t:t + W].T
            p = (win * weight).sum(-1) + (0 if bias is None else bias)
            P = (np.abs(win * weight)).sum(-1) + (0 if bias is None else np.abs(bias))
            e = (W + 2) * P
            if silu_on:  # the slope of silu is at most 1.1
                e = 1.1 * e + 16 * np.abs(silu(p))
                p = silu(p)
            y[i, t], ys[i, t] = p, e
    return y, last, ys


def conv_grads(dy, x, weight, bias=None, initial_state=None, seqlens=None, silu_on=True, dfinal=None):
    """Gradients of sum(y dy) + sum(final_state dfinal), and their scales."""
    nb, L, ch = x.shape
    W = weight.shape[1]
    ends = _ends(seqlens, nb, L)
    G = {"dx": np.zeros_like(x), "dweight": np.zeros_like(weight), "dbias": np.zeros(ch),
         "dinitial_state": np.zeros((nb, W - 1, ch))}
    S = {k: np.zeros_like(v) for k, v in G.items()}
    tokens = nb * L + 16
    for i in range(nb):
        first = np.zeros((W - 1, ch)) if initial_state is None else initial_state[i]
        seq = np.concatenate([first, x[i, :ends[i]]], 0)
        dseq, dS = np.zeros_like(seq), np.zeros_like(seq)
        if dfinal is not None:
            dseq[len(seq) - (W - 1):] += dfinal[i]
            dS[len(seq) - (W - 1):] += np.abs(dfinal[i])
        for t in range(ends[i]):
            win = seq[t:t + W].T
            p = (win * weight).sum(-1) + (0 if bias is None else bias)
            P = (np.abs(win * weight)).sum(-1) + (0 if bias is None else np.abs(bias))
            d, e = dy[i, t], 0.0
            if silu_on:  # |silu''| <= 1/2
                e = np.abs(d) * (0.5 * (W + 2) * P + 16 * sigmoid(p) * (1 + np.abs(p)))
                d = d * dsilu(p)
            G["dweight"] += d[:, None] * win
            S["dweight"] += (e + tokens * np.abs(d))[:, None] * np.abs(win)
            G["dbias"] += d
            S["dbias"] += e + tokens * np.abs(d)
            dseq[t:t + W] += (weight * d[:, None]).T
            dS[t:t + W] += (np.abs(weight) * (e + 8 * np.abs(d))[:, None]).T
        G["dinitial_state"][i], S["dinitial_state"][i] = dseq[:W - 1], dS[:W - 1]
        G["dx"][i, :ends[i]], S["dx"][i, :ends[i]] = dseq[W - 1:], dS[W - 1:]
    return G, S


def e4m3_values():
    """The 256 values of the 8-bit float (4 exponent bits, bias 7; 3 fraction bits; NaN at 0x7f and 0xff)."""
    out = np.zeros(256)
    for i in range(256):
        e, f = (i >> 3) & 15, i & 7
        v = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        out[i] = np.nan if (e == 15 and f == 7) else (-v if i & 128 else v)
    return out


def cache_rows(h, kind):
    """(bytes as their values, scales) of fp32 rows [..., n], each step rounded to fp32 as the format says."""
    h = np.asarray(h, np.float32)
    top = np.float32(127 if kind == "int8" else 448)
    with np.errstate(all="ignore"):
        m = np.abs(h).max(-1)
        held = ~(m < np.float32(2.0 ** -100))
        scale = np.where(held, m / top, np.float32(0)).astype(np.float32)
        scale = np.where(np.isfinite(m), scale, np.float32(np.nan))
        inv = np.where(held, top / m, np.float32(0)).astype(np.float32)
        q = (h * inv[..., None]).astype(np.float32)
    if kind == "int8":
        q = np.nan_to_num(np.rint(q), nan=0.0)
    else:
        vals = np.sort(e4m3_values()[:127])                      # 0 .. 448
        a = np.abs(np.nan_to_num(q.astype(np.float64)))
        hi = np.clip(np.searchsorted(vals, a), 0, len(vals) - 1)
        lo = np.maximum(hi - 1, 0)
        up = (vals[hi] - a < a - vals[lo]) | ((vals[hi] - a == a - vals[lo]) & (hi % 2 == 0))
        q = np.copysign(np.where(up | (a >= vals[hi]), vals[hi], vals[lo]), q)
    return q, scale
