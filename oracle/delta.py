"""The gated delta rule, its gradients and the norms around a block as plain
float64 loops, with error bounds.  Test infrastructure only.

``delta`` and ``delta_grads`` walk token by token; ``delta_bounds`` repeats the
kernels' chunk algebra in float64 to see how large the terms are whose rounding
reaches each output, and returns absolute bounds to first order:

* a product's computed operand carries a relative error of ``u2`` (two bf16 numbers 2^-16, two
  fp16 numbers 2^-22, and ``SUB`` as long as gradients are scaled to be of the size of 4 and more, fp32 2^-24;
  one number's half step is ``U1``);
* every product's fp32 sums and factors add ``W`` = 32 units of 2^-24 of the sum of its
  terms' magnitudes (sums run over at most 8 terms at a time in the unit, tiles after tiles
  in turn: 8 to 16 turns, and the decays' exponentials add 1 + |x| units, which fade with them);
* errors of states pass through a chunk by its own linear map, whose norm per
  token is e^g max(1, |1 - beta |k|^2|); within a chunk |T|, elementwise, carries them.
"""
from __future__ import annotations

import numpy as np

U2 = {"bf16": 2.0 ** -16, "f16": 2.0 ** -22, "f32": 2.0 ** -24}
U1 = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
SUB = {"bf16": 0.0, "f16": 2.0 ** -25, "f32": 0.0}
W = 32 * 2.0 ** -24


def _ends(seqlens, batch, L):
    return np.full(batch, L) if seqlens is None else np.clip(np.asarray(seqlens), 0, L)


# ---------------------------------------------------------------------------
# token by token
# ---------------------------------------------------------------------------
def delta(q, k, v, g, beta, h0=None, seqlens=None, scale=None):
    """(y [b, L, H, dv], h [b, H, dv, dk]); q, k [b, L, Hk, dk], v [b, L, H, dv], g, beta [b, L, H]."""
    nb, L, H, dv = v.shape
    dk, rep = q.shape[-1], H // q.shape[2]
    c = dk ** -0.5 if scale is None else scale
    h = np.zeros((nb, H, dv, dk)) if h0 is None else h0.copy()
    y = np.zeros_like(v)
    for b, end in enumerate(_ends(seqlens, nb, L)):
        for t in range(end):
            for n in range(H):
                kt, S = k[b, t, n // rep], np.exp(g[b, t, n]) * h[b, n]
                h[b, n] = S + beta[b, t, n] * np.outer(v[b, t, n] - S @ kt, kt)
                y[b, t, n] = c * h[b, n] @ q[b, t, n // rep]
    return y, h


def delta_grads(dy, q, k, v, g, beta, h0=None, seqlens=None, scale=None, dh=None):
    """Gradients of sum(y dy) + sum(h dh) by the reverse walk: dq, dk, dv, dg, dbeta, dh0."""
    nb, L, H, dv = v.shape
    dk, rep = q.shape[-1], H // q.shape[2]
    c = dk ** -0.5 if scale is None else scale
    G = {"dq": np.zeros_like(q), "dk": np.zeros_like(k), "dv": np.zeros_like(v), "dg": np.zeros_like(g),
         "dbeta": np.zeros_like(beta), "dh0": np.zeros((nb, H, dv, dk))}
    for b, end in enumerate(_ends(seqlens, nb, L)):
        for n in range(H):
            m = n // rep
            S = np.zeros((dv, dk)) if h0 is None else h0[b, n]
            kept = []
            for t in range(end):
                kept.append(S)
                S = np.exp(g[b, t, n]) * S
                S = S + beta[b, t, n] * np.outer(v[b, t, n] - S @ k[b, t, m], k[b, t, m])
            D = np.zeros((dv, dk)) if dh is None else dh[b, n].copy()
            for t in reversed(range(end)):
                kt, be, a = k[b, t, m], beta[b, t, n], np.exp(g[b, t, n])
                F = a * kept[t]
                miss = v[b, t, n] - F @ kt
                G["dq"][b, t, m] += c * (F + be * np.outer(miss, kt)).T @ dy[b, t, n]
                D = D + c * np.outer(dy[b, t, n], q[b, t, m])
                Dk = D @ kt
                G["dbeta"][b, t, n] = miss @ Dk
                G["dv"][b, t, n] = be * Dk
                G["dk"][b, t, m] += be * (D.T @ miss - F.T @ Dk)
                D = D - be * np.outer(Dk, kt)
                G["dg"][b, t, n] = (D * F).sum()
                D = a * D
            G["dh0"][b, n] = D
    return G


def delta_step(h, q, k, v, g, beta, scale=None):
    """One token: (y [b, H, dv], new h)."""
    y, hn = delta(q[:, None], k[:, None], v[:, None], g[:, None], beta[:, None], h0=h, scale=scale)
    return y[:, 0], hn


# ---------------------------------------------------------------------------
# the chunk algebra, and what rounding can do in it
# ---------------------------------------------------------------------------
def _decay(g):
    """D[i, j] = exp(g_{j+1} + .. + g_i) for j <= i, else 0."""
    n = len(g)
    D = np.zeros((n, n))
    for j in range(n):
        D[j:, j] = np.exp(np.concatenate([[0.0], np.cumsum(g[j + 1:])]))
    return D


def delta_bounds(kind, C, q, k, v, g, beta, h0=None, seqlens=None, scale=None, dy=None, dh=None):
    """Returns (values, bounds): dicts of y, h and, with dy, the gradients; values by the chunk algebra in float64."""
    nb, L, H, dv = v.shape
    dk, rep = q.shape[-1], H // q.shape[2]
    c = dk ** -0.5 if scale is None else scale
    u2, s = U2[kind] + W, SUB[kind]
    E2 = lambda x: u2 * np.abs(x) + s  # noqa: E731
    EN = lambda norm, s=s: u2 * norm + s * dk ** 0.5  # noqa: E731  of a column of dk elements, by its norm
    names = {"y": v, "h": np.zeros((nb, H, dv, dk))}
    if dy is not None:
        names |= {"dq": q, "dk": k, "dv": v, "dg": g, "dbeta": beta, "dh0": names["h"]}
    val, err = ({n: np.zeros_like(a) for n, a in names.items()} for _ in range(2))
    A_ = np.abs
    for b, end in enumerate(_ends(seqlens, nb, L)):
        for n in range(H):
            m = n // rep
            S = np.zeros((dk, dv)) if h0 is None else h0[b, n].T
            eS = np.zeros(dv)  # 2-norm of each column's error
            kept = []
            for t0 in range(0, end, C):
                at = slice(t0, min(t0 + C, end))
                Q, K, V, be = q[b, at, m], k[b, at, m], v[b, at, n], beta[b, at, n]
                D = _decay(g[b, at, n])
                st, en = D[:, 0] * np.exp(g[b, t0, n]), D[-1]
                kk, kn, qn = K @ K.T, np.linalg.norm(K, axis=1), np.linalg.norm(Q, axis=1)
                T = np.linalg.inv(np.eye(len(be)) + np.tril(be[:, None] * D * kk, -1))
                aT, low = A_(T), np.tril(A_(T), -1)
                P = D * (Q @ K.T)
                R = be[:, None] * (V - st[:, None] * (K @ S))
                N = T @ R
                Sn = np.linalg.norm(S, axis=0)
                # T: its own inversion, A's rounding through |T| |A| |T|
                eT = W * aT @ (np.tril(A_(be)[:, None] * D * np.outer(kn, kn), -1) @ aT)
                eR = W * A_(R) + A_(be)[:, None] * (st * kn)[:, None] * (EN(Sn) + eS) + W * A_(be)[:, None] * A_(V)
                eN = aT @ eR + (E2(low) + eT) @ A_(R) + low @ E2(R) + W * A_(N)
                Y = c * (st[:, None] * (Q @ S) + P @ N)
                val["y"][b, at, n] = Y
                aP = D * A_(Q @ K.T)
                eP = W * D * np.outer(qn, kn)
                err["y"][b, at, n] = A_(c) * (st[:, None] * (A_(Q) @ E2(S)) + (st * qn)[:, None] * eS
                                              + (E2(aP) + eP) @ A_(N) + aP @ (E2(N) + eN)) + W * A_(Y)
                kept.append((at, S, eS, N, eN, T, eT, P, eP, D, st, en, kk))
                # what the chunk's own map makes of the error it got, and what it adds
                grow = np.prod(np.exp(g[b, at, n]) * np.maximum(1.0, A_(1 - be * kn ** 2)))
                local = aT @ (A_(be)[:, None] * (st * kn)[:, None] * EN(Sn) + W * A_(be)[:, None] * A_(V) + W * A_(R)) \
                    + (E2(low) + eT) @ A_(R) + low @ E2(R) + W * A_(N)
                S = st[-1] * S + K.T @ (en[:, None] * N)
                eS = grow * eS + (en * kn) @ local + kn @ E2(en[:, None] * N) + W * st[-1] * Sn
            val["h"][b, n], err["h"][b, n] = S.T, np.broadcast_to(eS[:, None], (dv, dk))
            if dy is None:
                continue
            dS = np.zeros((dk, dv)) if dh is None else dh[b, n].T
            eD = np.zeros(dv)
            # fp16: operands that are gradients are held to 2^-25 where the largest of c dY and dh is 4 at least, and
            # the chunk's pairs where their largest is 2^10 or all of them are multiplied by 2^15
            top = max(abs(c) * A_(dy[b, :end, n]).max(initial=0.0), A_(dS).max())
            sg = s * top / 4
            G2 = lambda x: u2 * np.abs(x) + sg  # noqa: E731
            for at, S, eS, N, eN, T, eT, P, eP, D, st, en, kk in reversed(kept):
                Q, K, V, be, dY = q[b, at, m], k[b, at, m], v[b, at, n], beta[b, at, n], dy[b, at, n]
                kn, qn = np.linalg.norm(K, axis=1), np.linalg.norm(Q, axis=1)
                Dn, Sn, ab, ac = np.linalg.norm(dS, axis=0), np.linalg.norm(S, axis=0), A_(be), A_(c)
                aT, low, aP = A_(T), np.tril(A_(T), -1), A_(P)
                dN = en[:, None] * (K @ dS) + c * P.T @ dY
                Z = T.T @ dN
                edN0 = (en * kn)[:, None] * EN(Dn, sg) + ac * (E2(aP) + eP).T @ A_(dY) + W * A_(dN)
                edN = edN0 + (en * kn)[:, None] * eD
                more = (E2(low) + eT).T @ A_(dN) + low.T @ G2(dN) + W * A_(Z)
                eZ = aT.T @ edN + more
                val["dv"][b, at, n] = be[:, None] * Z
                err["dv"][b, at, n] = ab[:, None] * eZ
                # the state's parts
                X1, X2, X3 = dY @ S.T, Z @ S.T, (en[:, None] * N) @ dS.T
                e1 = A_(dY) @ E2(S).T + (A_(dY) @ eS)[:, None] * np.ones(dk)
                e2 = A_(Z) @ E2(S).T + G2(Z) @ A_(S).T + (A_(Z) @ eS)[:, None] + eZ @ A_(S).T
                aNe = en[:, None] * A_(N)
                e3 = aNe @ G2(dS).T + E2(aNe) @ A_(dS).T + (aNe @ eD)[:, None] + en[:, None] * (eN @ A_(dS).T)
                # as dots with a key or query the states' errors count by their norm
                d1 = (A_(Q) * (A_(dY) @ E2(S).T)).sum(1) + qn * (A_(dY) @ eS)
                d2 = (A_(K) * (A_(Z) @ E2(S).T + G2(Z) @ A_(S).T)).sum(1) + kn * (A_(Z) @ eS) \
                    + (A_(K) * (eZ @ A_(S).T)).sum(1)
                d3 = (A_(K) * (aNe @ G2(dS).T + E2(aNe) @ A_(dS).T)).sum(1) + kn * (aNe @ eD) \
                    + en * (A_(K) * (eN @ A_(dS).T)).sum(1)
                # the write terms are taken as a difference from the read terms
                d3 = d3 + W * (ab * st * (A_(K) * A_(X2)).sum(1))
                dP, Mz = np.tril(dY @ N.T), np.tril(Z @ N.T, -1)
                edP = np.tril(A_(dY) @ (E2(N) + eN).T)
                eM = np.tril(A_(Z) @ (E2(N) + eN).T + (G2(Z) + eZ) @ A_(N).T, -1)
                pP, pB = c * D * dP, -be[:, None] * D * Mz
                sp = s * (2.0 ** -10 * max(A_(pP).max(), A_(pB).max()) + 2.0 ** -15 * top / 4)
                P2 = lambda x: u2 * np.abs(x) + sp  # noqa: E731
                epP, epB = ac * D * edP + W * A_(pP), ab[:, None] * D * eM + W * A_(pB)
                val["dq"][b, at, m] += c * st[:, None] * X1 + pP @ K
                err["dq"][b, at, m] += ac * st[:, None] * e1 + (P2(pP) + epP) @ A_(K)
                val["dk"][b, at, m] += -(be * st)[:, None] * X2 + pB @ K + X3 + pB.T @ K + pP.T @ Q
                err["dk"][b, at, m] += (ab * st)[:, None] * e2 + e3 + (P2(pB) + epB) @ A_(K) \
                    + (P2(pB) + epB).T @ A_(K) + (P2(pP) + epP).T @ A_(Q)
                k2 = (K * X2).sum(1)
                val["dbeta"][b, at, n] = (Z * V).sum(1) - st * k2 - (D * kk * Mz).sum(1)
                err["dbeta"][b, at, n] = (W * A_(Z) * A_(V) + eZ * A_(V)).sum(1) + st * d2 + W * st * A_(k2) \
                    + (D * np.outer(kn, kn) * (eM + 2 * W * A_(Mz))).sum(1)
                F = np.tril(pP * (Q @ K.T) + pB * kk, -1)
                eF = np.tril((epP + 2 * W * A_(pP)) * np.outer(qn, kn) + (epB + 2 * W * A_(pB)) * np.outer(kn, kn), -1)
                read, write = c * st * (Q * X1).sum(1) - be * st * k2, (K * X3).sum(1)
                eread = ac * st * d1 + ab * st * d2 + W * (ac * st * (A_(Q) * A_(X1)).sum(1) + ab * st * (A_(K) * A_(X2)).sum(1))
                both = st[-1] * (S * dS).sum()
                eboth = st[-1] * (W * A_(S * dS).sum() + eS @ Dn + Sn @ eD)
                span = len(be)
                for t in range(span):
                    val["dg"][b, at.start + t, n] = F[t:, :t].sum() + read[t:].sum() + write[:t].sum() + both
                    # sums by rows less sums by columns: what cancels leaves the sums' own roundings
                    err["dg"][b, at.start + t, n] = eF[t:, :t].sum() + eread[t:].sum() + d3[:t].sum() + eboth \
                        + W * (A_(F)[t:].sum() + A_(F)[:, t:].sum() + A_(read)[t:].sum() + A_(write)[:t].sum())
                grow = np.prod(np.exp(g[b, at, n]) * np.maximum(1.0, A_(1 - be * kn ** 2)))
                dR = be[:, None] * Z
                dS = st[-1] * dS + c * (st[:, None] * Q).T @ dY - (st[:, None] * K).T @ dR
                eD = grow * eD + qn @ G2(c * st[:, None] * dY) + kn @ G2(st[:, None] * dR) \
                    + (st * kn * ab) @ (aT.T @ edN0 + more) + W * st[-1] * Dn
            val["dh0"][b, n], err["dh0"][b, n] = dS.T, np.broadcast_to(eD[:, None], (dv, dk))
    return val, err


# ---------------------------------------------------------------------------
# norms.  Scales count fp32 roundings (2^-24): rstd within 24 of itself (a sum of squares of up to 16384
# terms, 64 in turn and then by halves; square root and reciprocal), silu and its derivative within 16.
# ---------------------------------------------------------------------------
def _sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1 / (1 + e), e / (1 + e))


def gated_norm(x, weight=None, z=None, eps=1e-6, gate_first=False):
    """(y, rstd, y_scale, rstd_scale); x, z [rows, heads, dim]."""
    w = np.ones(x.shape[-1]) if weight is None else weight
    gate = np.ones_like(x) if z is None else z * _sigmoid(z)
    u = x * gate if gate_first else x
    rstd = 1 / np.sqrt((u * u).mean(-1) + eps)
    y = u * rstd[..., None] * w
    y = y if gate_first else y * gate
    return y, rstd, (48 + 16 * gate_first) * np.abs(y), (96 if gate_first else 64) * rstd


def gated_norm_grads(dy, x, weight=None, z=None, eps=1e-6, gate_first=False):
    """dicts (gradients, scales)."""
    w = np.ones(x.shape[-1]) if weight is None else weight
    z_, sig = (np.zeros_like(x), np.ones_like(x)) if z is None else (z, _sigmoid(z))
    gate = np.ones_like(x) if z is None else z * sig
    slope = sig * (1 + z_ * (1 - sig))
    aslope = sig * (1 + np.abs(z_))  # its terms' magnitudes
    u = x * gate if gate_first else x
    rstd = (1 / np.sqrt((u * u).mean(-1) + eps))[..., None]
    unit = u * rstd
    into = dy * w if gate_first else dy * w * gate
    mean, amean = (into * unit).mean(-1, keepdims=True), np.abs(into * unit).mean(-1, keepdims=True)
    du = rstd * (into - unit * mean)
    sdu = 200 * rstd * (np.abs(into) + np.abs(unit) * amean)
    n = x.shape[0] * x.shape[1]
    sums = 64 + min(n, 64) + n / 1024  # a thread's turns, then 1024 parts
    dn = dy if gate_first else dy * gate
    G = {"dx": du * gate if gate_first else du, "dweight": (dn * unit).sum((0, 1))}
    S = {"dx": (sdu + 16 * np.abs(du)) * (np.abs(gate) if gate_first else 1), "dweight": (64 + sums) * np.abs(dn * unit).sum((0, 1))}
    if z is not None:
        G["dz"] = (du * x if gate_first else dy * w * unit) * slope
        S["dz"] = (sdu * np.abs(x) + 32 * np.abs(du * x) if gate_first else 80 * np.abs(dy * w * unit)) * aslope
    return G, S


def residual_stream(x, residual=None, scale=None):
    """(r, r_scale)"""
    s = 1.0 if scale is None else scale
    r = s * x + (0.0 if residual is None else residual)
    return r, np.abs(s * x) + np.abs(r)


def residual_norm_grads(dy, r, weight=None, eps=1e-6, dr=None, x=None, scale=None):
    """dicts (gradients, scales), from r as it was kept."""
    w = np.ones(r.shape[-1]) if weight is None else weight
    G, S = gated_norm_grads(dy[:, None], r[:, None], w, eps=eps)
    du, sdu = G["dx"][:, 0], S["dx"][:, 0]
    if dr is not None:
        du, sdu = du + dr, sdu + np.abs(dr) + np.abs(du)
    s = 1.0 if scale is None else scale
    got = {"dresidual": du, "dx": du * s, "dweight": G["dweight"]}
    sc = {"dresidual": sdu, "dx": (sdu + np.abs(du)) * np.abs(s), "dweight": S["dweight"]}
    if scale is not None:
        got["dscale"] = (du * x).sum(0)
        sc["dscale"] = (np.abs(x) * (sdu + (128 + len(x) / 1024) * np.abs(du))).sum(0)
    return got, sc
