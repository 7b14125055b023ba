"""CPU oracle: the gated delta rule and the fused residual norm in float64
(test infrastructure, as oracle/retention.py).

Per (sequence, value head), row vectors, log decay g, write strength b:
    S <- e^g S;  x = b (v - k S);  S <- S + k^T x;  o = scale q S.
q, k [B, n, Hk, dk]; v, o [B, n, H, dv]; g, beta [B, n, H]; S [B, H, dk, dv].
Value head h uses key head h // (H // Hk).  With lengths, tokens at or behind
lengths[b] are not part of sequence b: zero output rows and gradients.

Written token by token, and the gradients as the reverse of the same
recurrence; the tests hold them to central finite differences.
"""
from __future__ import annotations

import numpy as np

F64 = np.float64


def _f64(x):
    return np.asarray(x, dtype=F64)


def _lengths(lengths, B, n):
    return [n] * B if lengths is None else [min(max(int(x), 0), n) for x in lengths]


def delta_recurrent(q, k, v, g, beta, scale, state=None, lengths=None):
    """Returns (o, S after the last token)."""
    q, k, v, g, beta = map(_f64, (q, k, v, g, beta))
    B, n, H, dv = v.shape
    dk, rep = q.shape[-1], H // q.shape[2]
    o = np.zeros((B, n, H, dv))
    S = np.zeros((B, H, dk, dv)) if state is None else _f64(state).copy()
    for b, length in enumerate(_lengths(lengths, B, n)):
        for h in range(H):
            s = S[b, h]
            for t in range(length):
                kt = k[b, t, h // rep]
                s = np.exp(g[b, t, h]) * s
                x = beta[b, t, h] * (v[b, t, h] - kt @ s)
                s = s + np.outer(kt, x)
                o[b, t, h] = scale * (q[b, t, h // rep] @ s)
            S[b, h] = s
    return o, S


def delta_backward(q, k, v, g, beta, d_out, scale, lengths=None):
    """Gradients (dq, dk, dv, dg, dbeta) of sum(o * d_out) without initial state."""
    q, k, v, g, beta, d_out = map(_f64, (q, k, v, g, beta, d_out))
    B, n, H, dv_ = v.shape
    dk_, rep = q.shape[-1], H // q.shape[2]
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    dg, db = np.zeros_like(g), np.zeros_like(beta)
    for b, length in enumerate(_lengths(lengths, B, n)):
        for h in range(H):
            c = h // rep
            s, seen = np.zeros((dk_, dv_)), []
            for t in range(length):
                faded = np.exp(g[b, t, h]) * s
                miss = v[b, t, h] - k[b, t, c] @ faded
                s = faded + np.outer(k[b, t, c], beta[b, t, h] * miss)
                seen.append((faded, miss, s))
            D = np.zeros((dk_, dv_))               # gradient of the state behind token t
            for t in range(length - 1, -1, -1):
                faded, miss, s = seen[t]
                do, kt, bt = d_out[b, t, h], k[b, t, c], beta[b, t, h]
                dq[b, t, c] += scale * (s @ do)
                D = D + scale * np.outer(q[b, t, c], do)
                dx = kt @ D
                dmiss = bt * dx
                db[b, t, h] = dx @ miss
                dv[b, t, h] = dmiss
                dk[b, t, c] += D @ (bt * miss) - faded @ dmiss
                D = D - np.outer(kt, dmiss)        # gradient of the faded state
                dg[b, t, h] = (D * faded).sum()
                D = np.exp(g[b, t, h]) * D
    return dq, dk, dv, dg, db


def _rms(x, eps):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def residual_norm(x, y, gate=None, post_norm=True, post=None, pre=None, scale=1.0, eps=1e-5):
    """(h, n): h = x + scale swish(gate) rms(y) post, n = rms(h) pre."""
    x, y = _f64(x), _f64(y)
    z = _rms(y, eps) if post_norm else y
    if post is not None:
        z = z * _f64(post)
    if gate is not None:
        gate = _f64(gate)
        z = z * gate / (1.0 + np.exp(-gate))
    h = x + scale * z
    n = _rms(h, eps)
    return h, n if pre is None else n * _f64(pre)


def residual_norm_backward(x, y, dn, dh=None, gate=None, post_norm=True, post=None, pre=None,
                           scale=1.0, eps=1e-5):
    """(dx, dy, dgate, dpost, dpre) of sum(n dn) + sum(h dh)."""
    x, y, dn = _f64(x), _f64(y), _f64(dn)
    hidden = x.shape[-1]
    post = np.ones(hidden) if post is None else _f64(post)
    pre = np.ones(hidden) if pre is None else _f64(pre)

    def rms_back(a, da_hat):
        r = 1.0 / np.sqrt((a * a).mean(-1, keepdims=True) + eps)
        return r * da_hat - a * r ** 3 * (da_hat * a).mean(-1, keepdims=True)

    yhat = _rms(y, eps) if post_norm else y
    z = yhat * post
    sw, dsw = 1.0, 0.0
    if gate is not None:
        gate = _f64(gate)
        sig = 1.0 / (1.0 + np.exp(-gate))
        sw, dsw = gate * sig, sig * (1.0 + gate * (1.0 - sig))
    h = x + scale * sw * z
    flat = tuple(range(x.ndim - 1))
    dpre = (dn * _rms(h, eps)).sum(flat)
    dx = rms_back(h, dn * pre) + (0.0 if dh is None else _f64(dh))
    dgate = None if gate is None else scale * dx * z * dsw
    dz = scale * dx * sw
    dpost = (dz * yhat).sum(flat)
    dy = rms_back(y, dz * post) if post_norm else dz * post
    return dx, dy, dgate, dpost, dpre
