"""CPU oracle: the gated delta rule in chunks of 64 tokens, with the roundings
to bf16 of the tensor-core path and none besides (test infrastructure).

Between the roundings everything is float64, so that a kernel differs from
this by its float32 arithmetic alone: where that moves a value across the
border between two bf16 numbers, by one step of it.  What the kernels hold in
two bf16 parts (2^-17 of it) is not rounded here.  `rounds` names the
roundings that are made (ALL of them by default); without any this is the
chunk form itself and equals oracle.delta_recurrent and delta_backward.

q, k, v, g, beta, d_out hold bf16 values; shapes as in oracle/delta.py.
"""
from __future__ import annotations

import numpy as np

from .delta import _f64, _lengths

CHUNK = 64
# forward: T^, W and Q~ as the chunks' operands, the state as an operand, the
# output itself; P and both uses of X are in two parts
FORWARD = ("T", "W", "Q", "S", "out")
# backward: T^ and W, the state and its gradient D as operands and as they are
# kept, dX where it meets W (dV takes it in two parts), dV as it leaves (dbeta
# takes it in two), the gradients that leave; Q~, P, X and the pairs are in two
BACKWARD = ("T", "W", "S", "D", "dX", "dV", "grads")
ALL = FORWARD + BACKWARD


def bf16(x):
    """x rounded to the nearest bf16 number, ties to even."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32)
    up = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return up.astype(np.uint32).view(np.float32).astype(x.dtype)


class _Chunk:
    """What a chunk's products take of its tokens, for a (sequence, head)."""

    def __init__(self, q, k, g, b, scale, rounds, two_parts, f, none=False):
        self.f, self.rounds, self.two = f, rounds, two_parts
        self.q, self.k, self.b, self.scale = q, k, b, f(scale)
        n = len(g)
        g = np.maximum(g, -105.0)          # e^g is 0 in float32 from here on
        G = np.cumsum(np.asarray(g, np.float64))
        self.decay = np.tril(np.exp(np.minimum(np.subtract.outer(G, G), 0.0))).astype(f)
        self.e = np.exp(G).astype(f)
        self.rest = self.decay[-1].copy()
        self.eL = self.e[-1]
        M = np.tril(k @ k.T, -1) * self.decay * b[:, None]
        T = np.linalg.inv(np.eye(n, dtype=f) + M)
        # in the backward T itself where a token writes nothing (b of 0)
        self.T, self.Tlo = self.part("T", T * np.where(none, f(1), b))
        W = (T * b * self.e) @ k
        self.W, self.Wlo = self.part("W", W)
        self.Q = q * (self.scale * self.e)[:, None]
        self.P = self.scale * (q @ k.T) * self.decay

    def round(self, name, x):
        return bf16(x) if name in self.rounds else x

    def part(self, name, x):
        """(the operand, its second part)"""
        hi = self.round(name, x)
        return hi, self.round(name, x - hi) if self.two else 0.0 * x

    def step(self, S, v):
        """(X, the state behind the chunk, the state as an operand: its parts)"""
        hi, lo = self.part("S", S)
        X = (self.T + self.Tlo) @ v - ((self.W + self.Wlo) @ hi + self.W @ lo)
        return X, self.eL * S + self.k.T @ (self.rest[:, None] * X), hi, lo


def _walks(q, k, v, g, beta, lengths):
    """(b, h, key head, slices of the chunks) of every (sequence, value head)"""
    B, n, H, _ = v.shape
    rep = H // q.shape[2]
    for b, length in enumerate(_lengths(lengths, B, n)):
        for h in range(H):
            yield b, h, h // rep, [slice(t, min(t + CHUNK, length)) for t in range(0, length, CHUNK)]


def delta_chunks(q, k, v, g, beta, scale, state=None, lengths=None, final_state=False, rounds=ALL,
                 dtype=np.float64):
    """(o, S after the last token).  final_state: as where one is asked for,
    with T^, W and the state in two bf16 parts."""
    f = dtype
    q, k, v, g, beta = (_f64(x).astype(f) for x in (q, k, v, g, beta))
    B, n, H, dv = v.shape
    o = np.zeros((B, n, H, dv), f)
    S = np.zeros((B, H, q.shape[-1], dv), f) if state is None else _f64(state).astype(f)
    for b, h, kh, chunks in _walks(q, k, v, g, beta, lengths):
        s = S[b, h]
        for c in chunks:
            w = _Chunk(q[b, c, kh], k[b, c, kh], g[b, c, h], beta[b, c, h], scale, rounds, final_state, f)
            X, s, hi, lo = w.step(s, v[b, c, h])
            o[b, c, h] = w.round("out", w.round("Q", w.Q) @ (hi + lo) + w.P @ X)
        S[b, h] = s
    return o, S


def delta_chunks_backward(q, k, v, g, beta, d_out, scale, lengths=None, rounds=ALL, dtype=np.float64):
    """Gradients (dq, dk, dv, dg, dbeta) of sum(o * d_out) without initial state."""
    f = dtype
    q, k, v, g, beta, d_out = (_f64(x).astype(f) for x in (q, k, v, g, beta, d_out))
    none = np.abs(beta) < 1e-15            # tokens that write nothing
    beta = np.where(none, f(0), beta)
    dq, dk, dv_ = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    dg, db = np.zeros_like(g), np.zeros_like(beta)
    for b, h, kh, chunks in _walks(q, k, v, g, beta, lengths):
        made, s = [], np.zeros((q.shape[-1], v.shape[-1]), f)
        for c in chunks:
            off = none[b, c, h]
            w = _Chunk(q[b, c, kh], k[b, c, kh], g[b, c, h], beta[b, c, h], scale, rounds, False, f, off)
            X, s, hi, _ = w.step(s, np.where(off[:, None], f(0), v[b, c, h]))
            made.append((c, w, X, hi))
        D = np.zeros_like(s)
        for c, w, X, S in reversed(made):
            do = d_out[b, c, h]
            Dh = w.round("D", D)                           # behind the chunk
            dX = w.P.T @ do + w.rest[:, None] * (w.k @ Dh)
            hi = w.round("dX", dX)
            D = w.eL * D + w.Q.T @ do - w.W.T @ hi
            full = w.T.T @ dX
            dV = w.round("dV", full)
            off = none[b, c, h][:, None]                   # there dV is the gradient of x
            A = w.scale * (do @ X.T) * w.decay
            B = -np.tril(dV @ X.T, -1) * w.decay
            from_q = w.scale * w.e[:, None] * (do @ S.T)
            from_k = -w.e[:, None] * (dV @ S.T)
            missed = (dV * v[b, c, h]).sum(1) + (w.k * from_k).sum(1) + (B * (w.k @ w.k.T)).sum(1)
            B, from_k = np.where(off, 0.0, B), np.where(off, 0.0, from_k)
            E = np.tril(A * (w.q @ w.k.T) + B * (w.k @ w.k.T), -1)
            to_D = w.rest[:, None] * (X @ Dh.T)
            dq[b, c, kh] += from_q + A @ w.k
            dk[b, c, kh] += from_k + to_D + A.T @ w.q + (B + B.T) @ w.k
            inter = (w.q * from_q).sum(1) + (w.k * from_k).sum(1) + E.sum(1) - E.sum(0)
            ahead = (w.k * to_D).sum(1)
            dg[b, c, h] = np.cumsum(inter[::-1])[::-1] + np.cumsum(ahead) - ahead + w.eL * (S * Dh).sum()
            db[b, c, h] = np.where(off[:, 0], missed, (full * X).sum(1) / np.where(off[:, 0], 1.0, w.b * w.b))
            dv_[b, c, h] = np.where(off, 0.0, dV)
    if "grads" in rounds:
        dq, dk, dg, db = (bf16(x) for x in (dq, dk, dg, db))
    return dq, dk, dv_, dg, db
