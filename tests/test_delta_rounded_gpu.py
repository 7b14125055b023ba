"""The tensor-core path's bf16 roundings: no more of them than documented.

The oracle's chunk form (oracle/delta_chunks.py) makes exactly the documented
roundings, in float64 between them.  Kernel and oracle are each compared with
the definition, and the kernel may not be further from it, for any (batch,
head), than the oracle is.

How close the two errors are: a kernel's float32 noise puts a value on the
other side of a border between two bf16 numbers only where it is about as far
from both, so its error keeps its size.  An error over a (batch, head) is then
a norm of N independent roundings of given sizes, N at least 64 for each token
(a row of X, of dV, of P or A, of the result; for dg and dbeta one number a
token).  Even if all of them were drawn anew, the ratio of two such norms has
a standard deviation of at most 1 / sqrt(N); the bound is three of them.  A
further rounding of a main operand (P, X, A or B, dV: 1.5e-3 and more of its
output, beside 1.7e-3 to 2.2e-3) raises the error by 20 % and more; 64 tokens
allow 4.7 %.
Short enough for walks of whole sequences: 11 chunks."""
import numpy as np
import pytest
import torch

import oracle
from helpers import record
from test_delta_gpu import bound, done, err, make, rn, states  # noqa: F401

pytestmark = pytest.mark.gpu

SHAPES = [  # n, Hk, H, dk, dv, lengths
    (704, 2, 2, 128, 128, [704, 500]), (300, 1, 3, 64, 256, [300, 0, 129]),
    (321, 1, 2, 128, 64, [64, 321]), (448, 2, 4, 64, 64, [447, 300]),
]


def ragged(seed, n, Hk, H, dk, dv, lens, dtype="bf16", decay=0.2):
    x, ref = make(seed, len(lens), n, Hk, H, dk, dv, dtype, decay)
    for t, r in zip(x, ref):
        for b, c in enumerate(lens):
            t[b, c:] = float("nan")
            r[b, c:] = 0.0
    return x, ref, torch.tensor(lens, dtype=torch.int32, device="cuda")


def per_head(x):
    """dg, dbeta [B, n, H] with their tokens as the values of a (batch, head)"""
    return x[..., None] if x.ndim == 3 else x


def no_further(got, rounded, want, lens, what):
    """Both against want, [B, n, heads, d] (a key head's gradients by key heads)
    or [B, n, heads]."""
    got = per_head(got.double().cpu().numpy())
    rounded, want = per_head(rounded), per_head(want)
    assert np.isfinite(got).all() and got.shape == rounded.shape == want.shape
    for b, tokens in enumerate(lens):
        assert not got[b, tokens:].any()
        for h in range(got.shape[2] if tokens else 0):
            size = np.linalg.norm(want[b, :, h])
            mine, theirs = (np.linalg.norm(x[b, :, h] - want[b, :, h]) / size for x in (got, rounded))
            record(mine, what)
            record(mine / theirs, what + " / rounded oracle")
            values = tokens * (64 if want.shape[3] > 1 else 1)
            assert mine < (1 + 3 / np.sqrt(values)) * theirs, (what, b, h)


@pytest.mark.parametrize("decay", [0.2, 0.02])
@pytest.mark.parametrize("n,Hk,H,dk,dv,lens", SHAPES)
def test_prefill(rn, n, Hk, H, dk, dv, lens, decay):
    x, ref, lengths = ragged(60 + n, n, Hk, H, dk, dv, lens, decay=decay)
    S, S0 = states(61, len(lens), H, dk, dv)
    want, _ = oracle.delta_recurrent(*ref[:5], dk ** -0.5, S0, lens)
    for final in (False, True):
        end = torch.empty_like(S) if final else None
        out = rn.retnet_delta_chunkwise(*x[:5], lengths=lengths, state_in=S, state_out=end, algo="tensor")
        done(rn)
        o, _ = oracle.delta_chunks(*ref[:5], dk ** -0.5, S0, lens, final_state=final)
        no_further(out, o, want, lens, "out")


@pytest.mark.parametrize("decay", [0.2, 0.02])
@pytest.mark.parametrize("n,Hk,H,dk,dv,lens", SHAPES)
def test_backward(rn, n, Hk, H, dk, dv, lens, decay):
    x, ref, lengths = ragged(62 + n, n, Hk, H, dk, dv, lens, decay=decay)
    got = rn.retnet_delta_backward(*x, lengths=lengths, algo="tensor")
    done(rn)
    rounded = oracle.delta_chunks_backward(*ref, dk ** -0.5, lens)
    want = oracle.delta_backward(*ref, dk ** -0.5, lens)
    for name, a, r, w in zip(("dq", "dk", "dv", "dg", "dbeta"), got, rounded, want):
        no_further(a, r, w, lens, name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,Hk,H,dk,dv,lens", SHAPES + [(150, 1, 2, 256, 64, [150, 77]),
                                                        (1100, 1, 1, 128, 64, [1100, 300, 640])])
def test_gates_gradients_of_every_head(rn, dtype, n, Hk, H, dk, dv, lens):
    """In float32 arithmetic, for each (batch, head) by itself: with 64 tokens
    and more, a head's dg and dbeta together have the size of their terms."""
    x, ref, lengths = ragged(64 + n, n, Hk, H, dk, dv, lens, dtype)
    got = rn.retnet_delta_backward(*x, lengths=lengths, algo="simt")[3:]
    done(rn)
    for a, w in zip(got, oracle.delta_backward(*ref, dk ** -0.5, lens)[3:]):
        assert err(per_head(a), per_head(w)) < bound(dtype)


@pytest.mark.parametrize("n,Hk,H,dk,dv,lens", [(2100, 1, 2, 128, 64, [2100, 700]), (2100, 1, 1, 128, 256, [64, 2100]),
                                               (1800, 2, 2, 64, 128, [1800, 0, 1000])])
def test_segments_for_every_head(rn, n, Hk, H, dk, dv, lens):
    """Walks in segments, where a state has also passed a segment's transition
    (one more S and X of the same sizes each way): at most twelve roundings of
    a norm's 2^-8 / sqrt(3) each, were none of them weakened on its way,
    sqrt(12 / 3) * 2^-8 = 7.8e-3, for each (batch, head) of 64 tokens or more."""
    x, ref, lengths = ragged(70 + n, n, Hk, H, dk, dv, lens, decay=0.02)
    out = rn.retnet_delta_chunkwise(*x[:5], lengths=lengths, algo="tensor")
    end = torch.empty(len(lens), H, dk, dv, device="cuda")
    with_state = rn.retnet_delta_chunkwise(*x[:5], lengths=lengths, state_out=end, algo="tensor")
    got = rn.retnet_delta_backward(*x, lengths=lengths, algo="tensor")
    done(rn)
    o, _ = oracle.delta_recurrent(*ref[:5], dk ** -0.5, None, lens)
    tol = 2 * 2.0 ** -8
    assert err(out, o) < tol and err(with_state, o) < tol
    for name, a, w in zip(("dq", "dk", "dv", "dg", "dbeta"), got,
                          oracle.delta_backward(*ref, dk ** -0.5, lens)):
        assert err(per_head(a), per_head(w)) < tol, name


def alike(seed, n, H, dk, dv, cos, decay):
    """As make, every key near one of its head (all the same: cos None)."""
    x, ref = make(seed, 1, n, H, H, dk, dv, "bf16", decay)
    rng = np.random.default_rng(seed)
    one = rng.standard_normal((1, 1, H, dk))
    k = one / np.linalg.norm(one, axis=-1, keepdims=True) + np.zeros((1, n, 1, 1))
    if cos is not None:
        k = cos * k + np.sqrt(1 - cos ** 2) * ref[1]
    x[1] = torch.from_numpy(k).bfloat16().cuda()
    ref[1] = x[1].double().cpu().numpy()
    return x, ref


@pytest.mark.parametrize("cos", [0.7, 0.95, None])
@pytest.mark.parametrize("n,H,dk,dv,decay", [(300, 2, 64, 64, 0.02), (500, 1, 128, 128, 0.002)])
def test_keys_that_nearly_repeat(rn, n, H, dk, dv, decay, cos):
    """Writes that mostly cancel: the rounded oracle's errors, no more (the
    roundings are independent as before).  A state's own, of writes that are
    kept to 2^-17 of themselves, from operands kept to as much (T^, W, S: as
    much again), against the norm of the writes that reach it: 2^-16."""
    x, ref = alike(80 + n, n, H, dk, dv, cos, decay)
    want, S = oracle.delta_recurrent(*ref[:5], dk ** -0.5)
    for final in (False, True):
        end = torch.empty(1, H, dk, dv, device="cuda") if final else None
        out = rn.retnet_delta_chunkwise(*x[:5], state_out=end, algo="tensor")
        done(rn)
        o, _ = oracle.delta_chunks(*ref[:5], dk ** -0.5, final_state=final)
        no_further(out, o, want, [n], "out")
    for h in range(H):
        writes, s = 0.0, np.zeros((dk, dv))
        for t in range(n):
            a = np.exp(ref[3][0, t, h])
            w = ref[4][0, t, h] * (ref[2][0, t, h] - a * ref[1][0, t, h] @ s)
            s = a * s + np.outer(ref[1][0, t, h], w)
            writes = a * a * writes + (ref[1][0, t, h] ** 2).sum() * (w ** 2).sum()
        e = np.linalg.norm(end[0, h].double().cpu().numpy() - S[0, h])
        assert record(e / np.sqrt(writes), "state / writes") < 2.0 ** -16
    got = rn.retnet_delta_backward(*x, algo="tensor")
    done(rn)
    for name, a, r, w in zip(("dq", "dk", "dv", "dg", "dbeta"), got,
                             oracle.delta_chunks_backward(*ref, dk ** -0.5),
                             oracle.delta_backward(*ref, dk ** -0.5)):
        no_further(a, r, w, [n], name)
