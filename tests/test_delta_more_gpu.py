"""The gated delta rule as its documentation allows it, where
test_delta_gpu.py does not go."""
import numpy as np
import pytest
import torch

import oracle
from helpers import record
from test_delta_gpu import DT, bound, done, err, make, rn, states  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ where tensors start
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H", [1, 3, 4])
def test_steps_through_slices_of_one_sequence(rn, dtype, H):
    """One token of one sequence is contiguous wherever it starts."""
    n, d = 9, 64
    (q, k, v, g, beta, _), ref = make(50 + H, 1, n, H, H, d, d, dtype)
    S, S0 = states(51, 1, H, d, d)
    out = torch.cat([rn.retnet_delta_recurrent(*(x[:, t:t + 1] for x in (q, k, v, g, beta)), S)
                     for t in range(n)], 1)
    done(rn)
    o, St = oracle.delta_recurrent(*ref[:5], d ** -0.5, S0)
    assert err(out, o) < bound(dtype) and err(S, St, 1) < 2e-5


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prefill_and_backward_of_later_tokens_and_sequences(rn, dtype):
    """Tokens 1 .. of one sequence with gradients written to slices, and
    lengths of the sequences 1 .. of a batch, give what copies give."""
    n, H, d = 70, 3, 64
    x, _ = make(52, 1, n, H, H, d, d, dtype)
    part, copy = [t[:, 1:] for t in x], [t[:, 1:].clone() for t in x]
    assert part[3].is_contiguous() and part[3].data_ptr() % 16
    dg, dbeta = torch.full_like(x[3], 9.0), torch.full_like(x[4], 9.0)
    got = rn.retnet_delta_backward(*part, dg=dg[:, 1:], dbeta=dbeta[:, 1:])
    for a, b in zip(got, rn.retnet_delta_backward(*copy)):
        assert torch.equal(a, b)
    assert got[3].data_ptr() == dg[:, 1:].data_ptr() and torch.equal(got[4], dbeta[:, 1:])
    assert (dg[:, 0] == 9).all() and (dbeta[:, 0] == 9).all()
    assert torch.equal(rn.retnet_delta_chunkwise(*part[:5]), rn.retnet_delta_chunkwise(*copy[:5]))

    B = 4
    x, _ = make(53, B, n, H, H, d, d, dtype)
    lengths = torch.tensor([5, 0, 70, 33], dtype=torch.int32, device="cuda")
    S, mine = torch.zeros(2, B - 1, H, d, d, device="cuda")
    part = [t[1:] for t in x]
    for call in (rn.retnet_delta_chunkwise, lambda *a, **kw: rn.retnet_delta_recurrent(
            *a, S.zero_() if kw["lengths"].data_ptr() % 16 else mine.zero_(), **kw)):
        assert torch.equal(call(*part[:5], lengths=lengths[1:]),
                           call(*part[:5], lengths=lengths[1:].clone()))
    assert torch.equal(S, mine)
    for a, b in zip(rn.retnet_delta_backward(*part, lengths=lengths[1:]),
                    rn.retnet_delta_backward(*part, lengths=lengths[1:].clone())):
        assert torch.equal(a, b)
    done(rn)


# ------------------------------------------------------------------ gates
@pytest.mark.parametrize("dtype,algo", [("bf16", "auto"), ("bf16", "simt"), ("f32", "auto")])
@pytest.mark.parametrize("Hk,H,dk,dv", [(2, 2, 64, 64), (1, 2, 128, 256)])
def test_values_of_tokens_that_write_nothing_have_no_gradient(rn, dtype, algo, Hk, H, dk, dv):
    """dv = beta r: exactly 0 where beta is."""
    B, n = 2, 200
    x, _ = make(54, B, n, Hk, H, dk, dv, dtype)
    off = torch.rand(B, n, H, device="cuda", generator=torch.Generator("cuda").manual_seed(1)) < 0.3
    off[:, 64:128], off[1, :, 0], off[:, 5], off[:, 70] = True, True, False, False
    x[4][off] = 0.0
    lengths = torch.tensor([200, 170], dtype=torch.int32, device="cuda")
    got = rn.retnet_delta_backward(*x, lengths=lengths, algo=algo)
    done(rn)
    assert not got[2][off].any()
    on = ~off
    on[1, 170:] = False
    assert got[2][on].any(-1).all() and got[4][:, :170][off[:, :170]].abs().max() > 0
    want = oracle.delta_backward(*(t.double().cpu().numpy() for t in x), dk ** -0.5, [200, 170])
    for b in range(B):
        for h in range(H):
            if want[2][b, :, h].any():
                e = np.linalg.norm(got[2][b, :, h].double().cpu().numpy() - want[2][b, :, h])
                assert e < bound(dtype, dtype == "bf16" and algo == "auto") * np.linalg.norm(want[2][b, :, h])


@pytest.mark.parametrize("dtype,algo", [("bf16", "tensor"), ("bf16", "simt"), ("f32", "auto")])
@pytest.mark.parametrize("n,Hk,H,dk,dv", [(200, 2, 2, 64, 64), (130, 1, 2, 128, 256), (1500, 1, 1, 128, 64)])
def test_backward_past_tokens_that_write_nothing_whatever_they_hold(rn, dtype, algo, n, Hk, H, dk, dv):
    """beta = 0 at tokens whose v (and, for some, k) is far beyond the others':
    x is 0 there, so no other token's gradient sees it."""
    B = 2
    (q, k, v, g, beta, do), _ = make(68, B, n, Hk, H, dk, dv, dtype, decay=0.05)
    rng = np.random.default_rng(69)
    off = torch.from_numpy(rng.random((B, n)) < 0.2).cuda()
    off[:, :3], off[:, 64:70] = torch.tensor([True, False, False], device="cuda"), True
    beta[off] = 0.0
    v[off] *= 1e30
    k[off] *= 100.0
    x = [q, k, v, g, beta, do]
    got = rn.retnet_delta_backward(*x, algo=algo)
    v2 = v.clone()
    v2[off] = torch.finfo(v.dtype).min
    lowest = rn.retnet_delta_backward(q, k, v2, g, beta, do, algo=algo)
    done(rn)
    tol = bound(dtype, dtype == "bf16" and algo == "tensor")
    ref = [t.double().cpu().numpy() for t in x]
    want = oracle.delta_backward(*ref, dk ** -0.5)
    at = off.cpu().numpy()
    for i, (name, a, b, w) in enumerate(zip(("dq", "dk", "dv", "dg", "dbeta"), got, lowest, want)):
        if name != "dbeta":
            assert torch.equal(a, b), name
        for here in (at, ~at):
            a_, w_ = a.double().cpu().numpy()[here], w[here]
            assert np.isfinite(a_).all(), name
            e, size = np.linalg.norm(a_ - w_), np.linalg.norm(w_)
            if name in ("dk", "dv") and here is at:        # nothing is written: nothing to change
                assert e == size == 0, name
            else:
                assert record(e / size, name) < tol, name
    assert torch.equal(got[4][~off], lowest[4][~off])


# ------------------------------------------------------------------ many sequences
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hk,H,dk,dv", [(1, 4, 64, 256), (2, 4, 128, 256), (4, 4, 256, 256),
                                        (8, 24, 128, 64)])
def test_step_of_many_sequences_of_which_some_are_over(rn, dtype, Hk, H, dk, dv):
    """A step's CTAs (444) take several (sequence, head, 32 columns) each, and
    pass over those of a sequence that is over."""
    B = 71
    assert B * H * dv // 32 > 3 * 444
    (q, k, v, g, beta, _), ref = make(55, B, 1, Hk, H, dk, dv, dtype)
    lens = np.random.default_rng(56).integers(-1, 3, B)
    lens[:4] = 0, 1, 0, 0
    over = torch.from_numpy(lens < 1).cuda()
    for x, r in zip((q, k, v, g, beta), ref):
        x[over], r[lens < 1] = float("nan"), 0.0
    S, S0 = states(57, B, H, dk, dv)
    out = torch.full_like(v, 7.0)
    lengths = torch.from_numpy(lens.astype(np.int32)).cuda()
    rn.retnet_delta_recurrent(q, k, v, g, beta, S, lengths=lengths, out=out)
    done(rn)
    o, St = oracle.delta_recurrent(*ref[:5], dk ** -0.5, S0, lens.tolist())
    assert (out[over] == 7).all() and torch.equal(S[over].cpu(), torch.from_numpy(S0[lens < 1]).float())
    assert err(out[~over], o[lens > 0]) < bound(dtype)
    assert err(S, St, 1) < 2e-5


# ------------------------------------------------------------------ infinities and NaN
@pytest.mark.parametrize("dtype,algo,chunk", [("bf16", "tensor", 64), ("bf16", "simt", 1),
                                              ("f32", "auto", 1)])
@pytest.mark.parametrize("which", ["v", "k", "g"])
def test_where_a_value_that_is_not_finite_goes(rn, dtype, algo, chunk, which):
    """To the outputs from its token on, of its head (of its channel, for v);
    on the tensor cores also to the earlier tokens of its chunk of 64.  Other
    sequences, heads, channels and chunks before keep their bits, and the
    gradients of other sequences and heads theirs."""
    B, n, H, d, at = 2, 200, 2, 64, 100
    x, _ = make(58, B, n, H, H, d, d, dtype)
    clean = rn.retnet_delta_chunkwise(*x[:5], algo=algo)
    grads = rn.retnet_delta_backward(*x, algo=algo)
    bad = [t.clone() for t in x]
    if which == "v":
        bad[2][0, at, 1, 5] = float("inf")
    elif which == "k":
        bad[1][0, at, 1, 5] = float("nan")
    else:
        bad[3][0, at, 1] = float("nan")
    out = rn.retnet_delta_chunkwise(*bad[:5], algo=algo)
    bad_grads = rn.retnet_delta_backward(*bad, algo=algo)
    done(rn)
    for a, b in zip((out, *bad_grads), (clean, *grads)):
        assert torch.equal(a[1], b[1]) and torch.equal(a[0, :, 0], b[0, :, 0])
    start = at // chunk * chunk
    assert torch.equal(out[0, :start, 1], clean[0, :start, 1])
    mine = out[0, at:, 1, 5:6] if which == "v" else out[0, at:, 1]
    assert not torch.isfinite(mine).any()
    if which == "v":
        rest = [c for c in range(d) if c != 5]
        assert torch.equal(out[0, :, 1, rest], clean[0, :, 1, rest])


@pytest.mark.parametrize("dtype,algo", [("bf16", "tensor"), ("bf16", "simt"), ("f32", "auto")])
def test_a_query_that_is_not_finite_spoils_its_own_output_alone(rn, dtype, algo):
    B, n, H, d, at = 2, 200, 2, 64, 100
    x, _ = make(59, B, n, 1, H, d, d, dtype)
    clean = rn.retnet_delta_chunkwise(*x[:5], algo=algo)
    x[0][0, at, 0, 5] = float("nan")
    out = rn.retnet_delta_chunkwise(*x[:5], algo=algo)
    done(rn)
    assert torch.isnan(out[0, at]).all()
    out[0, at] = clean[0, at]
    assert torch.equal(out, clean)


# ------------------------------------------------------------------ what the bits follow from
@pytest.mark.parametrize("dtype,B,n,Hk,H,dk,dv", [("bf16", 2, 200, 1, 2, 128, 128),
                                                  ("bf16", 1, 2000, 1, 1, 64, 256),
                                                  ("f32", 1, 1500, 1, 2, 128, 64)])
def test_equal_calls_give_equal_bits_whatever_the_workspace_held(rn, dtype, B, n, Hk, H, dk, dv):
    """Whole walks and walks in segments; workspaces of zeros, of NaN (all
    bits set) and of large numbers."""
    x, _ = make(65, B, n, Hk, H, dk, dv, dtype)
    lengths = torch.tensor([n - 70, n][-B:], dtype=torch.int32, device="cuda")
    shape = (B, H, Hk, n, dk, dv, DT[dtype])
    room = [rn.retnet_workspace(size(*shape), "cuda") for size in (
        rn.retnet_delta_workspace_size, rn.retnet_delta_backward_workspace_size)]
    seen = []
    for fill in (0x00, 0xFF, 0x7E):
        for ws in room:
            ws.fill_(fill)
        S = torch.full((B, H, dk, dv), float("nan"), device="cuda")
        seen.append((rn.retnet_delta_chunkwise(*x[:5], lengths=lengths, state_out=S, workspace=room[0]),
                     rn.retnet_delta_chunkwise(*x[:5], lengths=lengths, workspace=room[0].fill_(fill)), S,
                     *rn.retnet_delta_backward(*x, lengths=lengths, workspace=room[1])))
    done(rn)
    for a, *others in zip(*seen):
        assert torch.isfinite(a).all() and all(torch.equal(a, b) for b in others)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_recurrent_forms_give_a_sequence_the_same_bits_in_any_batch(rn, dtype):
    B, n, H, dk, dv = 5, 90, 2, 128, 64
    x, _ = make(66, B, n, H, H, dk, dv, dtype)
    S, _ = states(67, B, H, dk, dv)
    many = S.clone()
    one = torch.empty_like(S)
    out = rn.retnet_delta_recurrent(*x[:5], many)
    simt = rn.retnet_delta_chunkwise(*x[:5], state_in=S, state_out=one, algo="simt")
    for b in range(B):
        alone, s = [t[b:b + 1] for t in x[:5]], S[b:b + 1].clone()
        assert torch.equal(rn.retnet_delta_recurrent(*alone, s), out[b:b + 1])
        assert torch.equal(s, many[b:b + 1])
        assert torch.equal(rn.retnet_delta_chunkwise(*alone, state_in=S[b:b + 1], algo="simt"),
                           simt[b:b + 1])
    assert torch.equal(simt, out) and torch.equal(one, many)
    done(rn)


@pytest.mark.parametrize("B,n,Hk,H,dk,dv", [(4, 1, 1, 1, 128, 256), (1, 2, 1, 1, 64, 64), (2, 1, 1, 1, 128, 128),
                                            (2, 3, 2, 4, 64, 128), (1, 16, 2, 16, 128, 64), (5, 4, 1, 3, 64, 256)])
def test_backward_of_a_few_tokens_is_rounded_once(rn, B, n, Hk, H, dk, dv):
    """A handful of dg and dbeta may all be near 0 beside their terms, so these
    calls go in float32 arithmetic: every gradient of every token to one
    rounding of the result (2^-8 of a value at most) and float32's own, 2e-5 of
    terms up to five times the sum's norm, in each of several draws."""
    for seed in range(12):
        x, ref = make(100 + seed, B, n, Hk, H, dk, dv, "bf16")
        got = rn.retnet_delta_backward(*x)
        done(rn)
        for name, a, w in zip(("dq", "dk", "dv", "dg", "dbeta"), got, oracle.delta_backward(*ref, dk ** -0.5)):
            a, size = a.double().cpu().numpy(), np.linalg.norm(w)
            assert np.linalg.norm(a - w) <= (2.0 ** -8 + 1e-4) * size, (name, seed)
