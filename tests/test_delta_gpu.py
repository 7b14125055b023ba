"""GPU parity of the gated delta rule against the float64 oracle: recurrent,
chunkwise and backward, over types, head layouts, lengths and gates.

Error measure: ||gpu - oracle|| / ||oracle|| (2-norm) per (batch, head), the
worst one.  Bounds, from the roundings on the way:
  float32 math: a product's or a sum's rounding is 2^-24 of its size; a dot
    product over d <= 256 in partial sums of 32 and a few hundred tokens of a
    recurrence that does not grow (|k| = 1, beta <= 1, g <= 0) gather some
    hundred of them, 200 * 2^-24 = 1.2e-5; the bound is 2e-5.
  bf16 through float32 math: one rounding of the result, at most 2^-8 of each
    value and so of the norm, plus the above.
  bf16 on the tensor cores: operands are rounded to bf16 on the way, at most
    ten of them behind one another (for an output: T, W, S, X twice, Q, P and
    the result; for a gradient D, dX, T, dR, the pair products, S or X and the
    result).  Each moves a value by at most 2^-8, uniformly spread by
    2^-8 / sqrt(3); ten independent ones give sqrt(10 / 3) * 2^-8 = 7.1e-3
    of the norm where nothing cancels, and twice that is the bound, 1.5e-2.
    The final state is held to float32 precision in two bf16 parts (2^-18
    each): 6 such roundings and the float32 sums, bound 3e-5.
"""
import numpy as np
import pytest
import torch

import oracle
from helpers import record

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def rn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import linear_recurrent_sequence_02_b200 as lib
    from linear_recurrent_sequence_02_b200.build import build
    build()
    lib.load_library()
    return lib


def bound(dtype, tensor=False):
    return 2e-5 if dtype == "f32" else 1.5e-2 if tensor else 2.0 ** -8 + 2e-5


def tensor_path(dtype, dk, algo="auto", n=64):
    return dtype == "bf16" and dk in (64, 128) and algo != "simt" and (n > 16 or algo == "tensor")


def err(got, want, head_axis=2):
    """Worst relative 2-norm error over (batch, head)."""
    got = got.detach().double().cpu().numpy()
    assert got.shape == want.shape
    if not got.size:
        return 0.0
    assert np.isfinite(got).all()
    g = np.moveaxis(got, head_axis, 1).reshape(got.shape[0] * got.shape[head_axis], -1)
    w = np.moveaxis(want, head_axis, 1).reshape(g.shape)
    num, den = np.linalg.norm(g - w, axis=1), np.linalg.norm(w, axis=1)
    assert (num[den == 0] == 0).all()
    return record(float((num[den > 0] / den[den > 0]).max(initial=0.0)), "2-norm")


def together(w, a):
    """dg and dbeta, one number a token and head, as one (batch, head).  Each
    is a dot product: roundings of its d terms t_i, independent and of
    relative size u, move it by u sqrt(sum t_i^2), which is what a sum of d
    terms of either sign typically comes to, but not the one at hand, that may
    be near 0 (one token: t_i of 0.01, 128 of them, sum 0.0024 where 0.1 is
    typical, and a rounding's 2^-8 * 0.1 is 16 % of it).  The bound holds
    relative to all of them together."""
    return (w.reshape(1, -1, 1, 1), a.reshape(1, -1, 1, 1)) if w.ndim == 3 else (w, a)


def make(seed, B, n, Hk, H, dk, dv, dtype, decay=0.2):
    """Inputs on the GPU and the same values (after rounding) in float64."""
    rng = np.random.default_rng(seed)
    q, k = rng.standard_normal((2, B, n, Hk, dk))
    q /= np.linalg.norm(q, axis=-1, keepdims=True)
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    v, do = rng.standard_normal((2, B, n, H, dv))
    g = -decay * np.exp(0.7 * rng.standard_normal((B, n, H)))
    beta = 1.0 / (1.0 + np.exp(-rng.standard_normal((B, n, H))))
    gpu = [torch.from_numpy(np.ascontiguousarray(x)).to(DT[dtype]).cuda()
           for x in (q, k, v, g, beta, do)]
    return gpu, [x.double().cpu().numpy() for x in gpu]


def states(seed, B, H, dk, dv):
    s = np.random.default_rng(seed).standard_normal((B, H, dk, dv)).astype(np.float32) * 0.3
    return torch.from_numpy(s).cuda(), s.astype(np.float64)


def done(rn):
    torch.cuda.synchronize()
    rn.retnet_check_device_errors()


# ------------------------------------------------------------------ recurrent
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hk,H,dk,dv,n", [(4, 4, 64, 64, 1), (2, 6, 128, 64, 9),
                                          (1, 3, 256, 256, 2), (3, 3, 64, 256, 17)])
def test_recurrent(rn, dtype, Hk, H, dk, dv, n):
    B = 3
    (q, k, v, g, beta, _), ref = make(dk + n, B, n, Hk, H, dk, dv, dtype)
    S, S0 = states(7, B, H, dk, dv)
    out = rn.retnet_delta_recurrent(q, k, v, g, beta, S, scale=0.3)
    done(rn)
    o, St = oracle.delta_recurrent(*ref[:5], 0.3, S0)
    assert err(out, o) < bound(dtype)
    assert err(S, St, 1) < 2e-5


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [128, 256])
def test_recurrent_run_is_its_single_steps(rn, dtype, d):
    """Both in float32 arithmetic, sums in another order: the bound of float32
    math, and for bf16 outputs two roundings of nearly the same value."""
    B, n, H = 2, 11, 3
    (q, k, v, g, beta, _), _ = make(5, B, n, H, H, d, d, dtype)
    S, _ = states(8, B, H, d, d)
    S1, S2 = S.clone(), S.clone()
    out = rn.retnet_delta_recurrent(q, k, v, g, beta, S1)
    one = [rn.retnet_delta_recurrent(*(x[:, t:t + 1].contiguous() for x in (q, k, v, g, beta)), S2)
           for t in range(n)]
    done(rn)
    assert err(out, torch.cat(one, 1).double().cpu().numpy()) < bound(dtype)
    assert err(S1, S2.double().cpu().numpy(), 1) < 2e-5


@pytest.mark.parametrize("n", [1, 5])
def test_recurrent_lengths_leave_the_rest_alone(rn, n):
    B, H, dk, dv = 4, 2, 64, 128
    (q, k, v, g, beta, _), ref = make(6, B, n, H, H, dk, dv, "bf16")
    lengths = torch.tensor([n, 0, -3, n + 9], dtype=torch.int32, device="cuda")
    for x in (q, k, v, g, beta):
        x[1:3] = float("nan")                       # behind the lengths: never read
    for x in ref[:5]:
        x[1:3] = 0.0
    S, S0 = states(9, B, H, dk, dv)
    out = torch.full_like(v, 7.0)
    rn.retnet_delta_recurrent(q, k, v, g, beta, S, lengths=lengths, out=out)
    done(rn)
    o, St = oracle.delta_recurrent(*ref[:5], dk ** -0.5, S0, lengths.tolist())
    assert (out[1:3] == 7).all() and torch.equal(S[1:3].cpu(), torch.from_numpy(S0[1:3]).float())
    assert err(out[0::3], o[0::3]) < bound("bf16")
    assert err(S, St, 1) < 2e-5


# ------------------------------------------------------------------ chunkwise
SHAPES = [  # B, n, Hk, H, dk, dv
    (2, 1, 2, 2, 128, 128), (1, 63, 1, 2, 64, 64), (2, 64, 1, 1, 128, 64), (1, 65, 2, 4, 128, 256),
    (3, 200, 1, 3, 64, 128), (1, 321, 2, 2, 128, 128), (1, 130, 1, 1, 256, 128),
]


@pytest.mark.parametrize("dtype,algo", [("f32", "auto"), ("bf16", "auto"), ("bf16", "simt"),
                                        ("bf16", "tensor")])
@pytest.mark.parametrize("B,n,Hk,H,dk,dv", SHAPES)
def test_chunkwise(rn, dtype, algo, B, n, Hk, H, dk, dv):
    (q, k, v, g, beta, _), ref = make(n, B, n, Hk, H, dk, dv, dtype)
    if algo == "tensor" and dk == 256:              # there is none
        with pytest.raises(rn.RetnetError):
            rn.retnet_delta_chunkwise(q, k, v, g, beta, algo=algo)
        return
    S, S0 = states(10, B, H, dk, dv)
    end = torch.empty_like(S)
    out = rn.retnet_delta_chunkwise(q, k, v, g, beta, state_in=S, state_out=end, algo=algo)
    plain = rn.retnet_delta_chunkwise(q, k, v, g, beta, algo=algo)
    done(rn)
    tc = tensor_path(dtype, dk, algo, n)
    o, St = oracle.delta_recurrent(*ref[:5], dk ** -0.5, S0)
    assert err(out, o) < bound(dtype, tc)
    assert err(end, St, 1) < (3e-5 if tc else 2e-5)
    assert torch.equal(S.cpu(), torch.from_numpy(S0).float())
    o, _ = oracle.delta_recurrent(*ref[:5], dk ** -0.5)
    assert err(plain, o) < bound(dtype, tc)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(64, 128), (128, 256)])
def test_chunkwise_lengths(rn, dtype, dk, dv):
    """Padded batch: rows behind a length are NaN and neither read nor written."""
    B, n, Hk, H = 5, 150, 1, 2
    (q, k, v, g, beta, _), ref = make(11, B, n, Hk, H, dk, dv, dtype)
    lens = [150, 0, 1, 64, 129]
    for x, r in zip((q, k, v, g, beta), ref):
        for b, c in enumerate(lens):
            x[b, c:] = float("nan")
            r[b, c:] = 0.0
    S, S0 = states(12, B, H, dk, dv)
    out = torch.full_like(v, -3.0)
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    rn.retnet_delta_chunkwise(q, k, v, g, beta, lengths=lengths, state_in=S, state_out=S, out=out)
    done(rn)
    o, St = oracle.delta_recurrent(*ref[:5], dk ** -0.5, S0, lens)
    for b, c in enumerate(lens):
        assert (out[b, c:] == -3).all()
        out[b, c:] = 0
    assert err(out, o) < bound(dtype, tensor_path(dtype, dk))
    assert err(S, St, 1) < 3e-5


@pytest.mark.parametrize("dk,dv,H", [(128, 128, 2), (64, 256, 1), (128, 64, 3)])
def test_chunkwise_long_with_few_heads(rn, dk, dv, H):
    """Long enough for a walk in segments (4000 tokens, few heads), uneven
    lengths that end in different segments, the state updated in place."""
    B, n = 3, 4000
    (q, k, v, g, beta, _), ref = make(22, B, n, 1, H, dk, dv, "bf16", decay=0.02)
    lens = [4000, 0, 1500]
    for x, r in zip((q, k, v, g, beta), ref):
        for b, c in enumerate(lens):
            x[b, c:] = float("nan")
            r[b, c:] = 0.0
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    S, S0 = states(23, B, H, dk, dv)
    out, plain = torch.full_like(v, 5.0), torch.full_like(v, 5.0)
    rn.retnet_delta_chunkwise(q, k, v, g, beta, lengths=lengths, state_in=S, out=plain)
    rn.retnet_delta_chunkwise(q, k, v, g, beta, lengths=lengths, state_in=S, state_out=S, out=out)
    done(rn)
    o, St = oracle.delta_recurrent(*ref[:5], dk ** -0.5, S0, lens)
    for b, c in enumerate(lens):
        assert (out[b, c:] == 5).all() and (plain[b, c:] == 5).all()
        out[b, c:] = plain[b, c:] = 0
    assert err(out, o) < bound("bf16", True) and err(plain, o) < bound("bf16", True)
    # a state passes through the segments before it in two more parts each way
    assert err(S, St, 1) < 3e-5


@pytest.mark.parametrize("dk,dv,H,lens", [(128, 64, 2, [1501, 0, 700]), (64, 256, 3, [900, 64, 1500]),
                                          (128, 128, 1, [1501, 1501, 1])])
def test_float32_prefill_in_segments(rn, dk, dv, H, lens):
    """As above in float32 (the walk of single tokens in segments)."""
    B, n = 3, 1501
    (q, k, v, g, beta, _), ref = make(24, B, n, 1, H, dk, dv, "f32", decay=0.02)
    for x, r in zip((q, k, v, g, beta), ref):
        for b, c in enumerate(lens):
            x[b, c:] = float("nan")
            r[b, c:] = 0.0
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    assert rn.retnet_delta_workspace_size(B, H, 1, n, dk, dv, torch.float32) > 0
    S, S0 = states(25, B, H, dk, dv)
    whole_S = S.clone()
    out, whole = torch.full_like(v, 5.0), torch.full_like(v, 5.0)
    rn.retnet_delta_chunkwise(q, k, v, g, beta, lengths=lengths, state_in=S, state_out=S, out=out)
    rn.retnet_delta_chunkwise(q, k, v, g, beta, lengths=lengths, state_in=whole_S,
                              state_out=whole_S, out=whole, algo="simt")
    done(rn)
    o, St = oracle.delta_recurrent(*ref[:5], dk ** -0.5, S0, lens)
    for b, c in enumerate(lens):
        assert (out[b, c:] == 5).all() and (whole[b, c:] == 5).all()
        out[b, c:] = whole[b, c:] = 0
    for got, want, axis in ((out, o, 2), (whole, o, 2), (S, St, 1), (whole_S, St, 1)):
        assert err(got, want, axis) < bound("f32")


@pytest.mark.parametrize("dtype,dk,dv,Hk,H,lens", [
    ("f32", 64, 128, 1, 2, [1100, 0, 640]), ("f32", 128, 64, 2, 2, [64, 1100, 65]),
    ("bf16", 128, 128, 1, 1, [700, 1100, 1])])
def test_float32_backward_in_segments(rn, dtype, dk, dv, Hk, H, lens):
    """Float32 arithmetic, on either type."""
    B, n = 3, 1100
    x, ref = make(26, B, n, Hk, H, dk, dv, dtype, decay=0.02)
    for t, r in zip(x, ref):
        for b, c in enumerate(lens):
            t[b, c:] = float("nan")
            r[b, c:] = 0.0
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = rn.retnet_delta_backward(*x, lengths=lengths, algo="simt")
    done(rn)
    want = oracle.delta_backward(*ref, dk ** -0.5, lens)
    for name, a, w in zip(("dq", "dk", "dv", "dg", "dbeta"), got, want):
        for b, c in enumerate(lens):
            assert not a[b, c:].any(), name
        w, a = together(w, a)
        assert err(a, w) < bound(dtype), name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_chunkwise_gates_at_their_ends(rn, dtype):
    """g: -inf (the state is emptied), 0, and far below what float32 resolves;
    beta: 0 (nothing is written) and 1; a chunk of nothing but either."""
    B, n, H, d = 1, 256, 2, 64
    (q, k, v, g, beta, _), ref = make(13, B, n, H, H, d, d, dtype, decay=2.0)
    g[:, 10], g[:, 70:75], g[:, 100], beta[:, 30:40] = -float("inf"), 0.0, -5000.0, 0.0
    g[:, 128:192, 0], beta[:, 128:192, 1] = 0.0, 0.0
    beta[:, 50:60] = 1.0
    ref = [x.double().cpu().numpy() for x in (q, k, v, g, beta)]
    end = torch.empty(B, H, d, d, device="cuda")
    out = rn.retnet_delta_chunkwise(q, k, v, g, beta, state_out=end)
    done(rn)
    o, St = oracle.delta_recurrent(*ref, d ** -0.5)
    assert err(out, o) < bound(dtype, dtype == "bf16")
    assert err(end, St, 1) < 3e-5


def test_chunkwise_in_parts_continues_into_steps(rn):
    """A prompt in two prefills, then decoding from its state, against the whole."""
    B, n, H, d = 2, 300, 2, 128
    (q, k, v, g, beta, _), ref = make(14, B, n, H, H, d, d, "bf16")
    S = torch.empty(B, H, d, d, device="cuda")
    parts, at = [], 0
    for end in (100, 290):
        x = [t[:, at:end].contiguous() for t in (q, k, v, g, beta)]
        parts.append(rn.retnet_delta_chunkwise(*x, state_in=S if at else None, state_out=S))
        at = end
    for t in range(at, n):
        x = [t_[:, t:t + 1].contiguous() for t_ in (q, k, v, g, beta)]
        parts.append(rn.retnet_delta_recurrent(*x, S))
    done(rn)
    o, St = oracle.delta_recurrent(*ref[:5], d ** -0.5)
    assert err(torch.cat(parts, 1), o) < bound("bf16", True)
    assert err(S, St, 1) < 6e-5                     # two prefills' roundings and the steps'


def test_empty_calls(rn):
    (q, k, v, g, beta, do), _ = make(15, 2, 4, 1, 2, 64, 64, "bf16")
    e = [x[:, :0].contiguous() for x in (q, k, v, g, beta, do)]
    S, S0 = states(16, 2, 2, 64, 64)
    end = torch.empty_like(S)
    assert rn.retnet_delta_chunkwise(*e[:5], state_in=S, state_out=end).shape == (2, 0, 2, 64)
    assert torch.equal(end, S)
    rn.retnet_delta_chunkwise(*e[:5], state_out=end)
    assert not end.any()
    rn.retnet_delta_recurrent(*e[:5], S)
    assert torch.equal(S.cpu(), torch.from_numpy(S0).float())
    assert rn.retnet_delta_backward(*e)[0].shape == (2, 0, 1, 64)
    none = [x[:0] for x in (q, k, v, g, beta, do)]
    assert rn.retnet_delta_chunkwise(*none[:5]).shape[0] == 0
    done(rn)


# ------------------------------------------------------------------ backward
@pytest.mark.parametrize("dtype,algo", [("f32", "auto"), ("bf16", "auto"), ("bf16", "simt")])
@pytest.mark.parametrize("B,n,Hk,H,dk,dv", SHAPES)
def test_backward(rn, dtype, algo, B, n, Hk, H, dk, dv):
    x, ref = make(n + 1, B, n, Hk, H, dk, dv, dtype)
    got = rn.retnet_delta_backward(*x, algo=algo)
    again = rn.retnet_delta_backward(*x, algo=algo)
    done(rn)
    want = oracle.delta_backward(*ref, dk ** -0.5)
    tol = bound(dtype, tensor_path(dtype, dk, algo))
    for name, a, b, w in zip(("dq", "dk", "dv", "dg", "dbeta"), got, again, want):
        assert torch.equal(a, b), name
        w, a = together(w, a)
        if n == 1 and name == "dg":                 # nothing before the first token: dg is 0
            assert not w.any() and a.abs().max() == 0
            continue
        assert err(a, w) < tol, name


def test_backward_of_many_chunks(rn):
    """Several chunks for every CTA that walks over them, with uneven lengths."""
    B, n, Hk, H, dk, dv = 3, 1100, 4, 8, 64, 128
    x, ref = make(21, B, n, Hk, H, dk, dv, "bf16")
    lens = [1100, 500, 1037]
    for r in ref:
        for b, c in enumerate(lens):
            r[b, c:] = 0.0
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = rn.retnet_delta_backward(*x, lengths=lengths)
    again = [rn.retnet_delta_backward(*x, lengths=lengths) for _ in range(3)]
    done(rn)
    want = oracle.delta_backward(*ref, dk ** -0.5, lens)
    for i, (name, a, w) in enumerate(zip(("dq", "dk", "dv", "dg", "dbeta"), got, want)):
        assert all(torch.equal(a, g[i]) for g in again), name
        w, a = together(w, a)
        assert err(a, w) < bound("bf16", True), name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_backward_lengths_and_gates(rn, dtype):
    B, n, Hk, H, dk, dv = 4, 140, 2, 4, 64, 64
    (q, k, v, g, beta, do), _ = make(17, B, n, Hk, H, dk, dv, dtype)
    g[:, 20], g[:, 66], beta[:, 30], beta[:, 40] = -float("inf"), 0.0, 0.0, 1.0
    x = [q, k, v, g, beta, do]
    lens = [140, 0, 64, 65]
    ref = [t.double().cpu().numpy() for t in x]
    for t, r in zip(x, ref):
        for b, c in enumerate(lens):
            t[b, c:] = float("nan")
            r[b, c:] = 0.0
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = rn.retnet_delta_backward(*x, lengths=lengths)
    done(rn)
    want = oracle.delta_backward(*ref, dk ** -0.5, lens)
    for name, a, w in zip(("dq", "dk", "dv", "dg", "dbeta"), got, want):
        for b, c in enumerate(lens):
            assert not a[b, c:].any(), name
        w, a = together(w, a)
        assert err(a, w) < bound(dtype, dtype == "bf16"), name


@pytest.mark.parametrize("dk,dv,Hk,H,lens", [(128, 64, 1, 2, [2100, 700]), (64, 256, 2, 2, [1, 2100]),
                                             (64, 64, 8, 16, [2100])])
def test_backward_long_with_few_heads(rn, dk, dv, Hk, H, lens):
    """Long enough for walks in segments, of which some may be empty."""
    B, n = len(lens), 2100
    x, ref = make(27, B, n, Hk, H, dk, dv, "bf16", decay=0.02)
    for t, r in zip(x, ref):
        for b, c in enumerate(lens):
            t[b, c:] = float("nan")
            r[b, c:] = 0.0
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = rn.retnet_delta_backward(*x, lengths=lengths)
    done(rn)
    want = oracle.delta_backward(*ref, dk ** -0.5, lens)
    for name, a, w in zip(("dq", "dk", "dv", "dg", "dbeta"), got, want):
        for b, c in enumerate(lens):
            assert not a[b, c:].any(), name
        w, a = together(w, a)
        assert err(a, w) < bound("bf16", True), name


# ------------------------------------------------------------------ as a program uses them
def test_captured_graph_and_another_stream(rn):
    """A step and a prefill captured into one graph, replayed on new inputs."""
    B, n, H, d = 2, 130, 2, 128
    x, _ = make(18, B, n, H, H, d, d, "bf16")
    y, _ = make(19, B, n, H, H, d, d, "bf16")
    ws = rn.retnet_workspace(rn.retnet_delta_workspace_size(B, H, H, n, d, d, torch.bfloat16),
                             "cuda")
    S, out = torch.empty(B, H, d, d, device="cuda"), torch.empty_like(x[2])
    step_out = torch.empty_like(x[2][:, :1])
    steps = [t[:, :1].contiguous() for t in x[:5]]

    def call():
        rn.retnet_delta_chunkwise(*x[:5], state_out=S, out=out, workspace=ws)
        rn.retnet_delta_recurrent(*steps, S, out=step_out)

    call()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        call()
    for a, b in zip(x, y):
        a.copy_(b)
    for a, b in zip(steps, x):
        a.copy_(b[:, :1])
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (out, S, step_out)]
    with torch.cuda.stream(stream):
        call()
    done(rn)
    stream.synchronize()
    for a, b in zip(got, (out, S, step_out)):
        assert torch.equal(a, b)


def test_block_of_norms_projections_and_delta_rule(rn):
    """norm -> projections -> delta rule -> gated head norm -> projection ->
    residual norm, once over a prompt and once as prompt then steps."""
    B, n, H, d, hidden = 2, 96, 2, 128, 256
    torch.manual_seed(0)
    bf = dict(device="cuda", dtype=torch.bfloat16)
    x = torch.randn(B, n, hidden, **bf)
    w_qkvg = torch.randn(4 * H * d, hidden, **bf) / 16
    w_o = torch.randn(hidden, H * d, **bf) / 16
    gates = torch.randn(B, n, 2, H, **bf)
    g, beta = -torch.nn.functional.softplus(gates[:, :, 0]), torch.sigmoid(gates[:, :, 1])
    weight = torch.rand(hidden, device="cuda") + 0.5

    def block(x, g, beta, run):
        _, n1 = rn.retnet_residual_norm(x, torch.zeros_like(x), post_norm=False, pre_weight=weight)
        y = rn.retnet_linear(n1, w_qkvg).view(*x.shape[:2], 4, H, d)
        q, k = (torch.nn.functional.normalize(y[:, :, i].float(), dim=-1).bfloat16()
                for i in (0, 1))
        o = run(q.contiguous(), k.contiguous(), y[:, :, 2].contiguous(), g.contiguous(),
                beta.contiguous())
        o = rn.retnet_groupnorm_swish(o, y[:, :, 3].contiguous())
        y = rn.retnet_linear(o.view(*x.shape[:2], H * d), w_o)
        return rn.retnet_residual_norm(x, y, post_weight=weight, pre_weight=weight,
                                       residual_scale=0.5)

    whole = block(x, g, beta, rn.retnet_delta_chunkwise)
    S = torch.empty(B, H, d, d, device="cuda")
    cut = 70
    first = block(x[:, :cut].contiguous(), g[:, :cut], beta[:, :cut],
                  lambda *a: rn.retnet_delta_chunkwise(*a, state_out=S))
    rest = [block(x[:, t:t + 1].contiguous(), g[:, t:t + 1], beta[:, t:t + 1],
                  lambda *a: rn.retnet_delta_recurrent(*a, S)) for t in range(cut, n)]
    done(rn)
    for i in range(2):
        parts = torch.cat([first[i]] + [r[i] for r in rest], 1).double()
        w = whole[i].double()
        # both ways round the delta rule's output (1.5e-2) and, of that output,
        # the head norm and the projection keep the relative size
        assert ((parts - w).norm() / w.norm()).item() < 3e-2


def test_training_step_through_autograd(rn):
    """The pair of entry points as a torch autograd function; its gradients
    against differences of the loss along the gradient."""
    class Delta(torch.autograd.Function):
        @staticmethod
        def forward(ctx, *x):
            ctx.save_for_backward(*x)
            return rn.retnet_delta_chunkwise(*x)

        @staticmethod
        def backward(ctx, d_out):
            return rn.retnet_delta_backward(*ctx.saved_tensors, d_out.contiguous())

    B, n, H, d = 1, 100, 2, 64
    x, _ = make(20, B, n, H, H, d, d, "f32")
    w = x.pop()
    leaves = [t.clone().requires_grad_(True) for t in x]
    (Delta.apply(*leaves) * w).sum().backward()
    for i, leaf in enumerate(leaves):
        way = leaf.grad / leaf.grad.norm()
        step = 1e-2
        vals = []
        for s in (step, -step):
            y = [t.detach() + (s * way if j == i else 0) for j, t in enumerate(x)]
            vals.append((rn.retnet_delta_chunkwise(*y).double() * w.double()).sum().item())
        diff = (vals[0] - vals[1]) / (2 * step)
        want = leaf.grad.norm().item()
        # truncation step^2 = 1e-4 times the third derivative's relative size
        # (a few at most: the loss is a short polynomial in each input), and
        # float32 outputs: 1e-7 * |loss terms| / step
        assert abs(diff - want) < 5e-3 * want, i


def test_two_streams_at_once(rn):
    """A prefill and a backward that run beside each other, several times,
    give what each gives alone."""
    B, n, H, d = 2, 700, 8, 128
    x, _ = make(21, B, n, H, H, d, d, "bf16")
    y, _ = make(22, B, n, H, H, d, d, "bf16")
    S, want_S = torch.empty(B, H, d, d, device="cuda"), torch.empty(B, H, d, d, device="cuda")
    want = rn.retnet_delta_chunkwise(*x[:5], state_out=want_S)
    want_grads = rn.retnet_delta_backward(*y)
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(4):
        with torch.cuda.stream(streams[0]):
            out = rn.retnet_delta_chunkwise(*x[:5], state_out=S)
        with torch.cuda.stream(streams[1]):
            grads = rn.retnet_delta_backward(*y)
    done(rn)
    assert torch.equal(out, want) and torch.equal(S, want_S)
    for a, b in zip(grads, want_grads):
        assert torch.equal(a, b)


def noise(seed, *shape):
    """bf16 of little precision, made without a float32 copy."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(*shape, device="cuda", dtype=torch.bfloat16).uniform_(-0.5, 0.5, generator=gen)


def test_states_and_workspaces_beyond_32_bits(rn):
    """More than 2^31 state elements and workspaces above 2^32 bytes: the last
    sequences as they come out alone."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    B, H, d = 2050, 16, 256
    x = [noise(30 + i, B, 1, H, d) * 0.1 for i in range(3)]
    x += [noise(33, B, 1, H) - 0.5, noise(34, B, 1, H) + 0.5]
    S = torch.empty(B, H, d, d, device="cuda").uniform_(-0.5, 0.5)
    assert S.numel() > 2 ** 31
    mine = S[-1:].clone()
    out = rn.retnet_delta_recurrent(*x, S)
    alone = rn.retnet_delta_recurrent(*(t[-1:].contiguous() for t in x), mine)
    done(rn)
    assert torch.equal(out[-1:], alone) and torch.equal(S[-1:], mine)
    del S

    B, n, d = 128, 2048, 128
    x = [noise(40 + i, B, n, H, d) * 0.1 for i in range(2)] + [noise(42, B, n, H, d)]
    x += [noise(43, B, n, H) - 0.5, noise(44, B, n, H) + 0.5]
    size = rn.retnet_delta_workspace_size(B, H, H, n, d, d, torch.bfloat16)
    assert size > 2 ** 32
    S = torch.empty(B, H, d, d, device="cuda")
    out = rn.retnet_delta_chunkwise(*x, state_out=S)
    few = [t[-16:].contiguous() for t in x]        # as many as walk whole
    mine = torch.empty(16, H, d, d, device="cuda")
    alone = rn.retnet_delta_chunkwise(*few, state_out=mine)
    done(rn)
    assert torch.equal(out[-16:], alone) and torch.equal(S[-16:], mine)
    del out, S
    do = noise(45, B, n, H, d)
    grads = rn.retnet_delta_backward(*x, do)
    alone = rn.retnet_delta_backward(*few, do[-16:].contiguous())
    done(rn)
    for a, b in zip(grads, alone):
        assert torch.isfinite(b).all() and torch.equal(a[-16:], b)


def test_arguments_that_do_not_fit(rn):
    """The bindings name the argument that does not fit the others."""
    (q, k, v, g, beta, do), _ = make(28, 2, 5, 2, 4, 64, 128, "bf16")
    S = torch.zeros(2, 4, 64, 128, device="cuda")
    for kw, kind in ((dict(k=k[:1]), ValueError), (dict(k=k.float()), TypeError),
                     (dict(v=v[:, :4]), ValueError), (dict(g=g.cpu()), ValueError),
                     (dict(beta=beta[:, :, :2]), ValueError), (dict(state=S.double()), TypeError),
                     (dict(state=None), TypeError), (dict(out=v.transpose(1, 2)), ValueError),
                     (dict(lengths=torch.ones(2, device="cuda")), TypeError),
                     (dict(lengths=torch.ones(3, device="cuda", dtype=torch.int32)), ValueError)):
        args = dict(q=q, k=k, v=v, g=g, beta=beta, state=S)
        args.update(kw)
        with pytest.raises(kind):
            rn.retnet_delta_recurrent(**args)
    with pytest.raises(TypeError):
        rn.retnet_delta_backward(q, k, v, g, beta, None)
    for kw in (dict(dq=k.float()), dict(workspace=S)):
        with pytest.raises(TypeError):
            rn.retnet_delta_backward(q, k, v, g, beta, do, **kw)
    # a parameter is a tensor
    p = torch.nn.Parameter(q)
    assert torch.equal(rn.retnet_delta_chunkwise(p, k, v, g, beta),
                       rn.retnet_delta_chunkwise(q, k, v, g, beta))
    done(rn)
