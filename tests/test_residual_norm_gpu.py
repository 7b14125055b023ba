"""GPU parity of the fused residual norm and its gradients against the
float64 oracle.

Error measure: 2-norm relative error of each output.  Float32 math has 2^-24
a step and sums of up to 16384 terms in trees of depth 14 (fewer than 60
roundings in a row, and two fast functions of 2^-21): bound 2e-6 for
float32.  bf16 adds one rounding of the result, at most 2^-8 of each value.
Weight gradients are float32 in both."""
import numpy as np
import pytest
import torch

import oracle
from helpers import record

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
BOUND = {"f32": 2e-6, "bf16": 2.0 ** -8 + 2e-6}


@pytest.fixture(scope="module")
def rn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import linear_recurrent_sequence_02_b200 as lib
    from linear_recurrent_sequence_02_b200.build import build
    build()
    lib.load_library()
    return lib


def err(got, want):
    got = got.double().cpu().numpy()
    assert got.shape == want.shape
    if not want.size:
        return 0.0
    return record(float(np.linalg.norm(got - want) / np.linalg.norm(want)), "2-norm")


def make(seed, rows, hidden, dtype):
    rng = np.random.default_rng(seed)
    scale = np.array([2.0, 0.5, 1.0, 1.0, 1.0])[:, None, None]
    gpu = [torch.from_numpy(x).to(DT[dtype]).cuda()
           for x in scale * rng.standard_normal((5, rows, hidden))]
    w = [torch.from_numpy(1 + 0.2 * rng.standard_normal(hidden)).float().cuda() for _ in range(2)]
    return gpu, [t.double().cpu().numpy() for t in gpu], w, [t.double().cpu().numpy() for t in w]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,hidden", [(1, 8), (5, 264), (3, 512), (7, 520), (2, 2056),
                                         (3, 4104), (2, 8200), (1, 16384), (1300, 64)])
@pytest.mark.parametrize("gated,post_norm,weighted", [(True, True, True), (False, True, False),
                                                      (True, False, True)])
def test_forward_and_backward(rn, dtype, rows, hidden, gated, post_norm, weighted):
    (x, y, gate, dn, dh), ref, (post, pre), wref = make(rows + hidden, rows, hidden, dtype)
    kw = dict(post_norm=post_norm, eps=1e-5)
    gpu = dict(gate=gate if gated else None, post_weight=post if weighted and post_norm else None,
               pre_weight=pre if weighted else None, residual_scale=0.7, **kw)
    cpu = dict(gate=ref[2] if gated else None, post=wref[0] if weighted and post_norm else None,
               pre=wref[1] if weighted else None, scale=0.7, **kw)
    h, n = rn.retnet_residual_norm(x, y, **gpu)
    got = rn.retnet_residual_norm_backward(x, y, dn, dh if weighted else None, **gpu)
    torch.cuda.synchronize()
    rn.retnet_check_device_errors()
    h_ref, n_ref = oracle.residual_norm(ref[0], ref[1], **cpu)
    assert err(h, h_ref) < BOUND[dtype] and err(n, n_ref) < BOUND[dtype]
    want = oracle.residual_norm_backward(ref[0], ref[1], ref[3], ref[4] if weighted else None,
                                         **cpu)
    for name, a, w in zip(got._fields, got, want):
        if a is None:
            continue
        assert err(a, w) < (BOUND["f32"] if "weight" in name else BOUND[dtype]), name
    assert (got.dgate is None) == (not gated)
    assert (got.dpre_weight is None) == (not weighted)
    assert (got.dpost_weight is None) == (not (weighted and post_norm))


def test_in_place_and_leading_axes(rn):
    (x, y, gate, dn, dh), _, (post, pre), _ = make(3, 12, 136, "bf16")
    x, y, gate, dn, dh = (t.view(3, 4, 136) for t in (x, y, gate, dn, dh))
    kw = dict(gate=gate, post_weight=post, pre_weight=pre)
    h, n = rn.retnet_residual_norm(x, y, **kw)
    grads = rn.retnet_residual_norm_backward(x, y, dn, dh, **kw)
    again = rn.retnet_residual_norm_backward(x, y, dn, dh, dx=dh, dy=dn, **kw)
    assert again.dx is dh and again.dy is dn
    for a, b in zip(grads, again):
        assert torch.equal(a, b)
    rn.retnet_residual_norm(x, y, h=x, n=y, **kw)
    assert torch.equal(x, h) and torch.equal(y, n)


def test_rows_do_not_mix(rn):
    """A row of NaN, one of infinities and one of zeros stay by themselves."""
    (x, y, gate, dn, dh), _, (post, pre), _ = make(4, 6, 96, "f32")
    clean = rn.retnet_residual_norm(x, y, gate=gate, post_weight=post, pre_weight=pre)
    keep = [t.clone() for t in clean]
    x[1], y[2], y[3], x[3] = float("nan"), float("inf"), 0.0, 0.0
    h, n = rn.retnet_residual_norm(x, y, gate=gate, post_weight=post, pre_weight=pre)
    for a, b in zip((h, n), keep):
        assert torch.equal(a[[0, 4, 5]], b[[0, 4, 5]])
        assert not a[3].any()
    assert torch.isnan(n[1]).all()


def test_no_rows(rn):
    x = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    h, n = rn.retnet_residual_norm(x, x)
    assert h.shape == (0, 64)
    g = rn.retnet_residual_norm_backward(x, x, x, post_weight=w, pre_weight=w)
    assert not g.dpost_weight.any() and not g.dpre_weight.any()


def test_captured_graph(rn):
    (x, y, gate, dn, dh), _, (post, pre), _ = make(5, 40, 1032, "bf16")
    kw = dict(gate=gate, post_weight=post, pre_weight=pre)
    ws = rn.retnet_workspace(rn.retnet_residual_norm_backward_workspace_size(40, 1032), "cuda")
    rn.retnet_residual_norm_backward(x, y, dn, dh, workspace=ws, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = rn.retnet_residual_norm(x, y, **kw)
        grads = rn.retnet_residual_norm_backward(x, y, dn, dh, workspace=ws, **kw)
    x.add_(1.0)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip((*out, *grads), (*rn.retnet_residual_norm(x, y, **kw),
                                     *rn.retnet_residual_norm_backward(x, y, dn, dh, **kw))):
        assert torch.equal(a, b)


def test_offsets_beyond_32_bits(rn):
    """More than 2^31 elements a tensor: the last rows as they come out alone."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    rows, hidden = (1 << 31) // 8192 + 3, 8192
    gen = torch.Generator(device="cuda").manual_seed(6)
    x, y, dn = (torch.empty(rows, hidden, device="cuda", dtype=torch.bfloat16).uniform_(
        -1, 1, generator=gen) for _ in range(3))
    assert x.numel() > 2 ** 31
    last = [t[-3:].clone() for t in (x, y, dn)]
    grads = rn.retnet_residual_norm_backward(x, y, dn, dy=dn)
    for a, b in zip(grads[:2], rn.retnet_residual_norm_backward(*last)[:2]):
        assert torch.equal(a[-3:], b)
    del grads, dn
    out = rn.retnet_residual_norm(x, y, h=x, n=y)
    for a, b in zip(out, rn.retnet_residual_norm(*last[:2])):
        assert torch.equal(a[-3:], b)
    torch.cuda.synchronize()
    rn.retnet_check_device_errors()
