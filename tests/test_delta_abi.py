"""What the gated delta rule's and the residual norm's entry points refuse,
before anything is launched (CPU)."""
import ctypes

import pytest
import torch

import linear_recurrent_sequence_02_b200 as rn
from linear_recurrent_sequence_02_b200.build import build

P = ctypes.c_void_p
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 5


@pytest.fixture(scope="module")
def lib():
    build()
    return rn.load_library()


def shape(B=2, H=4, Hk=2, n=100, dk=64, dv=128, dt=0):
    return rn._DeltaShape(B, H, Hk, n, dk, dv, dt)


BAD_SHAPES = [
    (dict(B=-1), INVALID), (dict(n=-1), INVALID), (dict(H=0), INVALID), (dict(Hk=0), INVALID),
    (dict(H=3), INVALID), (dict(Hk=8), INVALID), (dict(H=257, Hk=257), INVALID),
    (dict(dk=0), INVALID), (dict(dt=2), INVALID), (dict(dk=96), UNSUPPORTED),
    (dict(dv=512), UNSUPPORTED), (dict(B=1 << 30, H=256, Hk=256), UNSUPPORTED),
    (dict(B=0, n=2 ** 31 - 1), UNSUPPORTED),
]


def calls(lib, s, **kw):
    """The three entry points' statuses on pointers that are never followed."""
    a = {"q": 1024, "g": 1024, "beta": 1024, "lengths": None, "scale": 1.0, "state": 1024,
         "out": 1024, "algo": 0, "ws": 1024, "wsb": 1 << 50, "dbeta": 1024}
    a.update(kw)
    s = None if s is None else ctypes.byref(s)
    x = (P(a["q"]), P(1024), P(1024), P(a["g"]), P(a["beta"]))
    return (lib.retnet_delta_recurrent(*x, a["scale"], P(a["lengths"]), P(a["state"]), P(a["out"]),
                                       s, None),
            lib.retnet_delta_chunkwise(*x, a["scale"], P(a["lengths"]), P(a["out"]), s,
                                       P(a["state"]), None, a["algo"], P(a["ws"]), a["wsb"], None),
            lib.retnet_delta_backward(*x, P(a["out"]), a["scale"], P(a["lengths"]), P(1024),
                                      P(1024), P(1024), P(1024), P(a["dbeta"]), s, a["algo"],
                                      P(a["ws"]), a["wsb"], None))


@pytest.mark.parametrize("bad,status", BAD_SHAPES)
def test_shapes(lib, bad, status):
    assert calls(lib, shape(**bad)) == (status,) * 3
    n = ctypes.c_size_t(0)
    for size in (lib.retnet_delta_workspace_size, lib.retnet_delta_backward_workspace_size):
        assert size(ctypes.byref(shape(**bad)), 0, ctypes.byref(n)) == status


@pytest.mark.parametrize("B,H,n,fits", [
    (1 << 23, 1, 1, True), ((1 << 23) + 1, 1, 1, False), (1 << 23, 1, 0, True),
    (1 << 15, 256, 64, True), (1 << 15, 256, 65, False), (1 << 17, 1, 4096, True),
    (1 << 17, 1, 4097, False), (1, 1, 1 << 29, True), (1, 1, (1 << 29) + 1, False),
    (3, 5, 64 * (2 ** 23 // 15), True), (3, 5, 64 * (2 ** 23 // 15) + 1, False),
])
def test_largest_shapes(lib, B, H, n, fits):
    """2^23 chunks of 64 tokens over all sequences and heads, and one more
    (workspace sizes only: nothing is launched)."""
    size = ctypes.c_size_t(0)
    for dk in (64, 256):
        for dtype in (0, 1):
            s = ctypes.byref(shape(B, H, H, n, dk, 256, dtype))
            for f in (lib.retnet_delta_workspace_size, lib.retnet_delta_backward_workspace_size):
                assert f(s, 0, ctypes.byref(size)) == (OK if fits else UNSUPPORTED)


def test_arguments(lib):
    s = shape()
    assert calls(lib, None) == (INVALID,) * 3
    for bad in (dict(q=None), dict(q=1032), dict(g=None), dict(beta=8), dict(lengths=4),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(out=None),
                dict(out=1032)):
        assert calls(lib, s, **bad) == (INVALID,) * 3, bad
    assert calls(lib, s, state=1032)[:2] == (INVALID,) * 2
    assert calls(lib, s, state=None)[0] == INVALID            # the prefill's may be missing
    assert calls(lib, s, dbeta=None)[2] == INVALID
    assert calls(lib, s, algo=3)[1:] == (INVALID,) * 2
    assert calls(lib, s, algo=2)[1:] == (UNSUPPORTED,) * 2    # float32 has no tensor-core path
    assert calls(lib, s, ws=None)[2] == WORKSPACE
    assert calls(lib, s, wsb=64)[2] == WORKSPACE
    assert calls(lib, s, ws=1024 + 256)[2] == WORKSPACE


def test_nothing_to_do(lib):
    none = dict(q=None, g=None, beta=None, out=None, ws=None, wsb=0, dbeta=None)
    assert calls(lib, shape(B=0), state=None, **none) == (OK,) * 3
    assert calls(lib, shape(n=0), state=None, **none) == (OK,) * 3


def norm(lib, rows=4, hidden=64, dtype=0, **kw):
    a = {"x": 1024, "h": 1024, "gate": 1024, "post_norm": 1, "post": 1024, "scale": 1.0,
         "eps": 1e-5, "dgate": 1024, "dpost": 1024, "dh": 1024, "ws": 1024, "wsb": 1 << 40}
    a.update(kw)
    p = rn._BlockNorm(a["gate"], a["post_norm"], a["post"], 1024, a["scale"], a["eps"])
    return (lib.retnet_residual_norm(P(a["x"]), P(1024), ctypes.byref(p), rows, hidden, dtype,
                                     P(a["h"]), P(1024), None),
            lib.retnet_residual_norm_backward(P(a["x"]), P(1024), P(1024), P(a["dh"]),
                                              ctypes.byref(p), rows, hidden, dtype, P(a["h"]),
                                              P(1024), P(a["dgate"]), P(a["dpost"]), P(1024),
                                              P(a["ws"]), a["wsb"], None))


def test_residual_norm_arguments(lib):
    for bad in (dict(rows=-1), dict(rows=1 << 31), dict(hidden=0), dict(hidden=60),
                dict(hidden=16392), dict(dtype=5), dict(x=None), dict(x=8), dict(h=None),
                dict(h=1028), dict(gate=1028), dict(post_norm=2), dict(post=1028),
                dict(eps=-1.0), dict(eps=float("nan")), dict(scale=float("inf"))):
        assert norm(lib, **bad) == (INVALID,) * 2, bad
    for bad in (dict(dgate=None), dict(gate=None), dict(dpost=1028), dict(dh=1028),
                dict(post_norm=0)):
        assert norm(lib, **bad)[1] == INVALID, bad
    for bad in (dict(ws=None), dict(wsb=16), dict(ws=1024 + 64)):
        assert norm(lib, **bad)[1] == WORKSPACE, bad
    assert norm(lib, rows=0, x=None, h=None)[0] == OK
    assert lib.retnet_residual_norm(P(1024), P(1024), None, 4, 64, 0, P(1024), P(1024), None) == INVALID


def test_bindings_refuse_what_does_not_fit(lib):
    """Host tensors, types and shapes stop in the binding."""
    x = torch.zeros(1, 4, 2, 64)
    g = torch.zeros(1, 4, 2)
    S = torch.zeros(1, 2, 64, 64)
    for call in (lambda: rn.retnet_delta_recurrent(x, x, x, g, g, S),
                 lambda: rn.retnet_delta_chunkwise(x, x, x, g, g),
                 lambda: rn.retnet_delta_backward(x, x, x, g, g, x),
                 lambda: rn.retnet_residual_norm(x, x),
                 lambda: rn.retnet_residual_norm_backward(x, x, x)):
        with pytest.raises(ValueError):
            call()
