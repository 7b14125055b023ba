"""The residual norm over more rows than the GPU holds CTAs, so that every
CTA (every warp, for short rows) of the backward walks several: its copies of
the next row, the sums that two rows share and the weights' gradients in its
registers, against the float64 oracle.

Bounds as in test_residual_norm_gpu.py, here for every row by itself.  A
weight's gradient is a sum over up to 5000 rows: at most 3 of them in a
register, 74 partial rows in a lane and 32 lanes, 109 roundings behind one
another, each at most 2^-24 of a partial sum that is no larger, in the norm
over the channels, than the whole.  They are independent:
sqrt(109 / 3) 2^-24 = 3.6e-7.  The terms' own errors, as the outputs' at most
60 * 2^-24 / sqrt(3) + 2 * 2^-21 where they add and less where their signs
differ from row to row, leave this inside the outputs' bound."""
import numpy as np
import pytest
import torch

import oracle
from helpers import record
from test_residual_norm_gpu import BOUND, make, rn  # noqa: F401

pytestmark = pytest.mark.gpu

# CTAs that the backward launches at most, 148 an SM count: 296 of 8 rows of
# 256 channels (two CTAs an SM), 592 .. 148 of one longer row
ROWS = [(5000, 64), (4801, 256), (3000, 264), (1500, 520), (1301, 1032), (700, 2056), (400, 4104),
        (310, 8200)]


def worst_row(got, want):
    got = got.double().cpu().numpy()
    assert got.shape == want.shape and np.isfinite(got).all()
    got, want = (np.atleast_2d(a) for a in (got, want))
    return record(float((np.linalg.norm(got - want, axis=1) / np.linalg.norm(want, axis=1)).max()),
                  "2-norm of a row")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,hidden", ROWS)
@pytest.mark.parametrize("gated,post_norm", [(True, True), (False, True), (True, False),
                                             (False, False)])
def test_many_rows(rn, dtype, rows, hidden, gated, post_norm):
    (x, y, gate, dn, dh), ref, (post, pre), wref = make(rows + hidden, rows, hidden, dtype)
    kw = dict(post_norm=post_norm, eps=1e-5)
    gpu = dict(gate=gate if gated else None, post_weight=post if post_norm else None,
               pre_weight=pre, residual_scale=0.7, **kw)
    cpu = dict(gate=ref[2] if gated else None, post=wref[0] if post_norm else None, pre=wref[1],
               scale=0.7, **kw)
    h, n = rn.retnet_residual_norm(x, y, **gpu)
    got = rn.retnet_residual_norm_backward(x, y, dn, dh, **gpu)
    # in place, which also shows that the sums' order does not change
    again = rn.retnet_residual_norm_backward(x, y, dn.clone(), dh.clone(), **gpu)
    dn2, dh2 = dn.clone(), dh.clone()
    in_place = rn.retnet_residual_norm_backward(x, y, dn2, dh2, dx=dh2, dy=dn2, **gpu)
    torch.cuda.synchronize()
    rn.retnet_check_device_errors()
    for a, b in zip((h, n), oracle.residual_norm(ref[0], ref[1], **cpu)):
        assert worst_row(a, b) < BOUND[dtype]
    want = oracle.residual_norm_backward(ref[0], ref[1], ref[3], ref[4], **cpu)
    for name, a, b, c, w in zip(got._fields, got, again, in_place, want):
        if a is None:
            assert name == "dgate" and not gated or name == "dpost_weight" and not post_norm
            continue
        assert torch.equal(a, b) and torch.equal(a, c), name
        assert worst_row(a, w) < (BOUND["f32"] if "weight" in name else BOUND[dtype]), name
