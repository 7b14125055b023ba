"""The gated delta rule as its documentation allows it, where
test_delta_gpu.py does not go."""
import pytest
import torch

import oracle
from test_delta_gpu import bound, done, err, make, rn, states  # noqa: F401

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
