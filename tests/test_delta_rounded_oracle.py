"""The chunk form of the gated delta rule in the oracle, with and without the
tensor-core path's roundings, against the token-by-token definition (CPU)."""
import numpy as np
import pytest
import torch

import oracle
from oracle.delta_chunks import BACKWARD, FORWARD, bf16


def make(seed, B, n, Hk, H, dk, dv, decay):
    rng = np.random.default_rng(seed)
    q, k = rng.standard_normal((2, B, n, Hk, dk))
    q /= np.linalg.norm(q, axis=-1, keepdims=True)
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    v, do = rng.standard_normal((2, B, n, H, dv))
    g = -decay * np.exp(0.7 * rng.standard_normal((B, n, H)))
    beta = 1.0 / (1.0 + np.exp(-rng.standard_normal((B, n, H))))
    return [bf16(x) for x in (q, k, v, g, beta, do)]


def norm_err(got, want):
    return np.linalg.norm(got - want) / np.linalg.norm(want)


def test_bf16_rounds_to_nearest_even():
    x = np.random.default_rng(0).standard_normal(4000).astype(np.float32).astype(np.float64)
    x = np.concatenate([x, [1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, 0.0, -0.0]])
    assert np.array_equal(bf16(x), torch.from_numpy(x).bfloat16().double().numpy())


@pytest.mark.parametrize("lens", [None, [0, 150, 65], [1, 64, 63]])
def test_without_roundings_it_is_the_definition(lens):
    """Float64 both: 2^-53 a step and a few hundred of them."""
    B, n, Hk, H, dk, dv = 3, 150, 1, 2, 16, 24
    x = make(1, B, n, Hk, H, dk, dv, 0.1)
    x[3][:, 20], x[4][:, 30], x[4][:, 31] = -np.inf, 0.0, 1.0
    S0 = np.random.default_rng(2).standard_normal((B, H, dk, dv))
    for a, b in zip(oracle.delta_chunks(*x[:5], 0.3, S0, lens, rounds=()),
                    oracle.delta_recurrent(*x[:5], 0.3, S0, lens)):
        assert norm_err(a, b) < 1e-12
    for a, b in zip(oracle.delta_chunks_backward(*x, 0.3, lens, rounds=()),
                    oracle.delta_backward(*x, 0.3, lens)):
        assert norm_err(a, b) < 1e-12


@pytest.mark.parametrize("decay", [0.2, 0.02])
def test_each_rounding_moves_the_outputs_by_no_more_than_its_own_size(decay):
    """A rounding is at most 2^-8 of a value, and, where the values spread over
    the binades as these do, 1.7e-3 of a norm (2^-8 / sqrt(3) at a binade's
    lower end, half of it at the upper).  Each operand's rounding reaches an
    output through sums that do not grow: at most 2^-8 of its norm.  All of
    them are independent."""
    x = make(3, 1, 300, 1, 2, 64, 64, decay)
    scale = 0.125
    cases = [(oracle.delta_recurrent(*x[:5], scale)[:1], FORWARD,
              lambda r: oracle.delta_chunks(*x[:5], scale, rounds=r)[:1]),
             (oracle.delta_backward(*x, scale), BACKWARD,
              lambda r: oracle.delta_chunks_backward(*x, scale, rounds=r))]
    for want, names, run in cases:
        shares = [[norm_err(a, w) for a, w in zip(run((name,)), want)] for name in names]
        assert np.max(shares) < 2.0 ** -8
        total = [norm_err(a, w) for a, w in zip(run(names), want)]
        assert np.all(np.array(total) < 1.3 * np.sqrt(np.square(shares).sum(0)))


def test_two_parts_keep_the_state():
    x = make(4, 1, 400, 1, 1, 64, 64, 0.02)
    want = oracle.delta_recurrent(*x[:5], 0.125)
    one = oracle.delta_chunks(*x[:5], 0.125)
    two = oracle.delta_chunks(*x[:5], 0.125, final_state=True)
    assert norm_err(two[1], want[1]) < 6 * 2.0 ** -18 < 1e-4 < norm_err(one[1], want[1])
