"""The layer's oracle against other statements of the same definitions (CPU)."""
import math

import numpy as np
import pytest

from oracle import layer as ol


def test_activations_at_known_points():
    assert ol.activation([-2.0, 0.0, 3.0], "relu").tolist() == [0, 0, 3]
    assert ol.activation(0.0, "silu") == 0 and abs(ol.activation(1.0, "silu") - 1 / (1 + math.exp(-1))) < 1e-15
    assert abs(ol.activation([1.0], "gelu")[0] - 0.8413447460685429) < 1e-15
    assert abs(ol.activation([-8.0], "gelu")[0] + 8 * 6.220960574271785e-16) < 1e-27
    assert abs(ol.activation([1.0], "gelu_tanh")[0] - 0.8411919906082768) < 1e-12
    assert ol.activation([5.0], None).tolist() == [5]


def test_linear_by_single_products():
    rs = np.random.RandomState(0)
    x, w, g, b, gb, res = (rs.standard_normal(s) for s in ((2, 3), (4, 3), (4, 3), 4, 4, (2, 4)))
    y = ol.linear(x, w, b, g, gb, "silu", res)
    for t in range(2):
        for n in range(4):
            z = sum(x[t, k] * g[n, k] for k in range(3)) + gb[n]
            want = z / (1 + math.exp(-z)) * (sum(x[t, k] * w[n, k] for k in range(3)) + b[n]) + res[t, n]
            assert abs(y[t, n] - want) < 1e-14


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_one_of_complex_numbers_and_keeps_relative_positions(interleaved):
    rs = np.random.RandomState(1)
    freq = [0.7, 0.01]
    x = rs.standard_normal((1, 1, 6))
    y = ol.qk_norm_rope(x, [5], 4, freq, interleaved, None, 0)
    pairs = [(0, 1), (2, 3)] if interleaved else [(0, 2), (1, 3)]
    for (a, b), f in zip(pairs, freq):
        z = complex(x[0, 0, a], x[0, 0, b]) * complex(math.cos(5 * f), math.sin(5 * f))
        assert abs(complex(y[0, 0, a], y[0, 0, b]) - z) < 1e-14
    assert (y[..., 4:] == x[..., 4:]).all()
    q, k = rs.standard_normal((2, 1, 1, 4))
    far = 10 ** 6
    dots = [(ol.qk_norm_rope(q, [p + 9], 4, freq, interleaved, None, 0) * ol.qk_norm_rope(k, [p], 4, freq, interleaved, None, 0)).sum() for p in (0, far)]
    assert abs(dots[0] - dots[1]) < 1e-12


def test_norm():
    x = np.arange(1.0, 9).reshape(1, 1, 8)
    y = ol.qk_norm_rope(x, [0], 0, [], False, np.full(8, 2.0), 0.5)
    assert np.allclose(y, 2 * x / math.sqrt(204 / 8 + 0.5), rtol=1e-15)


def test_log_probabilities():
    row = np.log(np.array([0.1, 0.2, 0.3, 0.4])) + 3
    logp, lse, h, ids, best = ol.token_logprobs(row, [2, -1, 4], 2, 1.0)
    assert abs(logp[0] - math.log(0.3)) < 1e-14 and logp[1] == 0 and math.isnan(logp[2]) and abs(lse - 3) < 1e-14
    assert abs(h + sum(p * math.log(p) for p in (0.1, 0.2, 0.3, 0.4))) < 1e-14
    assert ids.tolist() == [3, 2] and abs(best[0] - math.log(0.4)) < 1e-14
    assert ol.token_logprobs([1.0, 5.0, 5.0], [], 3, 1.0)[3].tolist() == [1, 2, 0]
    inf = math.inf
    logp, lse, h, ids, best = ol.token_logprobs([-inf, -inf], [0], 2, 1.0)
    assert (logp[0], lse, h, ids.tolist()) == (-inf, -inf, 0, [0, 1])
    assert ol.token_logprobs([-inf, 2.0], [0, 1], 2, 0.5)[0].tolist() == [-inf, 0]
    assert math.isnan(ol.token_logprobs([1.0, inf], [0], 1, 1.0)[1])
