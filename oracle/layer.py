"""A target layer around its attention, in plain NumPy and 64 bits: the product with its epilogue, norms and rotation of
queries and keys, log probabilities.  Written from the formulas, row by row where that is clearest."""
import math

import numpy as np


def activation(z, name):
    z = np.asarray(z, np.float64)
    if name == "relu":
        return np.where(z < 0, 0.0, z)
    if name == "silu":
        with np.errstate(over="ignore", invalid="ignore"):
            return z / (1 + np.exp(-z))
    if name == "gelu":
        return z * 0.5 * np.vectorize(lambda t: math.erfc(-t / math.sqrt(2)), otypes=[np.float64])(z)
    if name == "gelu_tanh":
        return 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def linear(x, weight, bias=None, gate=None, gate_bias=None, act=None, residual=None):
    y = x @ weight.T + (0 if bias is None else bias)
    if gate is None:
        y = activation(y, act)
    else:
        y = activation(x @ gate.T + (0 if gate_bias is None else gate_bias), act) * y
    return y if residual is None else y + residual


def qk_norm_rope(x, position, rot, inv_freq, interleaved, weight, eps, amplitude=1.0):
    """One tensor: x [rows, heads, head_dim], position [rows] (Python or NumPy integers of any size)."""
    y = np.array(x, np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * weight
    for t, pos in enumerate(position):
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            # (whole turns are taken off in integers: a product of 53 bits would lose far positions)
            angle = turn_angle(int(pos), inv_freq[i])
            c, s = amplitude * math.cos(angle), amplitude * math.sin(angle)
            u, v = y[t, :, a].copy(), y[t, :, b].copy()
            y[t, :, a], y[t, :, b] = u * c - v * s, v * c + u * s
    return y


def turn_angle(pos, freq):
    """pos * freq modulo 2 pi, by rational arithmetic (pi to 40 digits)."""
    from fractions import Fraction
    two_pi = 2 * Fraction(3141592653589793238462643383279502884197, 10 ** 39)
    return float(Fraction(freq) * pos % two_pi)


def token_logprobs(row, tokens, top, temperature):
    """One row: (logp of tokens, lse, entropy, top ids, their logp)."""
    row = np.asarray(row, np.float64)
    if np.isnan(row).any() or np.isposinf(row).any():
        return np.where(np.asarray(tokens) < 0, 0.0, math.nan), math.nan, math.nan, np.full(top, -1), np.full(top, math.nan)
    z = row / temperature
    m = z.max()
    order = sorted(range(len(row)), key=lambda v: (-row[v], v))[:top] if top else []
    if m == -math.inf:
        return np.array([0.0 if t < 0 else math.nan if t >= len(row) else -math.inf for t in tokens]), -math.inf, 0.0, np.array(order), np.full(top, -math.inf)
    d = z - m  # (differences to the maximum: beside fp32's lowest value, as masks use it, a logarithm would be lost)
    log_sum = math.log(np.exp(d).sum())
    p = np.exp(d - log_sum)
    entropy = log_sum - float(np.where(p > 0, p * np.where(p > 0, d, 0), 0).sum())
    logp = np.array([0.0 if t < 0 else math.nan if t >= len(row) else d[t] - log_sum for t in tokens])
    return logp, m + log_sum, entropy, np.array(order), np.array([d[v] - log_sum for v in order])
