"""Gated feed-forward operators in float64 (TEST INFRASTRUCTURE ONLY -- never imported by the product path).

Definitions (include/fp8q_ffn.h):
    * activations: SiLU g / (1 + e^-g), and GELU by its tanh form 0.5 g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3)));
    * gated product h = act(g) * u, and its gradient dg = dh * u * act'(g), du = dh * act(g);
    * 8-bit codes of a row: a = max(max|x|, 127 * 2^-126), s = fl32(a * fl32(1/127)), inv = fl32(127 * fl32(1/a)),
      q = round-half-even(fl32(x * inv));
    * integer product: a_scales[m] * b_scales[n] * sum_k A[m][k] B[n][k] (+ bias[n]).
"""

import numpy as np

SILU, GELU_TANH = 0, 1

_R = np.sqrt(2.0 / np.pi)
#: Floor on a row's max-abs: 127 * 2^-126.
INT8_FLOOR = np.float32(127.0 * 2.0 ** -126)


def _logistic(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def _gelu_arg(g):
    """0.5 (1 + tanh z) is the logistic function of 2 z, which keeps its digits where 1 + tanh z cancels."""
    return 2.0 * _R * (g + 0.044715 * g ** 3)


def act(g, kind):
    """act(g) in float64."""
    g = np.asarray(g, np.float64)
    if kind == SILU:
        return g * _logistic(g)
    return g * _logistic(_gelu_arg(g))


def act_slope(g, kind):
    """act'(g) in float64."""
    g = np.asarray(g, np.float64)
    if kind == SILU:
        s = _logistic(g)
        return s + g * s * _logistic(-g)
    s = _logistic(_gelu_arg(g))
    return s + g * s * _logistic(-_gelu_arg(g)) * 2.0 * _R * (1.0 + 3 * 0.044715 * g * g)


def gated(g, u, kind):
    return act(g, kind) * np.asarray(u, np.float64)


def gated_backward(dh, g, u, kind):
    """(dg, du) in float64."""
    dh = np.asarray(dh, np.float64)
    return dh * np.asarray(u, np.float64) * act_slope(g, kind), dh * act(g, kind)


def quant_int8_rows(x):
    """int8 codes [rows][cols] and float32 scales [rows] of a float32 array."""
    x = np.asarray(x, np.float32)
    amax = np.abs(x).max(axis=1) if x.shape[1] else np.zeros(x.shape[0], np.float32)
    a = np.maximum(amax, INT8_FLOOR).astype(np.float32)
    one = np.float32(1.0)
    s = (a * (one / np.float32(127.0))).astype(np.float32)
    inv = ((one / a).astype(np.float32) * np.float32(127.0)).astype(np.float32)
    q = np.rint((x * inv[:, None]).astype(np.float32))      # rint: half to even
    return q.astype(np.int8), s


def int8_gemm_ref(qa, sa, qb, sb, bias=None):
    """Exact integer sum, scaled in float64.  The sum goes through a float64 product, exact below 2^53."""
    y = np.asarray(qa, np.float64) @ np.asarray(qb, np.float64).T
    y = y * np.asarray(sa, np.float64)[:, None] * np.asarray(sb, np.float64)[None, :]
    return y if bias is None else y + np.asarray(bias, np.float64)[None, :]
