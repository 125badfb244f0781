"""Softmax decode over token ranges, float64: a sliding window with sinks, and a
sequence whose first tokens are a shared prefix.

    o = sum_i softmax(scale q.k_i)_i v_i,   lse = log sum_i exp(scale q.k_i)

over the tokens a sequence attends to; a row without tokens gives o = 0 and
lse = -inf.  Alongside each result stands how far an implementation with a
stated arithmetic may be from it.
"""
import numpy as np


def window_tokens(L, window, sinks):
    """Positions a sequence of L tokens attends to: t < sinks or t >= L - window."""
    t = np.arange(max(L, 0))
    return t[(t < sinks) | (t >= L - window)]


def softmax_rows(q, keys, vals, scale):
    """q [G, d], keys and vals [n, d]: (o [G, d], lse [G]) in float64."""
    q, keys, vals = (np.asarray(x, dtype=np.float64) for x in (q, keys, vals))
    if len(keys) == 0:
        return np.zeros((q.shape[0], vals.shape[1])), np.full(q.shape[0], -np.inf)
    x = scale * (q @ keys.T)
    m = x.max(axis=1, keepdims=True)
    e = np.exp(x - m)
    z = e.sum(axis=1, keepdims=True)
    return (e / z) @ vals, (m + np.log(z))[:, 0]


def error_bound(q, keys, vals, scale, split):
    """(bound on |o - o_ref| [G, d], bound on |lse - lse_ref| [G]) for fp32 sums.

    split: the query and the weights enter their products as a bf16 high and low
    part (at least).  Of a value in [1, 2) the high part leaves a rest of at most
    half a step, 2^-8, and a step of a rest below 2^-8 is at most 2^-16: hi + lo
    is the value to 2^-17.  Otherwise they enter as fp32 (2^-24).  With
    A = scale sum_d |q_d k_d|:
      dx  = A (r + d 2^-23) + 2^-22 (|x| + max |x|)
            the query's rounding r, the fp32 sum over d (one step of 2^-23 a
            term, whether it rounds or truncates), and x log2(e) - m rounded
            with x and m of that size;
      each weight: relative 2 dx + 2^-21 (exp2 to two steps, rescalings) + r;
      the sums over n tokens: n 2^-23 of the sum of magnitudes.
    """
    q, keys, vals = (np.asarray(x, dtype=np.float64) for x in (q, keys, vals))
    n, d = keys.shape
    if n == 0:
        return np.zeros((q.shape[0], vals.shape[1])), np.zeros(q.shape[0])
    r = 2.0 ** -17 if split else 2.0 ** -24
    x = scale * (q @ keys.T)
    A = scale * (np.abs(q) @ np.abs(keys).T)
    dx = A * (r + d * 2.0 ** -23) + 2.0 ** -22 * (np.abs(x) + np.abs(x).max(axis=1, keepdims=True))
    p = np.exp(x - x.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    rel = np.expm1(2 * dx) + 2.0 ** -21 + r + n * 2.0 ** -23
    # the weights' errors and the normaliser's (the mean of the weights' errors)
    mean_rel = (p * rel).sum(axis=1, keepdims=True)
    o = (p * rel) @ np.abs(vals) + mean_rel * (p @ np.abs(vals))
    lse = mean_rel[:, 0] + 2.0 ** -22 * (np.abs(x).max(axis=1) + np.log(n) + 1)
    return o, lse
