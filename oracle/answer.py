"""Plain numpy definitions (f64) of what ends a decode layer and a decode step:
Q1_0 . q8_0 products with an epilogue, the norms behind and before a block, log
probabilities. Test infrastructure; no code shared with the library."""
from __future__ import annotations

import numpy as np
from scipy.special import erfc

ACTS = ("none", "relu", "relu2", "gelu", "gelu_tanh", "silu")   # by the header's GD_ACT_ codes


def q1_values(w_aos):
    """f64 [rows, K] of Q1_0 blocks (uint8 [rows, K/128, 18])."""
    w = np.ascontiguousarray(w_aos)
    d = w[:, :, :2].copy().view(np.float16).astype(np.float64)
    s = np.unpackbits(w[:, :, 2:], axis=2, bitorder="little").astype(np.float64) * 2 - 1
    return (s * d).reshape(w.shape[0], -1)


def q8_values(a_aos, n: int):
    """f64 [n, K] of q8_0 blocks (uint8, 34 to a block)."""
    b = np.ascontiguousarray(a_aos).reshape(n, -1, 34)
    d = b[:, :, :2].copy().view(np.float16).astype(np.float64)
    return (b[:, :, 2:].copy().view(np.int8) * d).reshape(n, -1)


def act(t, code: int):
    t = np.asarray(t, np.float64)
    with np.errstate(over="ignore"):
        return {"none": lambda: t, "relu": lambda: np.maximum(t, 0), "relu2": lambda: np.maximum(t, 0) ** 2,
                "gelu": lambda: 0.5 * t * erfc(-t / np.sqrt(2)),
                "gelu_tanh": lambda: t / (1 + np.exp(-2 * np.sqrt(2 / np.pi) * (t + 0.044715 * t ** 3))),
                "silu": lambda: t / (1 + np.exp(-t))}[ACTS[code]]()


def act_slope(t, reach, code: int):
    """A bound on the activation's slope within `reach` of t."""
    if ACTS[code] == "relu2":
        return 2 * (np.abs(t) + reach)
    return 1.13   # the largest slopes are 1, 1, 1.129 (both GELUs) and 1.0998 (SiLU)


def product(w, a, bias, code: int):
    """(act(W a + bias) f64 [n, rows], how far f32 sums may be off it): w [rows, K] and a [n, K] f64."""
    t, size = a @ w.T, np.abs(a) @ np.abs(w).T
    off = (w.shape[1] / 128 + 9) * 2.0 ** -23 * size
    if bias is not None:
        t = t + bias
        off = off + 2.0 ** -24 * np.abs(t)
    v = act(t, code)
    # the activation's own error, taken where the f32 sum may lie
    own = 2.0 ** -23 * np.abs(v) if code in (0, 1, 2) else 2.0 ** -20 * (np.abs(t) + off)
    return v, act_slope(t, off, code) * off + own


def logprobs(x, tokens, k: int, scale: float = 1.0, cap: float = 0.0):
    """Of one row of logits (f32 values [V]): (log probabilities of `tokens`, entropy, ids and log probabilities of the k
    largest)."""
    x = np.asarray(x, np.float64)
    scale, cap = float(np.float32(scale)), float(np.float32(cap))
    if np.isnan(x).any() or (x == np.inf).any():
        return np.where((tokens >= 0) & (tokens < len(x)), np.nan, 0.0), np.nan, np.full(k, -1), np.full(k, np.nan)
    banned = x == -np.inf
    with np.errstate(invalid="ignore", divide="ignore"):
        z = scale * (cap * np.tanh(x / cap) if cap else x)
        z[banned] = -np.inf
        if banned.all():
            lp, entropy = np.full(len(x), -np.inf), 0.0
        else:
            top = int(np.argmax(z))
            d = z - z[top]
            e = np.exp(d)
            e[top] = 0
            s = e.sum()
            lp = d - np.log1p(s)
            entropy = np.log1p(s) - np.sum(np.where(e > 0, e * d, 0.0)) / (1 + s)
    order = np.argsort(-x, kind="stable")[:k]
    left = ~banned[order]
    ids = np.concatenate([np.where(left, order, -1), np.full(k - len(order), -1)])
    tops = np.concatenate([lp[order], np.full(k - len(order), -np.inf)])
    inside = (tokens >= 0) & (tokens < len(x))
    return np.where(inside, lp[np.clip(tokens, 0, len(x) - 1)], 0.0), entropy, ids, tops
