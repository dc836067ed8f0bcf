"""Plain numpy definitions (f64) of the steps around a decode layer's products:
the norm with an 8-bit output, rotary positions, the 8-bit cache's rows and
attention over them. Test infrastructure; no code shared with the library."""
from __future__ import annotations

import numpy as np


def math_round_codes(v):
    """Nearest whole number, halves towards +infinity, within [-127, 127]."""
    f = np.floor(v)
    return np.clip(f + (v - f >= 0.5), -127, 127)


def factor(a):
    """127 * (1 / a), each step rounded in f64; 0 for a = 0."""
    return 127.0 * np.divide(1.0, a, out=np.zeros_like(a), where=a > 0)


def rmsnorm_codes(h, weight, eps: float, group: int):
    """Codes int8 [n, K] and f32 scales [n, K/group] of the RMS norm of h
    (f32 [n, K]) times weight, one scale per `group` elements."""
    h = np.asarray(h, np.float32).astype(np.float64)
    n, K = h.shape
    rstd = 1.0 / np.sqrt(np.sum(h * h, axis=1) / K + float(np.float32(eps)))
    p = (h * np.asarray(weight, np.float32).astype(np.float64)).reshape(n, K // group, group)
    a = np.max(np.abs(p), axis=2)
    inv = factor(a)
    codes = math_round_codes(p * inv[:, :, None]).astype(np.int8).reshape(n, K)
    return codes, (a * rstd[:, None] / 127.0).astype(np.float32)


def q8_rows(x):
    """Codes int8 and f16 scales of f32 rows [..., D], 32 dims to a scale."""
    x = np.asarray(x, np.float32)
    p = x.astype(np.float64).reshape(-1, 32)
    a = np.max(np.abs(p), axis=1)
    inv = factor(a)
    codes = math_round_codes(p * inv[:, None]).astype(np.int8).reshape(x.shape)
    return codes, (a / 127.0).astype(np.float32).astype(np.float16).reshape(x.shape[:-1] + (-1,))


def rope_freqs(rot: int, base: float, scaling=None):
    """(frequencies f64 [rot/2], factor of cos and sin). scaling: a dict with
    "kind" linear / ntk / yarn / llama3 and its parameters."""
    i = np.arange(rot // 2, dtype=np.float64)
    s = scaling or {"kind": "none"}
    if s["kind"] == "ntk":
        base = base * s["factor"] ** (rot / (rot - 2))
    f = base ** (-2 * i / rot)
    if s["kind"] == "linear":
        return f / s["factor"], 1.0
    if s["kind"] == "yarn":
        def pair(turns):
            return rot * np.log(s["original_len"] / (turns * 2 * np.pi)) / (2 * np.log(base))
        lo, hi = max(np.floor(pair(s["high"])), 0), min(np.ceil(pair(s["low"])), rot - 1)
        t = np.clip((i - lo) / max(hi - lo, 0.001), 0, 1)
        return f / s["factor"] * t + f * (1 - t), s.get("attention") or 0.1 * np.log(s["factor"]) + 1
    if s["kind"] == "llama3":
        wavelen = 2 * np.pi / f
        smooth = (s["original_len"] / wavelen - s["low"]) / (s["high"] - s["low"])
        mid = (1 - smooth) * f / s["factor"] + smooth * f
        g = np.where(wavelen > s["original_len"] / s["low"], f / s["factor"], mid)
        return np.where(wavelen < s["original_len"] / s["high"], f, g), 1.0
    return f, 1.0


def rope_table(n_pos: int, rot: int, base: float, scaling=None):
    """(cos, sin) f64 [n_pos, rot/2, 2]."""
    f, factor = rope_freqs(rot, base, scaling)
    a = np.arange(n_pos, dtype=np.float64)[:, None] * f
    return np.stack([np.cos(a) * factor, np.sin(a) * factor], -1)


def rotate(x, table, positions, interleaved: bool, fused: bool = False):
    """f32 [n, heads, D] turned by the f32 table's angles: f64 sums rounded to f32;
    with `fused`, the second product is rounded to f32 before the sum."""
    second = (lambda v: v.astype(np.float32).astype(np.float64)) if fused else (lambda v: v)
    y = np.asarray(x, np.float32).astype(np.float64)
    cs = np.asarray(table, np.float32).astype(np.float64)[np.asarray(positions)]
    half = cs.shape[1]
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    x1, x2 = y[..., a], y[..., b]
    out = y.copy()
    out[..., a] = x1 * c - second(x2 * s)
    out[..., b] = x2 * c + second(x1 * s)
    return out.astype(np.float32)


def attention_rows(q, k, v, sees, scale: float, cap: float = 0.0):
    """Attention of query rows q [T, Hq, D] over k, v [Hkv, L, D]; sees [T, L]
    says which keys a row sees (none: zeros). f64 [T, Hq, D], and the largest
    |v| and scale * sum |q k| among what is seen."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    T, Hq, D = q.shape
    G = Hq // k.shape[0]
    out = np.zeros((T, Hq, D))
    vmax, smax = 0.0, 0.0
    for t in range(T):
        j = np.flatnonzero(sees[t])
        if not len(j):
            continue
        for h in range(Hq):
            kk, vv = k[h // G, j], v[h // G, j]
            s = float(np.float32(scale)) * (kk @ q[t, h])
            smax = max(smax, abs(scale) * float(np.max(np.abs(kk) @ np.abs(q[t, h]))))
            vmax = max(vmax, float(np.max(np.abs(vv))))
            if cap:
                s = cap * np.tanh(s / cap)
            p = np.exp(s - s.max())
            out[t, h] = (p @ vv) / p.sum()
    return out, vmax, smax
