"""CPU oracle of the decoder-layer operators (test infrastructure only).

Plain numpy, written from the formulas of include/bq_decode.h and sharing no
code with the CUDA path: float64 for the products, and IEEE float32 in the
stated order for the cache write, whose codes are compared bit for bit.
"""

from __future__ import annotations

import numpy as np

F32 = np.float32


def unpack4(p):
    """(..., n) packed bytes -> (..., 2 n) codes 0..15, low four bits first."""
    out = np.empty(p.shape[:-1] + (2 * p.shape[-1],), np.int64)
    out[..., 0::2] = p & 15
    out[..., 1::2] = p >> 4
    return out


def group_weights(codes, scale, zero, group):
    """Codes (N, K) (signed if zero is None, else 0..15) -> float64 weights."""
    z = 0.0 if zero is None else np.repeat(zero.astype(np.float64), group, axis=1)
    return (codes.astype(np.float64) - z) * np.repeat(scale.astype(np.float64), group, axis=1)


def activate(v, act):
    if act == "relu":
        return np.maximum(v, 0.0)
    if act == "gelu":
        from math import erfc
        return np.array([0.5 * x * erfc(-x / np.sqrt(2.0)) for x in v.ravel()]).reshape(v.shape)
    return v


def gemm_group(x, codes, scale, zero, group, act="none"):
    """(result, bound): the float64 product, and how far an evaluation may be from it that sums the codes of each
    group (as they are, or offset by 8) in fp32 and rounds once to fp16 at the end.  A chain of n fp32 additions of
    terms with absolute sum S is off by at most n 2**-23 S (2**-23: tensor cores may truncate); a group takes
    group / 16 + 8 of them, the groups K / group, the joining of parts of K at most 16 more."""
    w = group_weights(codes, scale, zero, group)
    y = x.astype(np.float64) @ w.T
    z = np.full_like(scale, 8) if zero is None else zero
    size = np.abs(np.repeat(scale.astype(np.float64), group, axis=1)) * \
        (15.0 + np.repeat(np.abs(z.astype(np.float64)) + 8.0, group, axis=1))
    total = np.abs(x.astype(np.float64)) @ size.T
    n = group / 16 + 8 + x.shape[1] / group + 16
    slope = 1.13 if act == "gelu" else 1.0          # largest derivative of GELU
    v = activate(y, act)
    return v, slope * n * 2.0 ** -23 * total + (2.0 ** -11 + 2.0 ** -20) * np.abs(v) + 2.0 ** -25


# ---- norm, rotation, write ------------------------------------------------------------------------------------------


def head_norm(x, weight, eps):
    """x (..., D) fp16 -> fp32, every operation rounded to fp32; the sum by neighbouring pairs."""
    y = x.astype(F32)
    if weight is None:
        return y
    s = y * y
    while s.shape[-1] > 1:
        s = s[..., 0::2] + s[..., 1::2]
    r = F32(1) / np.sqrt(s * F32(1.0 / x.shape[-1]) + F32(eps))
    return (y * r) * weight.astype(F32)


def rotate(y, cos, sin, positions, pairs):
    """y (T, heads, D) fp32, the first 2 * cos.shape[1] dims turned -> fp16."""
    y = y.copy()
    half = cos.shape[1]
    c, s = cos[positions][:, None, :], sin[positions][:, None, :]
    ia = np.arange(half) * 2 if pairs else np.arange(half)
    ib = ia + 1 if pairs else ia + half
    a, b = y[..., ia], y[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y.astype(np.float16)


def code_groups(x, group):
    """x (..., D) fp16 -> (codes 0..15, step fp16, low fp16, values fp16)."""
    y = x.astype(F32).reshape(x.shape[:-1] + (-1, group))
    low = y.min(-1) + F32(0)
    step = ((y.max(-1) - low) / F32(15)).astype(np.float16)
    st = step.astype(F32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        u = np.where(st > 0, np.rint((y - low[..., None]) / st), F32(0))
    u = np.clip(u, 0, 15).astype(F32)
    values = (u * st + low[..., None]).astype(np.float16)
    return u.reshape(x.shape).astype(np.uint8), step, low.astype(np.float16), values.reshape(x.shape)


def write(q, k, v, codes, params, slots, positions, cos, sin, q_weight, k_weight, eps, pairs):
    """Updates codes and params in place; returns (q_out, k_values, v_values)."""
    def turned(x, w):
        y = head_norm(x, w, eps)
        return rotate(y, cos, sin, positions, pairs) if cos is not None else y.astype(np.float16)
    page = codes.shape[3]
    group = 2 * codes.shape[4] // params.shape[4]
    values = []
    for i, x in enumerate((turned(k, k_weight), v)):
        u, step, low, val = code_groups(x, group)
        values.append(val)
        for t, slot in enumerate(slots):
            if slot >= 0:
                codes[slot // page, i, :, slot % page] = u[t][..., 0::2] | (u[t][..., 1::2] << 4)
                params[slot // page, i, :, slot % page] = np.stack([step[t], low[t]], -1)
    return turned(q, q_weight), values[0], values[1]


# ---- attention ------------------------------------------------------------------------------------------------------


def cache_values(codes, params, table_row, length):
    """Keys and values (2, heads, length, D) of one sequence in float64, and the lows of its values' groups."""
    page = codes.shape[3]
    blocks = table_row[: -(-length // page)]
    u = unpack4(codes[blocks]).astype(np.float64)
    group = u.shape[-1] // params.shape[4]
    step, low = np.repeat(params[blocks].astype(np.float64), group, axis=4).transpose(5, 0, 1, 2, 3, 4)

    def rows(x):
        return x.transpose(1, 2, 0, 3, 4).reshape(2, codes.shape[2], -1, u.shape[-1])[:, :, :length]
    return rows(u * step + low), rows(np.abs(low))[1]


def attention(q, codes, params, table, lens, cu_q, scale, window=0):
    """(out, lse, bound of out, bound of lse), float64.  The bounds are those of an evaluation with fp32 scores whose
    weights, times the values' steps, are rounded to fp16: 2**-11 for the rounding of the result, 2**-11 of each
    weighted term |v| + 2 |low| for the weights, and twice the error of a score (D + 16 fp32 additions)."""
    T, heads, D = q.shape
    kv = codes.shape[2]
    rep = heads // kv
    out, lse = np.zeros((T, heads, D)), np.full((T, heads), -np.inf)
    tol, tol_lse = np.full((T, heads, D), 2.0 ** -25), np.zeros((T, heads))
    if cu_q is None:
        cu_q = np.arange(len(lens) + 1)
    for b, n in enumerate(lens):
        m = int(cu_q[b + 1] - cu_q[b])
        if n == 0 or m == 0:
            continue
        x, low = cache_values(codes, params, table[b], int(n))
        for i in range(m):
            t, p = int(cu_q[b]) + i, int(n) - m + i
            begin = max(0, p + 1 - window) if window else 0
            if p < 0:
                continue
            for h in range(heads):
                k, v = x[0, h // rep, begin:p + 1], x[1, h // rep, begin:p + 1]
                qq = q[t, h].astype(np.float64)
                s = k @ qq * scale
                ds = abs(scale) * (D + 16) * 2.0 ** -23 * (np.abs(k) @ np.abs(qq)).max() * 2 + 2.0 ** -21 * np.abs(s).max()
                e = np.exp(s - s.max())
                w = e / e.sum()
                out[t, h] = w @ v
                lse[t, h] = s.max() + np.log(e.sum())
                tol[t, h] += 2.0 ** -11 * np.abs(out[t, h]) + \
                    (2.0 ** -11 + 2 * ds + 2.0 ** -20) * (w @ (np.abs(v) + 2 * low[h // rep, begin:p + 1]))
                tol_lse[t, h] = ds + 2.0 ** -20 + 2.0 ** -22 * abs(lse[t, h])
    return out, lse, tol, tol_lse
