"""Plain fp64 oracle of the MXFP4 and mixture-of-experts operators (test infrastructure).

Written from the definitions, in numpy: e2m1 codes under one power-of-two scale
per 32 values, and router -> top-k -> gated experts -> weighted sum.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x):
    """x [..., K] (any float array) -> (codes uint8 [..., K/2], scale bytes uint8 [..., K/32])."""
    v = np.asarray(x, dtype=np.float64)
    v = v.reshape(*v.shape[:-1], -1, 32)
    finite = np.isfinite(v).all(-1)
    a = np.where(np.isfinite(v), np.abs(v), 0.0)
    amax = a.max(-1)
    e = np.frexp(amax)[1] - 1                                  # floor(log2) of a positive number
    byte = np.where(amax > 0, np.clip(e - 2, -127, 127), -127) + 127
    r = a / np.ldexp(1.0, byte - 127)[..., None]
    # the nearest of the eight magnitudes, the even code where two are as near
    d = np.abs(r[..., None] - E2M1)
    order = np.array([0, 2, 4, 6, 1, 3, 5, 7])                 # even codes first: argmin takes the first smallest
    idx = order[np.argmin(d[..., order], -1)]
    idx = idx + 8 * np.signbit(v)
    byte = np.where(finite, byte, 255)
    idx = np.where(finite[..., None], idx, 0).reshape(*v.shape[:-2], -1)
    return (idx[..., 0::2] | (idx[..., 1::2] << 4)).astype(np.uint8), byte.astype(np.uint8)


def values(codes, scales):
    """fp64 values [..., K]."""
    idx = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = np.where(idx >= 8, -E2M1[idx & 7], E2M1[idx & 7])
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(s, 32, -1)


def gemm(x, w):
    """(x . w^T, sum of the products' magnitudes) for x [M, K], w [N, K] in fp64."""
    return x @ w.T, np.abs(x) @ np.abs(w).T


def sum_error(K):
    """Bound of an fp32 product sum over K, relative to the sum of magnitudes: at most 32 additions
    inside a matrix instruction, K / 32 instructions in a row, and the joins of partial sums (allowed 32),
    each off by one step of fp32 (an instruction may truncate)."""
    return (K / 32 + 64) * 2.0 ** -23


def route(x, w_router, k, renorm):
    """Chosen experts [T, k] and their weights, ties to the lowest index."""
    logits = x @ w_router.T
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :k]
    top = np.take_along_axis(logits, ids, 1)
    p = np.exp(top - top[:, :1])
    total = p.sum(1, keepdims=True) if renorm else np.exp(logits - top[:, :1]).sum(1, keepdims=True)
    return ids, p / total


def moe_layer(x, w_router, k, w_gate_up, w_down, renorm, out_eps):
    """(out, error bound) for x [T, H], w_gate_up [E, 2I, H], w_down [E, H, I] in fp64.

    The bound counts fp32 sums, h held in two 16-bit parts (2^-15 of each value
    in bf16; in fp16, under the row's scale, 2^-22 and 2^-38 of the row's
    largest), the fp32 silu and router weights (2^-20) and the output's rounding
    (out_eps / 2)."""
    ids, c = route(x, w_router, k, renorm)
    T, H = x.shape
    I = w_down.shape[2]
    out, err = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            wg, wd = w_gate_up[ids[t, j]], w_down[ids[t, j]]
            gu, mag = wg @ x[t], np.abs(wg) @ np.abs(x[t])
            g, u = gu[:I], gu[I:]
            dg, du = (sum_error(H) * mag)[:I], (sum_error(H) * mag)[I:]
            s = g / (1 + np.exp(-g))
            h = s * u
            dh = 1.1 * dg * (np.abs(u) + du) + np.abs(s) * du + np.abs(h) * 2.0 ** -15 + np.abs(h).max() * 2.0 ** -38
            y = wd @ h
            out[t] += c[t, j] * y
            err[t] += c[t, j] * (np.abs(wd) @ dh + (sum_error(I) + 2.0 ** -20) * (np.abs(wd) @ (np.abs(h) + dh)))
    return out, err * 1.01 + out_eps / 2 * (np.abs(out) + err)
