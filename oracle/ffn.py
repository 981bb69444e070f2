"""CPU oracle of the gated feed-forward block and of microscaled 4-bit floating
point, in numpy and 64-bit floating point, written from the definitions in
include/nmspmm.h.  Test infrastructure only; shares no code with the library.
"""
from __future__ import annotations

import math

import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
_erf = np.vectorize(math.erf, otypes=[np.float64])


# ------------------------------------------------------------------ activations

def act(v, name):
    v = np.asarray(v, np.float64)
    if name == "none":
        return v
    if name == "relu":
        return np.where(v > 0, v, 0.0)
    if name == "silu":
        return v * _sigmoid(v)
    return 0.5 * v * (1.0 + _erf(v / math.sqrt(2.0)))


def act_slope(v, name):
    """Derivative of act (relu: 0 at 0)."""
    v = np.asarray(v, np.float64)
    if name == "none":
        return np.ones_like(v)
    if name == "relu":
        return (v > 0).astype(np.float64)
    if name == "silu":
        s = _sigmoid(v)
        return s * (1.0 + v * (1.0 - s))
    return 0.5 * (1.0 + _erf(v / math.sqrt(2.0))) + v * np.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)


def _sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


# ------------------------------------------------------------------ gated block

def mask(W, N, M):
    """W with only the N largest magnitudes of every M kept, ties to the lower position."""
    W = np.asarray(W)
    g = W.reshape(W.shape[0], -1, M).astype(np.float64)
    rank = np.zeros(g.shape, np.int64)
    for p in range(M):
        for q in range(M):
            first = (np.abs(g[:, :, q]) > np.abs(g[:, :, p])) | ((np.abs(g[:, :, q]) == np.abs(g[:, :, p])) & (q < p))
            rank[:, :, p] += first & (q != p)
    return np.where((rank < N).reshape(W.shape), W, np.zeros_like(W))


def gated_pre(X, Wm, scale=None, bias=None):
    p = np.asarray(X, np.float64) @ np.asarray(Wm, np.float64).T
    if scale is not None:
        p = p * np.asarray(scale, np.float64)
    if bias is not None:
        p = p + np.asarray(bias, np.float64)
    return p


def gated(p, name):
    f = p.shape[1] // 2
    return act(p[:, :f], name) * p[:, f:]


def gated_dp(p, dY, name):
    p, dY = np.asarray(p, np.float64), np.asarray(dY, np.float64)
    f = p.shape[1] // 2
    g, u = p[:, :f], p[:, f:]
    return np.concatenate([dY * u * act_slope(g, name), dY * act(g, name)], axis=1)


# ------------------------------------------------------------------ microscaled values

def mx_quantize(x):
    """Codes [rows, k] (0 .. 15) and scale bytes [rows, k / 32] of x (float64 holds
    every fp32, fp16 and bf16 value exactly)."""
    x = np.asarray(x, np.float64)
    rows, k = x.shape
    b = x.reshape(rows, k // 32, 32)
    codes = np.zeros(b.shape, np.uint8)
    byte = np.zeros(b.shape[:2], np.uint8)
    for r in range(rows):
        for i in range(k // 32):
            v = b[r, i]
            if not np.all(np.isfinite(v)):
                byte[r, i] = 255
                continue
            top = np.abs(v).max()
            e = -127 if top == 0 else max(math.frexp(top)[1] - 1 - 2, -127)
            byte[r, i] = e + 127
            a = np.abs(v) / 2.0 ** e
            # distance to every level; a tie goes to the even code
            d = np.abs(a[:, None] - LEVELS[None, :])
            best = d.min(axis=1, keepdims=True)
            near = d == best
            even = near & (np.arange(8) % 2 == 0)
            pick = np.where(even.any(axis=1), even.argmax(axis=1), near.argmax(axis=1))
            codes[r, i] = pick + 8 * np.signbit(v)
    return codes.reshape(rows, k), byte


def mx_values(codes, byte):
    """What codes [rows, k] and scale bytes [rows, k / 32] stand for (byte 255: NaN)."""
    v = LEVELS[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127.0))
    return (v.reshape(*byte.shape, 32) * s[:, :, None]).reshape(codes.shape)


def mx_pack_codes(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def mx_pack_scales(byte):
    """Scale bytes in the tiled layout, byte by byte from the header's formula."""
    rows, nb = byte.shape
    n_kb = -(-nb // 8)
    out = np.zeros(-(-rows // 128) * n_kb * 1024, np.uint8)
    for r in range(rows):
        for b in range(nb):
            out[((r // 128) * n_kb + b // 8) * 1024 + ((b % 8) // 4) * 512 + (r % 32) * 16 + ((r % 128) // 32) * 4
                + b % 4] = byte[r, b]
    return out
