"""The 4-bit formats and operators restated in numpy, sums and functions in
fp64, with the error each fp32 implementation is allowed (derived here, beside
the value it bounds).  U = 2^-24 is half an ulp of fp32, relative."""
from __future__ import annotations

import numpy as np

D = 128
U = 2.0 ** -24


def bf16_bits(x) -> np.ndarray:
    """fp32 -> bf16 bit patterns, nearest even (finite values)."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)


def bf16_val(bits) -> np.ndarray:
    return (np.asarray(bits, np.uint32) << 16).view(np.float32).astype(np.float64)


# ---- weights -----------------------------------------------------------------

def quant_w4(w_bits):
    """bf16 bits [N][K] -> (bytes [N][K/2], scale bits [N][K/128])."""
    w = bf16_val(w_bits).astype(np.float32)
    g = w.reshape(w.shape[0], -1, 128)
    s_bits = bf16_bits(np.abs(g).max(-1) / np.float32(7))
    s = bf16_val(s_bits).astype(np.float32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        u = np.where(s > 0, np.clip(np.rint(g / s), -8, 7), 0).astype(np.int32) + 8
    u = u.reshape(w.shape)
    return (u[:, 0::2] | (u[:, 1::2] << 4)).astype(np.uint8), s_bits


def dequant_w4(b, s_bits):
    u = np.stack((b & 15, b >> 4), -1).reshape(b.shape[0], -1).astype(np.float64) - 8
    return u * np.repeat(bf16_val(s_bits), 128, axis=1)


def gemv_w4(x, b, s_bits, epi=0, resid=None, gamma_bits=None, eps=1e-6):
    """(y, tolerance), fp64 [M][N].

    Each product a w of the kernel is exact up to the split of a into two fp16
    terms (4 U a); a group's 128 products are added in at most 8 steps of 2^-22
    of the group's magnitude, and the groups' results and the partial sums of
    up to 32 warps in one fp32 add each.  A byte's two codes are one operand, at
    most 8 + 16 . 8 times a 16th of an activation, beside 8 times the other, so
    magnitudes count 8 (1 + 1 / 8) |a| s per product and code, below B = sum |a|
    9 s.  The normalisation adds 16 U."""
    x = np.asarray(x, np.float64)
    w = dequant_w4(b, s_bits)
    K = x.shape[1]
    a = x
    if gamma_bits is not None:
        a = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * bf16_val(gamma_bits)
    acc = a @ w.T
    B = 9 * np.abs(a) @ np.repeat(bf16_val(s_bits), 128, axis=1).T
    tol = B * U * (4 + 8 * 4 + K / 128 + 32 + 16)
    if epi == 1:
        y = np.asarray(resid, np.float64) + acc
        return y, tol + 2 * U * np.abs(y)
    if epi == 2:
        N = acc.shape[1] // 2
        g, up, tg, tu = acc[:, :N], acc[:, N:], tol[:, :N], tol[:, N:]
        silu = g / (1 + np.exp(-np.maximum(g, -700)))
        # |d silu / d g| <= 1.1; the function and the product round in a few U
        return silu * up, 1.1 * tg * np.abs(up) + tu * (np.abs(silu) + 1.1 * tg) + 16 * U * np.abs(silu * up)
    return acc, tol


# ---- cache ---------------------------------------------------------------------

def quant_kv4(rows_bits):
    """bf16 bits [..., 128] -> (bytes [..., 64], parameter bits [..., 2, 2])."""
    x = bf16_val(rows_bits).astype(np.float32)
    x = x.reshape(x.shape[:-1] + (2, 64))
    lo, hi = x.min(-1) + np.float32(0), x.max(-1)  # a minimum of -0 is stored as 0
    s_bits = bf16_bits((hi - lo) / np.float32(15))
    s = bf16_val(s_bits).astype(np.float32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        u = np.where(s > 0, np.clip(np.rint((x - lo[..., None]) / s), 0, 15), 0).astype(np.uint8)
    u = u.reshape(u.shape[:-1] + (8, 4, 2))
    b = np.swapaxes(u[..., 0] | (u[..., 1] << 4), -3, -2)
    return (np.ascontiguousarray(b).reshape(b.shape[:-3] + (64,)),
            np.stack((s_bits, bf16_bits(lo)), -1))


def dequant_kv4(b, par_bits):
    """The cache's values, fp64 [..., 128]."""
    b = np.swapaxes(np.asarray(b).reshape(b.shape[:-1] + (8, 2, 4)), -3, -2)
    u = np.stack((b & 15, b >> 4), -1).astype(np.float64)
    u = u.reshape(u.shape[:-4] + (2, 64))
    p = bf16_val(par_bits)
    v = p[..., 1:] + p[..., :1] * u
    return v.reshape(v.shape[:-2] + (128,))


def kv4_size(b, par_bits):
    """|middle of the range| + 8.5 scale per channel: what the terms of a sum over a
    cached value scale with, its code taken from the middle (at most 8 steps off
    it, and half a step where the middle is between two codes)."""
    p = bf16_val(par_bits)
    return np.repeat(np.abs(p[..., 1] + 7.5 * p[..., 0]) + 8.5 * np.abs(p[..., 0]), 64, axis=-1)


def norm_rope(x, gain_bits, pos, eps, theta):
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * bf16_val(gain_bits)
    ang = pos * theta ** (-2 * np.arange(64) / D)
    c, s = np.cos(ang), np.sin(ang)
    a, b = y[..., :64], y[..., 64:]
    return np.concatenate((a * c - b * s, b * c + a * s), -1)


def attention_kv4(qkv, qn_bits, kn_bits, k4, kp, v4, vp, n_q, n_kv, pos, eps=1e-6, theta=1e6):
    """The cache arrays (bytes and parameter bits, [n_kv][max_pos]...) with row
    pos written, and the output with its tolerance: (k4, kp, v4, vp, out, tol).

    A score is off by S = sum |q| kv4_size / sqrt(128) times the
    relative error of the query (norm, rotation and its split: 16 U), of the
    dot product (8 steps of 4 U and the half's terms: 48 U) and of the
    exponential's argument; a probability by twice the largest such error plus
    the exponential's own 8 U; the output by that and the sums over the
    positions (at most 64 + n / 512 adds to any value beyond 512 positions a
    warp), each of sum p kv4_size."""
    x = np.asarray(qkv, np.float64).reshape(-1, D)
    q = norm_rope(x[:n_q], qn_bits, pos, eps, theta)
    kb = bf16_bits(norm_rope(x[n_q:n_q + n_kv], kn_bits, pos, eps, theta).astype(np.float32))
    vb = bf16_bits(x[n_q + n_kv:].astype(np.float32))
    k4, kp, v4, vp = k4.copy(), kp.copy(), v4.copy(), vp.copy()
    k4[:, pos], kp[:, pos] = quant_kv4(kb)
    v4[:, pos], vp[:, pos] = quant_kv4(vb)
    n, G = pos + 1, n_q // n_kv
    out, tol = np.zeros((n_q, D)), np.zeros((n_q, D))
    for j in range(n_kv):
        k, v = dequant_kv4(k4[j, :n], kp[j, :n]), dequant_kv4(v4[j, :n], vp[j, :n])
        kz, vz = kv4_size(k4[j, :n], kp[j, :n]), kv4_size(v4[j, :n], vp[j, :n])
        qh = q[j * G:(j + 1) * G]
        z = qh @ k.T / np.sqrt(D)
        p = np.exp(z - z.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        S = (np.abs(qh) @ kz.T / np.sqrt(D)).max(-1, keepdims=True)
        out[j * G:(j + 1) * G] = p @ v
        tol[j * G:(j + 1) * G] = (p @ vz) * (2 * S * U * (16 + 48 + 8) + U * (8 + 16 + 64 + n / 512))
    return k4, kp, v4, vp, out.reshape(-1), tol.reshape(-1)


# ---- scores ----------------------------------------------------------------------

def code_logprobs(z, codes, top, T):
    """z [rows][n_cb][V] (fp32 values): logprob, entropy, top codes, their log
    probabilities and a tolerance [rows][n_cb] for each kind.

    (z - max) / T rounds in 3 U of itself, the sum of exponentials in 8 U plus
    one U per add of a chain (V / 128 adds and 64 joins at most) and in 3 U of
    the exponents that carry weight (|entropy| + log V); the logarithm adds
    4 U of its value."""
    z = np.asarray(z, np.float64)
    V = z.shape[-1]
    with np.errstate(invalid="ignore", divide="ignore"):
        d = (z - z.max(-1, keepdims=True)) / T
        e = np.exp(d)
        total = e.sum(-1, keepdims=True)
        lp = d - np.log(total)
        p = e / total
        ent = -np.where(p > 0, p * lp, 0).sum(-1)
    order = np.argsort(np.where(np.isnan(z), -np.inf, -z), axis=-1, kind="stable") if not np.isnan(z).any() else None
    got = np.where((codes >= 0) & (codes < V),
                   np.take_along_axis(lp, np.clip(codes, 0, V - 1)[..., None].astype(np.int64), -1)[..., 0], np.nan)
    at = order[..., :top] if order is not None else None
    at_lp = np.take_along_axis(lp, at, -1) if at is not None else None
    chain = U * (8 + V / 128 + 64 + 3 * (np.abs(ent) + np.log(V)) + 4 * np.log(V))

    def tol(value):
        return chain[..., None] + 8 * U * (np.abs(value) + np.log(V))
    return got, ent, at, at_lp, tol(got[..., None])[..., 0], chain * (2 + np.log(V)), (tol(at_lp) if at is not None else None)
