"""How exact decode attention over a 4-bit cache has to be: as the formula evaluated
in fp32 on the dequantised cache, in the 2-norm over all heads.  A bound on the
largest possible error (four_bit_ref.attention_kv4's) is wider than what one
position of thousands contributes; this one is not."""
import numpy as np

import four_bit_ref as ref

D = 128


def values(k4, kp, v4, vp, j, pos):
    return ref.dequant_kv4(k4[j, :pos + 1], kp[j, :pos + 1]), ref.dequant_kv4(v4[j, :pos + 1], vp[j, :pos + 1])


def off(x, want):
    return np.linalg.norm(np.asarray(x, np.float64).ravel() - want) / np.linalg.norm(want)


def allowed(q, k4, kp, v4, vp, n_q, n_kv, pos, want):
    """The 2-norm error, relative, that an output for the queries q (rotated, fp64) may have.

    Twice the error of softmax(q K^T / sqrt(128)) V in fp32 (numpy, which adds
    pairwise along the last axis), whose own is one sample, half an ulp, and what
    the queries' roundings bring, which that form does not have, as its q is rounded
    once: the root of the mean square, its reciprocal, the product with it, the
    gain, two products and a sum of the rotation and the factor log2(e) / sqrt(128)
    are eight roundings of at most U (rms U / sqrt(3)), the two fp16 parts 2 U more
    (rms 2 U / sqrt(3)): sqrt(8 + 4) / sqrt(3) = 2 U rms in a channel's q.  A score
    moves by 2 U sqrt(sum q^2 k^2 / 128) then, and a weight p by p times that and
    the scores' common move, together at most 3 U of it."""
    G, outs, size = n_q // n_kv, [], 0.0
    for j in range(n_kv):
        k, v = values(k4, kp, v4, vp, j, pos)
        qh = q[j * G:(j + 1) * G]
        size += ((qh * qh) @ (k * k).mean(0) / D).sum() / n_q
        z = qh.astype(np.float32) @ k.astype(np.float32).T / np.float32(np.sqrt(D))
        p = np.exp(z - z.max(-1, keepdims=True))
        vt = np.ascontiguousarray(v.T.astype(np.float32))
        outs += [(vt * p[g]).sum(-1) / p[g].sum() for g in range(G)]
    return 2 * off(np.concatenate(outs), want) + ref.U + 3 * ref.U * np.sqrt(size)


def judged(qkv, qn, kn, k4, kp, v4, vp, n_q, n_kv, pos):
    """The output in fp64, and the 2-norm error that is allowed."""
    rk4, rkp, rv4, rvp, want, _ = ref.attention_kv4(qkv, qn, kn, k4, kp, v4, vp, n_q, n_kv, pos)
    q = ref.norm_rope(np.asarray(qkv, np.float64).reshape(-1, D)[:n_q], qn, pos, 1e-6, 1e6)
    return want, allowed(q, rk4, rkp, rv4, rvp, n_q, n_kv, pos, want)


def dominated(qkv, qn, kn, k4, kp, pos, n_q, n_kv, at):
    """A copy of the keys in which head j's position at[j] (pos: the new row) takes
    almost all the weight: its key lies along the sum of the head's queries."""
    G = n_q // n_kv
    x = np.asarray(qkv, np.float64).reshape(-1, D).copy()
    k4, kp = k4.copy(), kp.copy()
    q = ref.norm_rope(x[:n_q], qn, pos, 1e-6, 1e6).reshape(n_kv, G, D).sum(1)
    for j, t in enumerate(at):
        if t < pos:
            k4[j, t], kp[j, t] = ref.quant_kv4(ref.bf16_bits((6.0 * q[j]).astype(np.float32)))
    return k4, kp
