"""The bound that decode attention over a 4-bit cache is held to sees one position
left out, and operands of 11 bits instead of 22 (mistakes made in the restatement;
no GPU needed)."""
import numpy as np
import pytest

import four_bit_ref as ref
import kv4_exactness as kx
import synth

D = 128


@pytest.mark.parametrize("n_q,n_kv,pos", [(4, 1, 8193), (8, 1, 8193), (2, 2, 3900), (16, 2, 1000), (4, 1, 70000)])
def test_the_bound_sees_one_position(n_q, n_kv, pos):
    rng = np.random.default_rng(pos)
    G = n_q // n_kv
    q = rng.standard_normal((n_q, D))
    k4, kp = ref.quant_kv4(synth.normal_bf16(1, 5, (n_kv, pos + 1, D)))
    v4, vp = ref.quant_kv4(synth.normal_bf16(1, 6, (n_kv, pos + 1, D)))
    k, v = ref.dequant_kv4(k4, kp), ref.dequant_kv4(v4, vp)

    def exact(left_out=None, q=q):
        outs = []
        for h in range(n_q):
            z = q[h] @ k[h // G].T / np.sqrt(D)
            if left_out is not None and h // G == n_kv - 1:
                z[left_out] = -np.inf
            p = np.exp(z - z.max())
            outs.append(p @ v[h // G] / p.sum())
        return np.concatenate(outs)

    want = exact()
    limit = kx.allowed(q, k4, kp, v4, vp, n_q, n_kv, pos, want)
    assert limit < 3e-6
    likely = int(np.argsort(k[-1] @ q[-1])[len(k[-1]) // 2])  # a position of middling weight
    for t in (likely, pos, 0):
        assert kx.off(exact(t), want) > 10 * limit, t
    assert kx.off(exact(q=q.astype(np.float16).astype(np.float64)), want) > 10 * limit
