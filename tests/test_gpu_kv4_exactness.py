"""Decode attention over a 4-bit cache, however a head's cache is divided and its
queries are grouped, is as exact as fp32 on the dequantised values; and every
position that can hold the weight is read."""
import numpy as np
import pytest

import kv4_exactness as kx
from test_gpu_four_bit import ATTN, DIVIDED, Attn, cache, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ads():
    import torch
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    import ar_decode_step_gb300.build as b
    b.build()
    import ar_decode_step_gb300 as m
    m.load()
    return m


# Beside the shapes tested for their values: each number of queries a head (1, 2, 4, 8)
# in one block, in a cluster and joined through the workspace, with heads so many
# that four and eight are not taken as two heads, and the longest caches.
MORE = [(8, 8, 150), (80, 80, 190), (16, 16, 2500), (4, 4, 9000), (2, 1, 150), (160, 80, 190), (2, 1, 12000), (320, 80, 150),
        (32, 8, 1500), (32, 8, 9000), (640, 80, 150), (128, 16, 1800), (128, 16, 7000), (48, 6, 3000), (4, 1, 70000),
        (8, 1, 70000), (1, 1, 70000), (2, 1, 70000), (32, 4, 21000)]
SHAPES = sorted({(n_q, n_kv, pos) for n_q, n_kv, _, pos in ATTN} | set(DIVIDED) | set(MORE))


@pytest.mark.parametrize("n_q,n_kv,pos", SHAPES)
def test_as_exact_as_fp32_on_the_values(ads, n_q, n_kv, pos):
    a = Attn(ads, n_q, n_kv, pos + 2, pos)
    a.call()
    want, limit = kx.judged(a.qkv, a.qn, a.kn, a.k4, a.kp, a.v4, a.vp, n_q, n_kv, pos)
    got = kx.off(host(a.out), want)
    assert got <= limit, (got, limit)


@pytest.mark.parametrize("n_q,n_kv,pos", [(32, 8, 100), (32, 8, 1279), (32, 8, 9000), (16, 2, 700), (64, 8, 4000), (2, 1, 8300),
                                          (8, 8, 500), (24, 3, 31)])
def test_one_position_holds_the_weight(ads, n_q, n_kv, pos):
    """The first, the last cached, either side of tiles' and shares' borders, the new row."""
    tiles = (pos + 15) // 16
    borders = [0, pos - 1, pos, 15, 16, 16 * (tiles // 2), 16 * (tiles // 2) - 1, 16 * (tiles - 1), 16 * (tiles - 1) - 1]
    borders += [16 * t + d for t in range(0, tiles, max(1, tiles // 23)) for d in (0, 15)]
    borders = sorted({t for t in borders if 0 <= t <= pos})
    k4, kp, v4, vp = cache(n_kv, pos + 2, 130)
    for i in range(0, len(borders), n_kv):
        at = [borders[(i + j) % len(borders)] for j in range(n_kv)]
        a = Attn(ads, n_q, n_kv, pos + 2, pos, arrays=(k4.copy(), kp.copy(), v4.copy(), vp.copy()))
        a.k4, a.kp = kx.dominated(a.qkv, a.qn, a.kn, a.k4, a.kp, pos, n_q, n_kv, at)
        a.d[3].copy_(_like(a.k4))
        a.d[5].copy_(_like(a.kp))
        a.call()
        a.check(str(at))


def _like(x):
    import torch
    return torch.from_numpy(x.view(np.int16) if x.dtype == np.uint16 else x).cuda()


@pytest.mark.parametrize("n_q,n_kv,pos", [(8, 2, 20), (8, 2, 700), (4, 1, 9000), (16, 2, 3000)])
@pytest.mark.parametrize("scale", [2.0 ** 98, 2.0 ** -100])
def test_values_of_extreme_size(ads, n_q, n_kv, pos, scale):
    """Value rows next to the largest and far below one: as exact as ordinary ones."""
    import four_bit_ref as ref
    import synth
    k4, kp, _, _ = cache(n_kv, pos + 2, 140)
    v = synth.normal_f32(1, 141, (n_kv, pos + 2, 128)).astype(np.float64) * scale
    v4, vp = ref.quant_kv4(ref.bf16_bits(v.astype(np.float32)))
    a = Attn(ads, n_q, n_kv, pos + 2, pos, arrays=(k4, kp, v4, vp))
    a.qkv[(n_q + n_kv) * 128:] *= np.float32(scale)
    a.d[0].copy_(_like(a.qkv))
    a.call()
    a.check()
    want, limit = kx.judged(a.qkv, a.qn, a.kn, a.k4, a.kp, a.v4, a.vp, n_q, n_kv, pos)
    got = kx.off(host(a.out), want)
    assert got <= limit, (got, limit)
