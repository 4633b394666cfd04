"""4-bit weights, the 4-bit cache and the decode attention over it, on the GPU,
against the fp64 restatement (four_bit_ref): formats bit for bit, sums within
the tolerances derived there."""
import numpy as np
import pytest

import four_bit_ref as ref
import synth

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def ads():
    import torch
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    import ar_decode_step_gb300.build as b
    b.build()
    import ar_decode_step_gb300 as m
    m.load()
    return m


def dev(a):
    import torch
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).cuda()


def host(t):
    a = t.cpu().numpy()
    return a.view(np.uint16) if a.dtype == np.int16 else a


def bits(t):
    import torch
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


def near(got, want, tol, where=""):
    err = np.abs(got.astype(np.float64) - want)
    assert np.isfinite(got).all() and (err <= tol).all(), \
        f"{where}: {err.max()} at {np.unravel_index(np.argmax(err - tol), err.shape)}, allowed {tol.flat[np.argmax(err - tol)]}"


# ---- weights -----------------------------------------------------------------------

@pytest.mark.parametrize("shape", [(1, 128), (37, 1280), (2560, 4096)])
def test_quantize_w4_bit_exact(ads, shape):
    w = synth.normal_bf16(0, 700 + shape[0], shape, std=0.02)
    w[0, :64] = 0x0001                             # subnormals beside ordinary weights
    if shape[0] > 1:
        w[3, :128] = 0                             # scale 0
        w[4, :128] = 0x0080                        # the smallest normal numbers: a subnormal scale
        w[5, :4] = [0x7F7F, 0xFF7F, 0x7E80, 0]     # the largest finite ones
        w[6, :128] = ref.bf16_bits(np.arange(128) - 63.5)  # many ties
    b, s = ref.quant_w4(w)
    q, sc = ads.quantize_w4_weight(dev(w))
    assert np.array_equal(bits(sc), s)
    assert np.array_equal(host(q), b)


def weights(N, K, seed):
    return ref.quant_w4(synth.normal_bf16(0, seed, (N, K), std=0.02))


GEMV = [(1, 1, 128, 0, False), (1, 17, 256, 1, True), (1, 160, 4096, 1, False), (2, 48, 1280, 2, True),
        (3, 1026, 2560, 0, True), (4, 500, 384, 0, True), (5, 33, 12288, 1, False), (6, 15, 640, 2, False),
        (7, 16, 128, 2, True), (8, 2560, 9728, 1, False), (1, 9728, 2560, 2, True), (1, 2560, 9728, 1, False),
        (1, 6144, 2560, 0, True), (8, 8208, 2560, 0, True), (4, 9728, 2560, 2, True), (3, 40, 384, 2, False),
        (4, 700, 12288, 2, True), (8, 1300, 4096, 2, True), (2, 4001, 9728, 1, False), (1, 30000, 256, 1, False),
        (4, 20, 2432, 2, False), (8, 33, 2432, 0, True)]


@pytest.mark.parametrize("M,N,K,epi,norm", GEMV)
def test_gemv_w4(ads, M, N, K, epi, norm):
    import torch
    rows = 2 * N if epi == 2 else N
    b, s = weights(rows, K, 800 + N % 97)
    x = synth.normal_f32(5, 900 + M, (M, K), std=1.5)
    x[0, :128] *= 3000.0        # an outlier group
    x[-1, K - 128:] *= 1e-4     # and one of small values
    x[:, 5] = 0
    resid = synth.normal_f32(5, 901, (M, N)) if epi == 1 else None
    gamma = synth.normal_bf16(3, 902, (K,), std=0.02, mean=1.0) if norm else None
    want, tol = ref.gemv_w4(x, b, s, epi, resid, gamma)
    pad = torch.full((2 * M * N + 64,), 7.25, device="cuda")
    y = pad[32:32 + M * N].view(M, N)
    args = (dev(x), dev(b), dev(s), y, epi, None if resid is None else dev(resid), None if gamma is None else dev(gamma))
    ads.gemv_w4(*args)
    near(host(y), want, tol)
    first = y.clone()
    assert (pad[:32] == 7.25).all() and (pad[32 + M * N:] == 7.25).all()  # nothing else written
    ads.gemv_w4(*args)
    assert torch.equal(first, y)
    if epi == 1:  # in place
        y.copy_(dev(resid))
        ads.gemv_w4(*args[:5], y, args[6])
        assert torch.equal(first, y)


@pytest.mark.parametrize("scale", [1e-30, 1e30])
@pytest.mark.parametrize("norm", [False, True])
def test_gemv_w4_extreme_inputs(ads, scale, norm):
    """Inputs far outside the 16-bit ranges; normalised, they are ordinary
    (1e30 squared overflows fp32, so that one is left out)."""
    import torch
    if norm and scale > 1:
        scale = 1e15
    b, s = weights(40, 512, 31)
    x = synth.normal_f32(5, 31, (2, 512)) * np.float32(scale)
    x[1] = 0
    gamma = synth.normal_bf16(3, 902, (512,), std=0.02, mean=1.0) if norm else None
    want, tol = ref.gemv_w4(x, b, s, 0, None, gamma)
    y = torch.empty((2, 40), device="cuda")
    ads.gemv_w4(dev(x), dev(b), dev(s), y, 0, None, None if gamma is None else dev(gamma))
    near(host(y), want, tol)
    assert (y[1] == 0).all()


def test_gemv_w4_non_finite_input_reaches_its_row_only(ads):
    import torch
    b, s = weights(64, 256, 33)
    x = synth.normal_f32(5, 33, (3, 256))
    x[0, 17], x[2, 200] = np.nan, np.inf
    y = torch.empty((3, 64), device="cuda")
    ads.gemv_w4(dev(x), dev(b), dev(s), y)
    assert not torch.isfinite(y[0]).any()
    want, tol = ref.gemv_w4(x[1:2], b, s)
    near(host(y[1:2]), want, tol)
    w = ref.dequant_w4(b, s)[:, 200]
    assert not torch.isfinite(y[2][torch.from_numpy(w != 0).cuda()]).any()


# ---- cache -----------------------------------------------------------------------------

def cache(n_kv, max_pos, seed, std=1.0):
    """A 4-bit cache of N(0, std) rows, host arrays (k4, k_par, v4, v_par)."""
    k4, kp = ref.quant_kv4(synth.normal_bf16(1, seed, (n_kv, max_pos, D), std=std))
    v4, vp = ref.quant_kv4(synth.normal_bf16(1, seed + 1, (n_kv, max_pos, D), std=std))
    return k4, kp, v4, vp


@pytest.mark.parametrize("n_kv,stride,max_pos,p0,p1", [(1, 1, 1, 0, 1), (3, 40, 57, 5, 38), (8, 300, 141, 0, 141),
                                                       (2, 2050, 4096, 1999, 2050), (40, 9, 9, 8, 9)])
def test_quantize_kv4_bit_exact_and_back(ads, n_kv, stride, max_pos, p0, p1):
    import torch
    k = synth.normal_bf16(1, 50, (n_kv, stride, D))
    v = synth.normal_bf16(1, 51, (n_kv, stride, D), std=30.0)
    k[0, p0, :64] = 0x3F80              # a constant half
    k[0, p0, 64:] = 0x0001              # subnormals
    v[0, p1 - 1, 3] = 0x7E00            # 4e37 among ordinary values
    v[-1, p0] = ref.bf16_bits(np.arange(128) / 2)
    k4 = torch.full((n_kv, max_pos, 64), 0xA5, dtype=torch.uint8, device="cuda")
    v4 = k4.clone()
    kp = torch.full((n_kv, max_pos, 2, 2), 0x1234, dtype=torch.int16, device="cuda")
    vp = kp.clone()
    ads.quantize_kv4(dev(k), dev(v), k4, v4, kp, vp, p0, p1)
    for src, b, p in ((k, k4, kp), (v, v4, vp)):
        rb, rp = ref.quant_kv4(src[:, p0:p1])
        assert np.array_equal(host(b)[:, p0:p1], rb) and np.array_equal(host(p)[:, p0:p1], rp)
        out = np.ones(max_pos, bool)
        out[p0:p1] = False
        assert (host(b)[:, out] == 0xA5).all() and (host(p)[:, out] == 0x1234).all()
    ko = torch.full((n_kv, p1 + 3, D), 0x4321, dtype=torch.int16, device="cuda")
    vo = ko.clone()
    ads.dequantize_kv4(k4, v4, kp, vp, ko, vo, p0, p1)
    for src, o in ((k, ko), (v, vo)):
        vals = ref.dequant_kv4(*ref.quant_kv4(src[:, p0:p1]))
        assert np.array_equal(host(o)[:, p0:p1], ref.bf16_bits(vals.astype(np.float32)))
        assert (host(o)[:, :p0] == 0x4321).all() and (host(o)[:, p1:] == 0x4321).all()


def test_quantize_kv4_non_finite_halves_read_as_nan(ads):
    import torch
    k = synth.normal_bf16(1, 52, (1, 4, D))
    k[0, 0, 7], k[0, 1, 100], k[0, 2, 1] = 0x7FC0, 0xFF80, 0x7F80
    k[0, 3, :2] = [0x7F7F, 0xFF7F]  # a range beyond fp32
    k4 = torch.zeros((1, 4, 64), dtype=torch.uint8, device="cuda")
    v4, kp = k4.clone(), torch.zeros((1, 4, 2, 2), dtype=torch.int16, device="cuda")
    vp, o, o2 = kp.clone(), torch.zeros((1, 4, D), dtype=torch.bfloat16, device="cuda"), None
    o2 = o.clone()
    ads.quantize_kv4(dev(k), dev(k), k4, v4, kp, vp, 0, 4)
    ads.dequantize_kv4(k4, v4, kp, vp, o, o2, 0, 4)
    nan = torch.isnan(o[0]).view(4, 2, 64).all(-1).cpu().numpy()
    none = (~torch.isnan(o[0])).view(4, 2, 64).all(-1).cpu().numpy()
    want = np.array([[True, False], [False, True], [True, False], [True, False]])
    assert np.array_equal(nan, want) and np.array_equal(none, ~want) and torch.equal(o.isnan(), o2.isnan())


class Attn:
    """One call's device tensors, rows past pos filled with what must not be read."""

    def __init__(self, ads, n_q, n_kv, max_pos, pos, seed=60, std=1.0, arrays=None):
        import torch
        self.ads, self.n_q, self.n_kv, self.pos = ads, n_q, n_kv, pos
        self.qkv = synth.normal_f32(5, seed + pos % 101, ((n_q + 2 * n_kv) * D,), std=1.5)
        self.qn = synth.normal_bf16(3, seed + 1, (D,), std=0.02, mean=1.0)
        self.kn = synth.normal_bf16(3, seed + 2, (D,), std=0.02, mean=1.0)
        self.k4, self.kp, self.v4, self.vp = arrays or cache(n_kv, max_pos, seed + 3, std)
        for b in (self.k4, self.v4):
            b[:, pos:] = 0xFF
        for p in (self.kp, self.vp):
            p[:, pos:] = 0x7FFF  # NaN
        self.d = [dev(a) for a in (self.qkv, self.qn, self.kn, self.k4, self.v4, self.kp, self.vp)]
        self.out = torch.full((n_q * D,), np.nan, device="cuda")
        self.row = torch.full((2, n_kv, D), np.nan, device="cuda")
        self.ws = torch.zeros(ads.kv4_workspace_bytes(n_q, n_kv), dtype=torch.uint8, device="cuda")

    def call(self, stream=None, ws=None):
        self.ads.attention_decode_kv4(*self.d, self.out, self.n_q, self.n_kv, self.pos, self.ws if ws is None else ws,
                                      kv_row=self.row, stream=stream)

    def check(self, where=""):
        rk4, rkp, rv4, rvp, out, tol = ref.attention_kv4(self.qkv, self.qn, self.kn, self.k4, self.kp, self.v4,
                                                         self.vp, self.n_q, self.n_kv, self.pos)
        near(host(self.out), out, tol, where)
        for got, want in zip(self.d[3:], (rk4, rv4, rkp, rvp)):
            assert np.array_equal(host(got), want), where  # row pos written, no other touched
        rows = np.stack((ref.dequant_kv4(rk4[:, self.pos], rkp[:, self.pos]),
                         ref.dequant_kv4(rv4[:, self.pos], rvp[:, self.pos])))
        near(host(self.row), rows, ref.U * 2 * np.abs(rows).max(-1, keepdims=True) + 0 * rows, where)


ATTN = [(32, 8, 32, 0), (32, 8, 300, 1), (32, 8, 300, 15), (32, 8, 300, 16), (32, 8, 300, 31), (32, 8, 300, 32),
        (32, 8, 300, 33), (32, 8, 300, 211), (32, 8, 300, 299), (1, 1, 5, 4), (2, 1, 130, 127), (8, 1, 1100, 1099),
        (16, 2, 1100, 1000), (3, 3, 700, 515), (20, 5, 700, 640), (40, 40, 70, 66), (6, 3, 97, 96), (32, 8, 2048, 1279),
        (161, 161, 40, 38), (24, 3, 9000, 8191)]


@pytest.mark.parametrize("n_q,n_kv,max_pos,pos", ATTN)
def test_attention_kv4(ads, n_q, n_kv, max_pos, pos):
    import torch
    a = Attn(ads, n_q, n_kv, max_pos, pos)
    a.call()
    a.check()
    first = a.out.clone()
    a.out.fill_(np.nan)
    a.call()  # the row is rewritten as it was; the workspace is ready again
    assert torch.equal(first, a.out)
    a.check()


def test_attention_kv4_long(ads):
    """Past the context's own limit of 65536 positions, most of them in one head."""
    a = Attn(ads, 4, 1, 70001, 70000)
    a.call()
    a.check()


@pytest.mark.parametrize("pos", [40, 3000, 60000])
def test_attention_kv4_is_as_exact_as_fp32_on_the_values(ads, pos):
    """The 2-norm of the error stays within that of the formula evaluated in fp32 on
    the dequantised cache (numpy, which adds pairwise), also where the values of
    many positions cancel to a small result."""
    a = Attn(ads, 4, 1, pos + 1, pos)
    a.call()
    k4, kp, v4, vp, want, _ = ref.attention_kv4(a.qkv, a.qn, a.kn, a.k4, a.kp, a.v4, a.vp, 4, 1, pos)
    q = ref.norm_rope(a.qkv.astype(np.float64).reshape(-1, D)[:4], a.qn, pos, 1e-6, 1e6).astype(np.float32)
    k = ref.dequant_kv4(k4[0], kp[0]).astype(np.float32)
    v = ref.dequant_kv4(v4[0], vp[0]).astype(np.float32)
    z = q @ k.T / np.float32(np.sqrt(D))
    p = np.exp(z - z.max(-1, keepdims=True))
    plain = (p[:, :, None] * v[None]).sum(1) / p.sum(-1, keepdims=True)
    err = lambda x: np.linalg.norm(x.astype(np.float64).ravel() - want) / np.linalg.norm(want)
    assert err(host(a.out)) <= 2 * err(plain) + ref.U


def test_attention_kv4_far_offsets(ads):
    """Heads whose rows lie past 2^32 bytes: only the rows read are filled."""
    import torch
    n_kv, max_pos, pos = 66, 1 << 20, 40
    small = Attn(ads, n_kv, n_kv, pos + 1, pos)
    k4 = torch.empty((n_kv, max_pos, 64), dtype=torch.uint8, device="cuda")
    v4 = torch.empty_like(k4)
    kp = torch.empty((n_kv, max_pos, 2, 2), dtype=torch.int16, device="cuda")
    vp = torch.empty_like(kp)
    for big, part in zip((k4, v4, kp, vp), small.d[3:]):
        big[:, :pos + 1] = part
    assert k4.numel() > 1 << 32
    qkv, qn, kn = small.d[:3]
    ads.attention_decode_kv4(qkv, qn, kn, k4, v4, kp, vp, small.out, n_kv, n_kv, pos, small.ws, kv_row=small.row)
    small.d[3:] = [t[:, :pos + 1].contiguous() for t in (k4, v4, kp, vp)]
    small.check()


@pytest.mark.parametrize("pos", [20, 700])
def test_attention_kv4_wide_ranges(ads, pos):
    """Value rows from 1e-12 to 1e12, growing and shrinking along the cache, and
    keys strong enough that one position takes almost all the weight."""
    n_kv, G = 2, 4
    rng = np.random.default_rng(3)
    k = synth.normal_f32(1, 70, (n_kv, pos + 1, D))
    k[0] *= 20.0
    v = synth.normal_f32(1, 71, (n_kv, pos + 1, D))
    v *= 10.0 ** rng.uniform(-12, 12, (n_kv, pos + 1, 1))
    v[:, :, 64:] *= 1e-6
    k4, kp = ref.quant_kv4(ref.bf16_bits(k.astype(np.float32)))
    v4, vp = ref.quant_kv4(ref.bf16_bits(v.astype(np.float32)))
    a = Attn(ads, n_kv * G, n_kv, pos + 1, pos, arrays=(k4, kp, v4, vp))
    a.call()
    a.check()


def test_attention_kv4_constant_rows(ads):
    """Halves of scale 0 (all channels equal) in the cache and in the new row."""
    k4, kp, v4, vp = cache(2, 60, 80)
    kp[0, :, :, 0] = 0
    vp[:, ::2, :, 0] = 0
    a = Attn(ads, 8, 2, 60, 59, arrays=(k4, kp, v4, vp))
    a.qkv[(8 + 2) * D:] = 2.5
    a.d[0] = dev(a.qkv)
    a.call()
    a.check()


def test_attention_kv4_nan_row_reaches_its_head_only(ads):
    import torch
    k4, kp, v4, vp = cache(3, 400, 81)
    kp[1, 250, 0] = 0x7FFF
    a = Attn(ads, 6, 3, 400, 399, arrays=(k4, kp, v4, vp))
    a.call()
    o = a.out.view(3, 2, D)
    assert torch.isnan(o[1]).all() and torch.isfinite(o[0]).all() and torch.isfinite(o[2]).all()


def test_attention_kv4_streams_and_graphs(ads):
    """Two captured graphs, each with its workspace, replayed at once on two
    streams, and eager calls of other shapes over one workspace in between."""
    import torch
    a, b = Attn(ads, 32, 8, 1500, 1400, seed=90), Attn(ads, 16, 2, 3000, 2900, seed=95)
    for x in (a, b):
        x.call()
    torch.cuda.synchronize()
    streams, graphs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for x, s in zip((a, b), streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            x.call(stream=s.cuda_stream)
        graphs.append(g)
        x.out.fill_(np.nan)
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    a.check("graph a")
    b.check("graph b")
    shared = torch.zeros(ads.kv4_workspace_bytes(64, 8), dtype=torch.uint8, device="cuda")
    for n_q, n_kv, pos in ((64, 8, 500), (8, 1, 1000), (32, 8, 3), (10, 5, 777), (64, 8, 500)):
        if ads.kv4_workspace_bytes(n_q, n_kv) <= shared.numel():
            c = Attn(ads, n_q, n_kv, pos + 1, pos)
            c.call(ws=shared)
            c.check("shared workspace")


# Cached positions at which the way a head's cache is divided changes (one block, a
# cluster of blocks of two to sixteen, blocks joined through the workspace), for
# each number of queries a head, with shares of the channels that do not come
# out even.
DIVIDED = [(32, 8, 192), (32, 8, 193), (32, 8, 2047), (32, 8, 6144), (32, 8, 6145), (4, 1, 8192), (4, 1, 8193),
           (8, 1, 12288), (8, 1, 12289), (16, 2, 2900), (2, 2, 3900), (2, 2, 8300), (12, 6, 1800), (6, 3, 9100),
           (16, 16, 1000), (33, 33, 700), (9, 9, 5000), (160, 40, 900),
           # eight queries a head: two heads of four, or one of eight
           (8, 1, 0), (24, 3, 31), (16, 2, 200), (32, 4, 9728), (32, 4, 19500), (40, 5, 2000), (40, 5, 4100),
           (128, 16, 900), (128, 16, 1800), (800, 100, 70)]


@pytest.mark.parametrize("n_q,n_kv,pos", DIVIDED)
def test_attention_kv4_however_a_head_is_divided(ads, n_q, n_kv, pos):
    import torch
    a = Attn(ads, n_q, n_kv, pos + 3, pos)
    a.call()
    a.check()
    first = a.out.clone()
    for _ in range(3):
        a.out.fill_(np.nan)
        a.call()
        assert torch.equal(first, a.out)


def test_attention_kv4_long_caches_in_two_graphs(ads):
    """Calls that join through their workspaces, two captured and replayed at once on
    two streams, then a short and a long one in turn over one workspace."""
    import torch
    pair = Attn(ads, 32, 8, 9001, 9000, seed=91), Attn(ads, 16, 2, 14501, 14500, seed=96)
    for x in pair:
        x.call()
    torch.cuda.synchronize()
    streams, graphs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for x, s in zip(pair, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            x.call(stream=s.cuda_stream)
            x.call(stream=s.cuda_stream)
        graphs.append(g)
        x.out.fill_(np.nan)
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for x in pair:
        x.check("graph")
    shared = torch.zeros(ads.kv4_workspace_bytes(32, 8), dtype=torch.uint8, device="cuda")
    for n_q, n_kv, pos in ((32, 8, 500), (4, 1, 9000), (32, 8, 7000), (32, 8, 100), (8, 4, 12000)):
        c = Attn(ads, n_q, n_kv, pos + 1, pos)
        c.ws = shared
        c.call()
        c.check("shared workspace")


# ---- a decoder layer of them ---------------------------------------------------------------

def test_layer_of_four_bit_operators(ads):
    """One decoder layer, W4 weights and a 4-bit cache, five positions through
    it back to back on one stream and a captured last one, then the head and
    the codes' log probabilities: every operator checked from the very inputs
    that it got."""
    import torch
    H, I, n_q, n_kv, V, ncb, eps = 512, 1152, 8, 2, 66, 4, 1e-6
    A = n_q * D
    shapes = dict(qkv=(A + 2 * n_kv * D, H), o=(H, A), gu=(2 * I, H), down=(H, I), head=(ncb * V, H))
    W = {n: weights(*sh, 300 + i) for i, (n, sh) in enumerate(shapes.items())}
    dW = {n: (dev(b), dev(s)) for n, (b, s) in W.items()}
    gains = {n: synth.normal_bf16(3, 310 + i, (H if i < 3 else D,), std=0.02, mean=1.0)
             for i, n in enumerate(("ln_in", "ln_post", "final", "qn", "kn"))}
    dG = {n: dev(g) for n, g in gains.items()}
    P, max_pos = 5, 21
    kb = synth.normal_bf16(1, 320, (n_kv, max_pos, D))
    vb = synth.normal_bf16(1, 321, (n_kv, max_pos, D))
    k4 = torch.zeros((n_kv, max_pos, 64), dtype=torch.uint8, device="cuda")
    v4, kp = k4.clone(), torch.zeros((n_kv, max_pos, 2, 2), dtype=torch.int16, device="cuda")
    vp = kp.clone()
    p0 = 16
    ads.quantize_kv4(dev(kb), dev(vb), k4, v4, kp, vp, 0, p0)
    ws = torch.zeros(ads.kv4_workspace_bytes(n_q, n_kv), dtype=torch.uint8, device="cuda")
    x = synth.normal_f32(5, 330, (P, H))
    codes = np.array([[3, 9, 65, 0]], np.int32)
    dcodes = dev(codes)
    f = lambda n: torch.empty((1, n), device="cuda")
    steps = []

    def step(i, s, stream=None):
        pos = p0 + i
        ads.gemv_w4(s["h0"], *dW["qkv"], s["qkv"], gamma_dev=dG["ln_in"], eps=eps, stream=stream)
        ads.attention_decode_kv4(s["qkv"].view(-1), dG["qn"], dG["kn"], k4, v4, kp, vp, s["a"].view(-1), n_q, n_kv,
                                 pos, ws, eps=eps, stream=stream)
        ads.gemv_w4(s["a"], *dW["o"], s["h1"], epi=1, resid_dev=s["h0"], stream=stream)
        ads.gemv_w4(s["h1"], *dW["gu"], s["m"], epi=2, gamma_dev=dG["ln_post"], eps=eps, stream=stream)
        ads.gemv_w4(s["m"], *dW["down"], s["h2"], epi=1, resid_dev=s["h1"], stream=stream)
        ads.gemv_w4(s["h2"], *dW["head"], s["z"], gamma_dev=dG["final"], eps=eps, stream=stream)
        s["score"] = ads.code_logprobs(s["z"], dcodes, V, top=3, stream=stream)

    for i in range(P):
        s = dict(h0=dev(x[i:i + 1]), qkv=f(shapes["qkv"][0]), a=f(A), h1=f(H), m=f(I), h2=f(H), z=f(ncb * V))
        steps.append(s)
        if i < P - 1:
            step(i, s)
        else:
            torch.cuda.synchronize()
            st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                step(i, s, st.cuda_stream)
            g.replay()
            g.replay()
    torch.cuda.synchronize()
    rk4, rkp = ref.quant_kv4(kb)
    rv4, rvp = ref.quant_kv4(vb)
    for i, s in enumerate(steps):
        h = {n: host(t) for n, t in s.items() if n != "score"}
        near(h["qkv"], *ref.gemv_w4(h["h0"], *W["qkv"], gamma_bits=gains["ln_in"], eps=eps), f"qkv {i}")
        rk4, rkp, rv4, rvp, out, tol = ref.attention_kv4(h["qkv"], gains["qn"], gains["kn"], rk4, rkp, rv4, rvp, n_q,
                                                         n_kv, p0 + i, eps)
        near(h["a"][0], out, tol, f"attention {i}")
        near(h["h1"], *ref.gemv_w4(h["a"], *W["o"], 1, h["h0"]), f"o {i}")
        near(h["m"], *ref.gemv_w4(h["h1"], *W["gu"], 2, gamma_bits=gains["ln_post"], eps=eps), f"gate/up {i}")
        near(h["h2"], *ref.gemv_w4(h["m"], *W["down"], 1, h["h1"]), f"down {i}")
        near(h["z"], *ref.gemv_w4(h["h2"], *W["head"], gamma_bits=gains["final"], eps=eps), f"head {i}")
        lp, ent, at, at_lp, t_lp, t_ent, t_at = ref.code_logprobs(h["z"].reshape(1, ncb, V), codes, 3, 1.0)
        got = [host(t) for t in s["score"]]
        near(got[0], lp, t_lp, f"logprob {i}")
        near(got[1], ent, t_ent, f"entropy {i}")
        assert np.array_equal(got[2], at)
        near(got[3], at_lp, t_at, f"alternatives {i}")
    assert np.array_equal(host(k4)[:, :p0 + P], rk4[:, :p0 + P]) and np.array_equal(host(kp)[:, :p0 + P], rkp[:, :p0 + P])
    assert np.array_equal(host(v4)[:, :p0 + P], rv4[:, :p0 + P]) and np.array_equal(host(vp)[:, :p0 + P], rvp[:, :p0 + P])


def test_prefix_parked_in_four_bits_and_restored(ads):
    """A context's bf16 prefix moved into a 4-bit cache and back through
    tts_get_kv / tts_set_kv: the context holds the 4-bit values and decodes."""
    import torch
    from helpers import reduced_dims, to_binding_dims
    d = reduced_dims()
    dec = ads.Decoder(to_binding_dims(d), ads.DeviceWeights(synth.make_weights(d)), 40)
    dec.prefill(synth.delayed_prompt_codes(11))
    k, v = dec.get_kv(0, 11)
    kd, vd = dev(k), dev(v)
    for l in range(d.n_layers):
        k4 = torch.zeros((d.n_kv, 11, 64), dtype=torch.uint8, device="cuda")
        v4, kp = k4.clone(), torch.zeros((d.n_kv, 11, 2, 2), dtype=torch.int16, device="cuda")
        vp = kp.clone()
        ads.quantize_kv4(kd[l], vd[l], k4, v4, kp, vp, 0, 11)
        ads.dequantize_kv4(k4, v4, kp, vp, kd[l], vd[l], 0, 11)
    dec.reset()
    dec.set_kv(kd, vd, 11)
    k2, v2 = dec.get_kv(0, 11)
    for a, b in ((k, k2), (v, v2)):
        assert np.array_equal(b, ref.bf16_bits(ref.dequant_kv4(*ref.quant_kv4(a)).astype(np.float32)))
    dec.decode_step(synth.random_codes(1)[0])
    assert np.isfinite(dec.get_logits()).all() and dec.state()[0] == 12
    dec.close()
