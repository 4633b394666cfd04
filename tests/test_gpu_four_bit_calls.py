"""Calls of the 4-bit operators and the code scoring on the GPU: empty batches,
tensors that the library cannot read, streams, captured first calls."""
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


@pytest.mark.parametrize("V,top", [(1026, 5), (1026, 0), (40000, 3)])
def test_code_logprobs_of_an_empty_batch(ads, V, top):
    import torch
    lp, ent, at, at_lp = ads.code_logprobs(torch.empty((0, 2 * V), device="cuda"),
                                           torch.empty((0, 2), dtype=torch.int32, device="cuda"), V, top=top)
    assert lp.shape == ent.shape == (0, 2) and at.shape == at_lp.shape == (0, 2, top)
    assert at.dtype == torch.int32 and lp.dtype == torch.float32


def test_tensors_of_another_type_size_or_layout_are_refused(ads):
    """One change each, on tensors of the GPU that is used; nothing is launched."""
    import torch
    x, w4 = torch.randn((2, 256), device="cuda"), torch.zeros((6, 128), dtype=torch.uint8, device="cuda")
    s, y = torch.ones((6, 2), dtype=torch.bfloat16, device="cuda"), torch.full((2, 6), 7.0, device="cuda")
    z, codes = torch.randn((3, 40), device="cuda"), torch.zeros((3, 4), dtype=torch.int32, device="cuda")
    gamma = torch.ones(256, dtype=torch.float16, device="cuda")
    bad = [lambda: ads.gemv_w4(x.half(), w4, s, y), lambda: ads.gemv_w4(x, w4, s.half(), y),
           lambda: ads.gemv_w4(x, w4, s, y, gamma_dev=gamma), lambda: ads.gemv_w4(x, w4[:5], s, y),
           lambda: ads.gemv_w4(x.t().contiguous().t(), w4, s, y), lambda: ads.gemv_w4(x, w4, s, y.cpu()),
           lambda: ads.code_logprobs(z, codes.float(), 10), lambda: ads.code_logprobs(z, codes.t().contiguous().t(), 10),
           lambda: ads.code_logprobs(z[:2], codes, 10), lambda: ads.code_logprobs(z[:, ::2], codes[:, :2].contiguous(), 10),
           lambda: ads.quantize_w4_weight(torch.zeros((4, 256), dtype=torch.float16, device="cuda"))]
    for call in bad:
        with pytest.raises(ads.TtsError) as e:
            call()
        assert e.value.status == -1
    assert (y == 7.0).all()
    ads.gemv_w4(x, w4, s, y)
    assert ads.code_logprobs(z, codes, 10, top=2)[2].dtype == torch.int32


def stream_of(t):
    """The stream whose memory pool tensor t is of."""
    import torch
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's")


def test_results_belong_to_the_stream_they_are_written_on(ads):
    """The allocator hands memory on in the order of one stream: results made on
    torch's current stream and written on another could be in use there still."""
    import torch
    z, codes = torch.randn((4, 8 * 1026), device="cuda"), torch.zeros((4, 8), dtype=torch.int32, device="cuda")
    w = torch.randn((64, 512), device="cuda").bfloat16()
    want, packed = ads.code_logprobs(z, codes, 1026, top=5), ads.quantize_w4_weight(w)
    torch.cuda.synchronize()
    current, launch = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(current):
        for stream in (None, launch.cuda_stream, current.cuda_stream):
            got = ads.code_logprobs(z, codes, 1026, top=5, stream=stream)
            q = ads.quantize_w4_weight(w, stream=stream)
            assert [stream_of(t) for t in (*got, *q)] == [stream or 0] * 6
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip((*got, *q), (*want, *packed)))
    assert torch.cuda.current_stream() == torch.cuda.default_stream()


def test_results_written_beside_a_busy_current_stream(ads):
    """Memory that the current stream has freed, with its last writes to come, is not
    handed to results written on another stream."""
    import torch
    z, codes = torch.randn((256, 8 * 1026), device="cuda"), torch.zeros((256, 8), dtype=torch.int32, device="cuda")
    want = ads.code_logprobs(z, codes, 1026, top=5)
    torch.cuda.synchronize()
    current, launch = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(current):
        mine = [torch.empty_like(t) for t in want]
        torch.cuda._sleep(20_000_000)  # about 10 ms
        for t in mine:
            t.fill_(3)
        del mine, t
        got = ads.code_logprobs(z, codes, 1026, top=5, stream=launch.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def weights(N, K, seed, std=0.02):
    return ref.quant_w4(synth.normal_bf16(0, seed, (N, K), std=std))


def near(got, want, tol):
    err = np.abs(got.astype(np.float64) - want)
    assert np.isfinite(got).all() and (err <= tol).all(), (err / tol).max()


def dev(a):
    import torch
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).cuda()


@pytest.mark.parametrize("M,N,K,epi", [(1, 40, 256, 0), (2, 40, 512, 1), (4, 33, 1280, 0), (7, 64, 384, 0), (8, 2560, 9728, 0)])
def test_gemv_w4_activations_up_to_the_largest_number(ads, M, N, K, epi):
    """Activations next to fp32's end under weights that bring the products back:
    neither a pair's combination nor a group's sum before its scale overflows."""
    import torch
    b, s = weights(N, K, 41, std=1e-6)
    rng = np.random.default_rng(K)
    x = (rng.uniform(2.5e38, 3.4e38, (M, K)) * rng.choice([-1.0, 1.0], (M, K))).astype(np.float32)
    x[-1, 128:] *= np.float32(1e-30)
    resid = (rng.standard_normal((M, N)) * 1e32).astype(np.float32) if epi else None
    want, tol = ref.gemv_w4(x, b, s, epi, resid)
    y = torch.empty((M, N), device="cuda")
    ads.gemv_w4(dev(x), dev(b), dev(s), y, epi, None if resid is None else dev(resid))
    near(y.cpu().numpy(), want, tol)


@pytest.mark.parametrize("M", [1, 2, 4, 8])
@pytest.mark.parametrize("N,K,epi,norm", [(40, 256, 0, False), (40, 256, 2, True), (2560, 9728, 1, False), (17, 12288, 0, True)])
def test_gemv_w4_a_vector_with_a_non_finite_activation_is_nan(ads, M, N, K, epi, norm):
    """All of its results, whatever the weights there, and none of the others'."""
    import torch
    b, s = weights(2 * N if epi == 2 else N, K, 43)
    gamma = synth.normal_bf16(3, 44, (K,), std=0.02, mean=1.0) if norm else None
    resid = synth.normal_f32(5, 45, (M, N)) if epi == 1 else None
    clean = synth.normal_f32(5, 46, (M, K))
    want, tol = ref.gemv_w4(clean, b, s, epi, resid, gamma)
    for at, (bad, k) in enumerate([(np.nan, 0), (np.inf, K - 1), (-np.inf, K // 2), (np.nan, 129 % K)]):
        x, m = clean.copy(), at % M
        x[m, k] = bad
        y = torch.zeros((M, N), device="cuda")
        ads.gemv_w4(dev(x), dev(b), dev(s), y, epi, None if resid is None else dev(resid), None if gamma is None else dev(gamma))
        y = y.cpu().numpy()
        assert np.isnan(y[m]).all(), (bad, k)
        others = np.arange(M) != m
        near(y[others], want[others], tol[others]) if others.any() else None


def test_a_late_copy_is_waited_for_a_second_time(tmp_path):
    """A kernel that was off the GPU for longer than a wait's limit finds its
    copies at the second wait (here an arrival 1.3 s late; limits are 1 s)."""
    import os
    import shutil
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = str(tmp_path / "check")
    subprocess.run([shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc", "-std=c++17", "-O2", "-gencode",
                    "arch=compute_103a,code=sm_103a", "--expt-relaxed-constexpr", "-I", os.path.join(root, "include"), "-I",
                    os.path.join(root, "ar_decode_step_gb300", "csrc"),
                    os.path.join(root, "tests", "host", "mbar_arrived_check.cu"), "-o", exe],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.parametrize("V", [40, 1026, 9001, 70000])
@pytest.mark.parametrize("T,scale", [(1e30, 1e30), (1e37, 3e37), (3e38, 1e38), (1e-37, 1e-37), (2.0 ** -126, 2.0 ** -126)])
def test_code_logprobs_at_extreme_temperatures(ads, V, T, scale):
    """Logits and temperatures at both ends of fp32, whose quotients are ordinary:
    neither a difference of two logits nor the entropy's sum overflows."""
    import torch
    T = float(np.float32(T))
    z = np.clip(synth.normal_f32(7, V, (5, 2, V), std=2.5).astype(np.float64) * scale, -3.4e38, 3.4e38).astype(np.float32)
    z[1, 0, ::5] = -np.inf
    z[2, 0, :2] = np.float32(3.4e38) * np.float32([1, -1]) if scale > 1 else z[2, 0, :2]
    codes = np.random.default_rng(V).integers(0, V, (5, 2)).astype(np.int32)
    codes[2, 0] = 1
    lp, ent, at, at_lp, t_lp, t_ent, t_at = ref.code_logprobs(z, codes, 7, T)
    got = [t.cpu().numpy() for t in ads.code_logprobs(dev(z.reshape(5, -1)), dev(codes), V, top=7, temperature=T)]
    for g, w, t in ((got[0], lp, t_lp), (got[1], ent, t_ent), (got[3], at_lp, t_at)):
        fine = np.isfinite(w)
        assert np.array_equal(g[~fine], w[~fine]) and (np.abs(g[fine] - w[fine]) <= t[fine]).all(), \
            (np.abs(g[fine] - w[fine]) / t[fine]).max()
    assert np.array_equal(got[2], at)


FIRST = """
import sys
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import numpy as np, torch
import ar_decode_step_gb300 as ads
ads.load()
g = torch.Generator(device="cuda").manual_seed(1)
f = lambda *s: torch.randn(s, generator=g, device="cuda")
u = lambda *s: torch.randint(0, 256, s, generator=g, device="cuda", dtype=torch.uint8)
b = lambda *s: f(*s).bfloat16()
n_kv, n = 2, 9001
cache = [u(n_kv, n, 64), u(n_kv, n, 64), b(n_kv, n, 2, 2).abs(), b(n_kv, n, 2, 2)]
rows, back = [b(n_kv, 40, 128) for _ in range(2)], [b(n_kv, 40, 128) for _ in range(2)]
ws = torch.zeros(ads.kv4_workspace_bytes(16, n_kv), dtype=torch.uint8, device="cuda")
qkv, gains, outs = f(20 * 128), [b(128), b(128)], [f(16 * 128) for _ in range(3)]
x, w, s, y = f(8, 9728), u(2560, 4864), b(2560, 76).abs(), f(8, 2560)
w2, s2, y2 = u(2 * 700, 128), b(2 * 700, 2).abs(), f(1, 700)
z, codes = f(3, 8 * 1026), torch.randint(0, 1026, (3, 8), generator=g, device="cuda", dtype=torch.int32)
zl, cl = f(2, 70000), torch.randint(0, 70000, (2, 1), generator=g, device="cuda", dtype=torch.int32)
wb = b(32, 256)


def every(stream):
    k4, v4, kp, vp = cache
    ads.quantize_kv4(*rows, k4, v4, kp, vp, 0, 40, stream=stream)
    for o, pos in zip(outs, (20, 1000, 9000)):
        ads.attention_decode_kv4(qkv, *gains, k4, v4, kp, vp, o, 16, n_kv, pos, ws, stream=stream)
    ads.dequantize_kv4(k4, v4, kp, vp, *back, 0, 40, stream=stream)
    ads.gemv_w4(x, w, s, y, stream=stream)
    ads.gemv_w4(x[:1, :256].contiguous() if stream is None else x1, w2, s2, y2, epi=2, stream=stream)
    return [*ads.code_logprobs(z, codes, 1026, top=5, stream=stream), *ads.code_logprobs(zl, cl, 70000, top=20, stream=stream),
            *ads.quantize_w4_weight(wb, stream=stream), *outs, *back, y, y2]


x1 = x[:1, :256].contiguous()
torch.cuda.synchronize()
side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=side):
    got = every(side.cuda_stream)
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in got]
want = every(None)
torch.cuda.synchronize()
assert all(torch.equal(p, q) for p, q in zip(got, want)), [torch.equal(p, q) for p, q in zip(got, want)]
assert all(torch.isfinite(t.float()).all() for t in want)
print("same", len(want))
"""


def test_first_calls_of_a_process_inside_a_capture():
    """What a call prepares once per device (limits, room for clusters, the module
    itself) may be prepared while a stream is being captured."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=root)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr[-2000:]


def test_calls_from_two_threads(ads):
    """Each with its stream, tensors and workspace: the answers are those of one after the other."""
    import threading
    import torch
    n_q, n_kv, n = 16, 2, 5001
    made = []
    for i in range(2):
        k4 = torch.randint(0, 256, (n_kv, n, 64), device="cuda", dtype=torch.uint8)
        par = torch.rand((n_kv, n, 2, 2), device="cuda").bfloat16()
        made.append(dict(k4=k4, v4=k4.flip(1).contiguous(), k_par=par, v_par=par.flip(1).contiguous(),
                         qkv=torch.randn((n_q + 2 * n_kv) * D, device="cuda"), q_norm=torch.ones(D, device="cuda").bfloat16(),
                         k_norm=torch.ones(D, device="cuda").bfloat16(), out=torch.zeros(n_q * D, device="cuda"), n_q=n_q,
                         n_kv=n_kv, pos=n - 1 - 2000 * i,
                         workspace=torch.zeros(ads.kv4_workspace_bytes(n_q, n_kv), dtype=torch.uint8, device="cuda")))
    x, w = torch.randn((4, 2560), device="cuda"), torch.randint(0, 256, (256, 1280), device="cuda", dtype=torch.uint8)
    s = torch.rand((256, 20), device="cuda").bfloat16()
    want = []
    for m in made:
        ads.attention_decode_kv4(**m)
        y = torch.zeros((4, 256), device="cuda")
        ads.gemv_w4(x, w, s, y)
        torch.cuda.synchronize()
        want.append((m["out"].clone(), y))
    wrong = []

    def work(i):
        stream = torch.cuda.Stream()
        y = torch.zeros((4, 256), device="cuda")
        torch.cuda.synchronize()
        for _ in range(200):
            ads.attention_decode_kv4(**made[i], stream=stream.cuda_stream)
            ads.gemv_w4(x, w, s, y, stream=stream.cuda_stream)
        stream.synchronize()
        if not (torch.equal(made[i]["out"], want[i][0]) and torch.equal(y, want[i][1])):
            wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not wrong


@pytest.mark.parametrize("M", [3, 4])
@pytest.mark.parametrize("N,K,norm", [(9728, 2560, True), (16384, 2560, False), (6144, 2560, True), (4096, 2048, True), (500, 12288, False), (1152, 512, True)])
def test_gemv_w4_gate_up_of_four_vectors_in_both_forms(ads, M, N, K, norm):
    """The sums in a place of their own, or where a warp's first activations were."""
    import torch
    b, s = weights(2 * N, K, 47)
    x = synth.normal_f32(5, 48 + M, (M, K), std=1.5)
    gamma = synth.normal_bf16(3, 49, (K,), std=0.02, mean=1.0) if norm else None
    want, tol = ref.gemv_w4(x, b, s, 2, None, gamma)
    pad = torch.full((M * N + 64,), 7.25, device="cuda")
    y = pad[32:32 + M * N].view(M, N)
    args = (dev(x), dev(b), dev(s), y, 2, None, None if gamma is None else dev(gamma))
    ads.gemv_w4(*args)
    near(y.cpu().numpy(), want, tol)
    first = y.clone()
    ads.gemv_w4(*args)
    assert torch.equal(first, y) and (pad[:32] == 7.25).all() and (pad[32 + M * N:] == 7.25).all()
