"""The 4-bit operators' and the code scoring's refusals: every bad argument is
found on the host before any device call (no GPU needed; the pointers are
aligned stand-ins, never dereferenced)."""
import ctypes

import numpy as np
import pytest

import four_bit_ref as ref

ARG, FULL, STATE = -1, -3, -6
A = [0x1000000 * (i + 1) for i in range(16)]  # far apart, 16-byte aligned


@pytest.fixture(scope="module")
def lib():
    import ar_decode_step_gb300.build as b
    b.build()
    import ar_decode_step_gb300 as m
    return m.load()


def refuse(f, good, bad, want=ARG):
    """f(**good with one change) returns `want` for every change in `bad`."""
    for change in bad:
        args = dict(good)
        args.update(change)
        assert f(*args.values()) == want, change


def test_quantize_w4_refusals(lib):
    good = dict(W=A[0], N=16, K=256, W4=A[1], s=A[2], stream=None)
    refuse(lib.tts_quantize_w4_weight, good,
           [dict(W=None), dict(W4=None), dict(s=None), dict(N=0), dict(N=-4), dict(K=0), dict(K=64), dict(K=200),
            dict(W=A[0] + 8), dict(W4=A[1] + 4), dict(s=A[2] + 2)])


def test_gemv_w4_refusals(lib):
    good = dict(x=A[0], W4=A[1], s=A[2], resid=None, gamma=None, y=A[3], M=1, N=48, K=256, epi=0, eps=1e-6,
                stream=None)
    refuse(lib.tts_gemv_w4, good,
           [dict(x=None), dict(W4=None), dict(s=None), dict(y=None), dict(M=0), dict(M=9), dict(N=0),
            dict(N=(1 << 24) + 1), dict(K=0), dict(K=192), dict(K=12416), dict(epi=3), dict(epi=-1),
            dict(epi=1), dict(resid=A[4]), dict(epi=2, resid=A[4]), dict(gamma=A[5], eps=-1.0),
            dict(gamma=A[5], eps=float("nan")), dict(x=A[0] + 4), dict(W4=A[1] + 8), dict(s=A[2] + 2),
            dict(y=A[3] + 2), dict(gamma=A[5] + 8), dict(epi=1, resid=A[4] + 2),
            # y over an input that other blocks still read
            dict(y=A[0]), dict(y=A[0] + 1020), dict(y=A[1] + 48 * 128 - 4), dict(y=A[2] + 48 * 4 - 4),
            dict(gamma=A[5], y=A[5] + 508), dict(epi=1, resid=A[3] + 4)])


KV = dict(k=A[0], v=A[1], n_kv=2, p0=0, p1=8, stride=16, k4=A[2], v4=A[3], k_par=A[4], v_par=A[5], max_pos=16,
          stream=None)


def test_quantize_kv4_refusals(lib):
    bad = [dict({n: None}) for n in ("k", "v", "k4", "v4", "k_par", "v_par")]
    bad += [dict({n: KV[n] + 8}) for n in ("k", "v", "k4", "v4", "k_par", "v_par")]
    bad += [dict(n_kv=0), dict(p0=-1), dict(p0=9), dict(stride=7), dict(max_pos=0), dict(max_pos=(1 << 20) + 1)]
    refuse(lib.tts_quantize_kv4, KV, bad)
    bad += [dict(k=A[2]), dict(v=A[2] + 2 * 16 * 64 - 16), dict(k4=A[1] + 2 * 16 * 256 - 16), dict(v_par=A[0] + 64)]
    refuse(lib.tts_quantize_kv4, KV, bad)
    refuse(lib.tts_quantize_kv4, KV, [dict(p1=17), dict(max_pos=7)], FULL)
    assert lib.tts_quantize_kv4(*dict(KV, p0=5, p1=5).values()) == 0  # nothing to do


def test_dequantize_kv4_refusals(lib):
    order = ("k4", "v4", "k_par", "v_par", "n_kv", "p0", "p1", "max_pos", "k", "v", "stride", "stream")
    good = {n: KV[n] for n in order}
    bad = [dict({n: None}) for n in ("k", "v", "k4", "v4", "k_par", "v_par")]
    bad += [dict({n: KV[n] + 8}) for n in ("k", "v", "k4", "v4", "k_par", "v_par")]
    bad += [dict(n_kv=-2), dict(p0=-1), dict(p0=9), dict(stride=7), dict(max_pos=0)]
    refuse(lib.tts_dequantize_kv4, good, bad)
    refuse(lib.tts_dequantize_kv4, good, [dict(p1=17)], FULL)
    assert lib.tts_dequantize_kv4(*dict(good, p0=8).values()) == 0


def test_attention_kv4_refusals(lib):
    import ar_decode_step_gb300 as m
    n = m.kv4_workspace_bytes(32, 8)
    good = dict(qkv=A[0], qn=A[1], kn=A[2], k4=A[3], v4=A[4], k_par=A[5], v_par=A[6], out=A[7], kv_row=None, n_q=32,
                n_kv=8, max_pos=64, pos=3, eps=1e-6, theta=1e6, ws=A[8], ws_bytes=n, stream=None)
    ptrs = ("qkv", "qn", "kn", "k4", "v4", "k_par", "v_par", "out", "ws")
    bad = [dict({p: None}) for p in ptrs] + [dict({p: good[p] + 8}) for p in ptrs] + [dict(kv_row=A[9] + 4)]
    bad += [dict(n_q=24), dict(n_q=8, n_kv=3), dict(n_q=0), dict(n_kv=0), dict(n_q=128), dict(n_q=8192, n_kv=8192),
            dict(max_pos=0), dict(max_pos=(1 << 20) + 1), dict(pos=-1), dict(eps=-1e-6), dict(theta=0.0),
            dict(theta=float("inf")), dict(theta=float("nan")), dict(ws_bytes=n - 1), dict(ws_bytes=0)]
    refuse(lib.tts_attention_decode_kv4, good, bad)
    # written over something that another block reads, or twice
    row = 128 * 4
    bad += [dict(out=A[0]), dict(out=A[0] + 48 * row - 16), dict(kv_row=A[0] + 16), dict(kv_row=A[7]),
            dict(out=A[3] + 8 * 64 * 64 - 16), dict(v4=A[3]), dict(v_par=A[5] + 16), dict(ws=A[7] + 32 * row - 16),
            dict(out=A[8] + n - 16), dict(out=A[2])]
    refuse(lib.tts_attention_decode_kv4, good, bad)
    refuse(lib.tts_attention_decode_kv4, good, [dict(pos=64), dict(pos=1 << 20)], FULL)


def test_workspace_size(lib):
    import ar_decode_step_gb300 as m
    n = ctypes.c_size_t()
    assert lib.tts_attention_kv4_workspace(32, 8, None) == ARG
    for n_q, n_kv in ((24, 8), (0, 1), (8, 0), (48, 3)):
        assert lib.tts_attention_kv4_workspace(n_q, n_kv, ctypes.byref(n)) == ARG
    # what callers may allocate without asking
    for n_kv in (1, 2, 3, 5, 8, 40, 161, 512):
        for G in (1, 2, 4, 8):
            assert 0 < m.kv4_workspace_bytes(n_kv * G, n_kv) <= 4096 + 4 * n_kv + 520 * n_kv * G * (160 // n_kv + 1)


def test_code_logprobs_refusals(lib):
    good = dict(z=A[0], ld=8208, codes=A[1], rows=4, n_cb=8, V=1026, T=1.0, top=5, lp=A[2], ent=A[3], at=A[4],
                at_lp=A[5], stream=None)
    refuse(lib.tts_code_logprobs, good,
           [dict(z=None), dict(ld=8207), dict(rows=-1), dict(n_cb=0), dict(n_cb=9), dict(V=1), dict(V=(1 << 20) + 1),
            dict(T=0.0), dict(T=-1.0), dict(T=float("inf")), dict(T=float("nan")), dict(T=1e-39), dict(top=-1),
            dict(top=33), dict(V=4, top=5), dict(codes=None), dict(lp=None), dict(at=None), dict(at_lp=None),
            dict(top=0), dict(z=A[0] + 2), dict(codes=A[1] + 1), dict(ent=A[3] + 2)])
    assert lib.tts_code_logprobs(*dict(good, rows=0).values()) == 0


def test_get_logprobs_without_context(lib):
    assert lib.tts_get_logprobs(None, None, 1.0, 0, None, None, None, None) == STATE


def test_binding_refuses_tensors_the_library_cannot_read(lib):
    """Shapes, strides, element sizes and devices are the binding's to check."""
    import torch
    import ar_decode_step_gb300 as m
    x = torch.zeros((1, 256))
    for call in (lambda: m.quantize_w4_weight(torch.zeros((4, 256), dtype=torch.bfloat16)),
                 lambda: m.gemv_w4(x, torch.zeros((4, 128), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.int16),
                                   torch.zeros((1, 4))),
                 lambda: m.code_logprobs(torch.zeros((2, 40)), torch.zeros((2, 4), dtype=torch.int32), 10)):
        with pytest.raises(m.TtsError) as e:
            call()
        assert e.value.status == ARG


# ---- the restatement itself, against values worked out by hand -----------------------

def test_restatement_formats():
    w = np.zeros((1, 256), np.float32)
    w[0, :4] = [7.0, -7.0, 2.5, -1.5]  # scale 1: ties to even
    b, s = ref.quant_w4(ref.bf16_bits(w))
    assert ref.bf16_val(s).tolist() == [[1.0, 0.0]]
    assert [b[0, 0] & 15, b[0, 0] >> 4, b[0, 1] & 15, b[0, 1] >> 4] == [15, 1, 10, 6]
    assert (b[0, 2:] == 0x88).all()
    row = np.zeros(128, np.float32)
    row[:64] = np.arange(64) % 16 - 3  # minimum -3, scale 1
    row[64:] = 5.0                     # constant half: scale 0
    b, p = ref.quant_kv4(ref.bf16_bits(row))
    assert ref.bf16_val(p).tolist() == [[1.0, -3.0], [0.0, 5.0]]
    assert np.array_equal(ref.dequant_kv4(b, p), row.astype(np.float64))
    assert [b[0] & 15, b[0] >> 4, b[8] & 15, b[4]] == [0, 1, 8, 0]
