"""Python binding of the GB300 batch-1 TTS decode-step library (libtts_decode.so).

Argument marshalling only: every step of the decode path runs in the CUDA
kernels behind the C ABI declared in ``include/tts_decode.h``.  PyTorch is used
for device memory and streams.  There is no fallback: importing this package
raises if the CUDA library has not been built, and every call raises
``TtsError`` on a non-zero status.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtts_decode.so")

TTS_BF16 = 0
TTS_FP8 = 1

_STATUS = {0: "ok", -1: "bad argument", -2: "code out of range", -3: "context full",
           -4: "CUDA error", -5: "device error flag set", -6: "not initialised", -7: "unsupported"}


class TtsError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} -> {status} ({_STATUS.get(status, 'unknown')})")
        self.status = status


class tts_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in
                ("n_layers", "hidden", "n_q_heads", "n_kv_heads", "head_dim", "inter",
                 "n_codebooks", "cb_vocab", "max_pos")] + \
               [("rms_eps", ctypes.c_float), ("rope_theta", ctypes.c_float),
                ("precision", ctypes.c_int), ("stream", ctypes.c_void_p), ("options", ctypes.c_int)]


# tts_config.options bits
OPT_SEPARATE_KERNELS = 1
OPT_PREFILL_STEPS = 2


_PP = ctypes.POINTER(ctypes.c_void_p)


class tts_weights(ctypes.Structure):
    _fields_ = [("embed", ctypes.c_void_p), ("head", ctypes.c_void_p), ("final_norm", ctypes.c_void_p)] + \
               [(n, _PP) for n in ("wqkv", "wo", "wgu", "wd", "sqkv", "so", "sgu", "sd",
                                   "ln_in", "ln_post", "q_norm", "k_norm")]


# Every symbol include/tts_decode.h declares, with its ctypes signature.
_I, _VP, _F = ctypes.c_int, ctypes.c_void_p, ctypes.c_float
SIGNATURES = {
    "tts_init": (_I, [ctypes.POINTER(tts_config), ctypes.POINTER(tts_weights), ctypes.POINTER(_VP)]),
    "tts_shutdown": (_I, [_VP]),
    "tts_reset": (_I, [_VP]),
    "tts_prefill": (_I, [_VP, _VP, _I]),
    "tts_decode_step": (_I, [_VP, _VP, _VP]),
    "tts_decode_steps": (_I, [_VP, _I, _VP]),
    "tts_rewind": (_I, [_VP, _I, _I]),
    "tts_set_input": (_I, [_VP, _VP]),
    "tts_set_sampling": (_I, [_VP, ctypes.c_float, ctypes.c_ulonglong]),
    "tts_decode_until_eoc": (_I, [_VP, _I, _VP, _VP]),
    "tts_prefix_save": (_I, [_VP]),
    "tts_set_fp8_scales": (_I, [_VP, _VP]),
    "tts_fp8_calibrate": (_I, [_VP, _I, _VP]),
    "tts_prefix_restore": (_I, [_VP]),
    "tts_set_kv": (_I, [_VP, _VP, _VP, _I, _I]),
    "tts_get_kv": (_I, [_VP, _VP, _VP, _I, _I]),
    "tts_get_logits": (_I, [_VP, _VP]),
    "tts_get_hidden": (_I, [_VP, _VP]),
    "tts_set_frame": (_I, [_VP, _I, _I]),
    "tts_get_state": (_I, [_VP, _VP, _VP, _VP]),
    "tts_last_steps_ms": (_I, [_VP, _VP]),
    "tts_time_gemv": (_I, [_VP, _I, _I, _VP]),
    "tts_trace_step": (_I, [_VP, _VP, _I, _VP, _VP]),
    "tts_debug_layer_states": (_I, [_VP, _VP, _VP, _VP, _I]),
    "tts_gemm_bf16": (_I, [_VP, _VP, _VP, _I, _I, _I, _I, _I, _VP]),
    "tts_gemm_fp8": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _VP]),
    "tts_gemm_tiled": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _I, _I, _VP]),
    "tts_debug_prefill_states": (_I, [_VP, _VP, _I, _VP, ctypes.c_longlong]),
    "tts_debug_expire_wait": (_I, [_VP]),
    "tts_quantize_fp8_weight": (_I, [_VP, _I, _I, _VP, _VP, _VP]),
    "tts_attention_decode": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _F, _F, _VP]),
    "tts_attention_decode_noalloc": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _F, _F, _VP]),
    "tts_quantize_w4_weight": (_I, [_VP, _I, _I, _VP, _VP, _VP]),
    "tts_gemv_w4": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _F, _VP]),
    "tts_quantize_kv4": (_I, [_VP, _VP, _I, _I, _I, _I, _VP, _VP, _VP, _VP, _I, _VP]),
    "tts_dequantize_kv4": (_I, [_VP, _VP, _VP, _VP, _I, _I, _I, _I, _VP, _VP, _I, _VP]),
    "tts_attention_kv4_workspace": (_I, [_I, _I, ctypes.POINTER(ctypes.c_size_t)]),
    "tts_attention_decode_kv4": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _F, _F, _VP,
                                      ctypes.c_size_t, _VP]),
    "tts_code_logprobs": (_I, [_VP, ctypes.c_longlong, _VP, _I, _I, _I, _F, _I, _VP, _VP, _VP, _VP, _VP]),
    "tts_get_logprobs": (_I, [_VP, _VP, _F, _I, _VP, _VP, _VP, _VP]),
    "tts_status_str": (ctypes.c_char_p, [_I]),
}

_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libtts_decode.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise ImportError(f"{path} is missing: build it with "
                              "`python -m ar_decode_step_gb300.build` (nvcc, sm_103a)")
        L = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _call(name: str, *args) -> None:
    rc = getattr(_lib or load(), name)(*args)
    if rc != 0:
        raise TtsError(name, rc)


def status_str(code: int) -> str:
    return load().tts_status_str(code).decode()


def _ptr(a: np.ndarray) -> int:
    assert a.flags["C_CONTIGUOUS"]
    return a.ctypes.data


# ----------------------------------------------------------------------------
# Device weights (torch is only the allocator here)
# ----------------------------------------------------------------------------

def _torch():
    import torch
    return torch


def _to_dev_u16(a: np.ndarray, device):
    torch = _torch()
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).to(device, non_blocking=False)


def gemm_bf16(a_dev, b_dev, c_dev, epi: int = 0, splits: int = 0, stream=None):
    """C = A . B^T on the tensor cores (see tts_gemm_bf16): a_dev [M][K] and
    b_dev [N][K] (epi 2: [2N][K]) bf16 CUDA tensors; c_dev fp32 [M][N]
    (epi 0, 1) or bf16 [M][N] (epi 2); splits 0 lets the library choose the
    K split, n > 0 fixes it."""
    M, K = a_dev.shape
    N = c_dev.shape[1]
    _call("tts_gemm_bf16", a_dev.data_ptr(), b_dev.data_ptr(), c_dev.data_ptr(), M, N, K, epi, splits, stream)


def gemm_fp8(a8_dev, b8_dev, a_scale_dev, b_scale_dev, c_dev, epi: int = 0, stream=None):
    """tts_gemm_fp8: a8_dev [M][K] and b8_dev [N][K] (epi 2: [2N][K]) uint8
    E4M3 CUDA tensors with fp32 scales [M] and [N] (epi 2: [2N]); c_dev fp32
    [M][N] (epi 0, 1) or bf16 [M][N] (epi 2)."""
    M, K = a8_dev.shape
    N = c_dev.shape[1]
    _call("tts_gemm_fp8", a8_dev.data_ptr(), b8_dev.data_ptr(), a_scale_dev.data_ptr(), b_scale_dev.data_ptr(),
          c_dev.data_ptr(), M, N, K, epi, stream)


def gemm_tiled(a_dev, b_dev, c_dev, epi: int, tile_rows: int, tile_cols: int, splits: int,
               a_scale_dev=None, b_scale_dev=None, stream=None):
    """tts_gemm_tiled: tts_gemm_bf16 (uint8 operands with scales: tts_gemm_fp8)
    with an explicit tile of tile_rows (128 or 256) x tile_cols output
    columns and the K range split over `splits` CTAs."""
    M, K = a_dev.shape
    N = c_dev.shape[1]
    fp8 = a_scale_dev is not None
    _call("tts_gemm_tiled", a_dev.data_ptr(), b_dev.data_ptr(), a_scale_dev.data_ptr() if fp8 else None,
          b_scale_dev.data_ptr() if fp8 else None, c_dev.data_ptr(), M, N, K, epi, 1 if fp8 else 0,
          tile_rows, tile_cols, splits, stream)


def quantize_fp8_weight(w_dev, stream=None):
    """Per-row E4M3 quantisation on the GPU; w_dev: int16 (bf16 bits) [N][K].
    Returns (uint8 [N][K], float32 [N]) device tensors."""
    torch = _torch()
    N, K = w_dev.shape
    q = torch.empty((N, K), dtype=torch.uint8, device=w_dev.device)
    s = torch.empty((N,), dtype=torch.float32, device=w_dev.device)
    _call("tts_quantize_fp8_weight", w_dev.data_ptr(), N, K, q.data_ptr(), s.data_ptr(),
          stream if stream is not None else None)
    return q, s


def attention_decode(qkv, q_norm, k_norm, k_cache, v_cache, out, n_q: int, n_kv: int, pos: int,
                     eps: float = 1e-6, rope_theta: float = 1e6, stream=None) -> None:
    """tts_attention_decode on torch device tensors (fp32 qkv/out, int16 bf16 bits)."""
    max_pos = k_cache.shape[-2]
    _call("tts_attention_decode", qkv.data_ptr(), q_norm.data_ptr(), k_norm.data_ptr(), k_cache.data_ptr(),
          v_cache.data_ptr(), out.data_ptr(), n_q, n_kv, max_pos, pos, eps, rope_theta, stream)


# ----------------------------------------------------------------------------
# 4-bit weights, 4-bit cache, scores of codes
# ----------------------------------------------------------------------------

# The library sees an address of each tensor and nothing else, so the binding
# checks that a tensor is of its element type and size, contiguous, and on the
# current device like the others.  The checks are written out: they are host time
# of every launch, and by a loop over (tensor, type, size) attention_decode_kv4's
# ten tensors took 1.6 us more (9.6 us a call against 8.0).
_types = None  # fp32, int32, uint8, bf16 (or its bits), whether there are several devices


def _get_types():
    global _types
    torch = _torch()
    _types = (torch.float32, torch.int32, torch.uint8, (torch.bfloat16, torch.int16, torch.uint16),
              torch.cuda.device_count() > 1)
    return _types


def _elsewhere(dev: int, several: bool) -> bool:
    """Whether device number dev (below 0: the host) is not the current one."""
    return dev < 0 or (several and dev != _torch().cuda.current_device())


def _fresh(stream, dev: int, make):
    """make()'s new tensors, allocated for `stream` (None: the default stream) on
    device number dev.  The allocator reuses memory in the order of the stream it was
    asked on: results of torch's current stream, written on another, could still be
    in use by what ran before on the current one."""
    torch = _torch()
    if torch._C._cuda_getCurrentRawStream(dev) == (stream or 0):  # (current_stream() takes 3 us)
        return make()
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, dev) if stream else torch.cuda.default_stream(dev)):
        return make()


def _opt(t):
    return None if t is None else t.data_ptr()


def quantize_w4_weight(w_dev, stream=None):
    """tts_quantize_w4_weight on w_dev, bf16 (or int16 bf16 bits) [N][K]:
    returns (uint8 [N][K/2], bfloat16 [N][K/128]) device tensors, made for
    `stream` (None: the default stream, whatever torch's current one is)."""
    _, _, u8, bf16, several = _types or _get_types()
    N, K = w_dev.shape
    dev = w_dev.get_device()
    if w_dev.dtype not in bf16 or not w_dev.is_contiguous() or _elsewhere(dev, several):
        raise TtsError("tts_quantize_w4_weight", -1)
    empty, device = _torch().empty, w_dev.device
    q, s = _fresh(stream, dev, lambda: (empty((N, K // 2), dtype=u8, device=device),
                                        empty((N, K // 128), dtype=bf16[0], device=device)))
    _call("tts_quantize_w4_weight", w_dev.data_ptr(), N, K, q.data_ptr(), s.data_ptr(), stream)
    return q, s


def gemv_w4(x_dev, w4_dev, s_dev, y_dev, epi: int = 0, resid_dev=None, gamma_dev=None, eps: float = 1e-6,
            stream=None) -> None:
    """tts_gemv_w4: x_dev fp32 [M][K], w4_dev uint8 [N][K/2] and s_dev bf16
    [N][K/128] (epi 2: 2N rows, gate then up), y_dev fp32 [M][N]; resid_dev
    fp32 [M][N] for epi 1 (y_dev itself to add in place); gamma_dev bf16 [K]
    normalises x."""
    f32, _, u8, bf16, several = _types or _get_types()
    M, K = x_dev.shape
    N = y_dev.shape[-1]
    rows = 2 * N if epi == 2 else N
    dev = x_dev.get_device()
    if (x_dev.dtype is not f32 or not x_dev.is_contiguous()
            or w4_dev.dtype is not u8 or w4_dev.numel() != rows * (K // 2)
            or w4_dev.get_device() != dev or not w4_dev.is_contiguous()
            or s_dev.dtype not in bf16 or s_dev.numel() != rows * (K // 128)
            or s_dev.get_device() != dev or not s_dev.is_contiguous()
            or y_dev.dtype is not f32 or y_dev.numel() != M * N
            or y_dev.get_device() != dev or not y_dev.is_contiguous()
            or resid_dev is not None and (resid_dev.dtype is not f32 or resid_dev.numel() != M * N
                                          or resid_dev.get_device() != dev or not resid_dev.is_contiguous())
            or gamma_dev is not None and (gamma_dev.dtype not in bf16 or gamma_dev.numel() != K
                                          or gamma_dev.get_device() != dev or not gamma_dev.is_contiguous())
            or _elsewhere(dev, several)):
        raise TtsError("tts_gemv_w4", -1)
    _call("tts_gemv_w4", x_dev.data_ptr(), w4_dev.data_ptr(), s_dev.data_ptr(), _opt(resid_dev), _opt(gamma_dev),
          y_dev.data_ptr(), M, N, K, epi, eps, stream)


def _kv4_cache(fn: str, k4, v4, k_par, v_par):
    """The heads, positions a head and device of a 4-bit cache's tensors, checked."""
    _, _, u8, bf16, several = _types or _get_types()
    n_kv, max_pos, row = k4.shape
    n = n_kv * max_pos
    dev = k4.get_device()
    if (row != 64 or k4.dtype is not u8 or not k4.is_contiguous()
            or v4.dtype is not u8 or v4.numel() != n * 64 or v4.get_device() != dev or not v4.is_contiguous()
            or k_par.dtype not in bf16 or k_par.numel() != n * 4
            or k_par.get_device() != dev or not k_par.is_contiguous()
            or v_par.dtype not in bf16 or v_par.numel() != n * 4
            or v_par.get_device() != dev or not v_par.is_contiguous() or _elsewhere(dev, several)):
        raise TtsError(fn, -1)
    return n_kv, max_pos, dev


def _bf16_rows(fn: str, k_dev, v_dev, n_kv: int, dev: int) -> int:
    """The positions a head of bf16 caches [n_kv][positions][128], checked."""
    bf16 = _types[3]
    stride = k_dev.shape[1]
    n = n_kv * stride * 128
    if (k_dev.dtype not in bf16 or k_dev.numel() != n or k_dev.get_device() != dev or not k_dev.is_contiguous()
            or v_dev.dtype not in bf16 or v_dev.numel() != n or v_dev.get_device() != dev
            or not v_dev.is_contiguous()):
        raise TtsError(fn, -1)
    return stride


def quantize_kv4(k_dev, v_dev, k4, v4, k_par, v_par, p0: int, p1: int, stream=None) -> None:
    """tts_quantize_kv4: positions [p0, p1) of bf16 caches [n_kv][stride][128]
    into the 4-bit cache: k4, v4 uint8 [n_kv][max_pos][64], k_par, v_par bf16
    [n_kv][max_pos][2][2]."""
    n_kv, max_pos, dev = _kv4_cache("tts_quantize_kv4", k4, v4, k_par, v_par)
    stride = _bf16_rows("tts_quantize_kv4", k_dev, v_dev, n_kv, dev)
    _call("tts_quantize_kv4", k_dev.data_ptr(), v_dev.data_ptr(), n_kv, p0, p1, stride, k4.data_ptr(), v4.data_ptr(),
          k_par.data_ptr(), v_par.data_ptr(), max_pos, stream)


def dequantize_kv4(k4, v4, k_par, v_par, k_dev, v_dev, p0: int, p1: int, stream=None) -> None:
    """tts_dequantize_kv4: the values of positions [p0, p1) of a 4-bit cache into
    bf16 caches [n_kv][stride][128]."""
    n_kv, max_pos, dev = _kv4_cache("tts_dequantize_kv4", k4, v4, k_par, v_par)
    stride = _bf16_rows("tts_dequantize_kv4", k_dev, v_dev, n_kv, dev)
    _call("tts_dequantize_kv4", k4.data_ptr(), v4.data_ptr(), k_par.data_ptr(), v_par.data_ptr(), n_kv, p0, p1,
          max_pos, k_dev.data_ptr(), v_dev.data_ptr(), stride, stream)


def kv4_workspace_bytes(n_q: int, n_kv: int) -> int:
    """tts_attention_kv4_workspace: bytes of the zeroed scratch that
    attention_decode_kv4 wants."""
    n = ctypes.c_size_t()
    _call("tts_attention_kv4_workspace", n_q, n_kv, ctypes.byref(n))
    return n.value


def attention_decode_kv4(qkv, q_norm, k_norm, k4, v4, k_par, v_par, out, n_q: int, n_kv: int, pos: int, workspace,
                         kv_row=None, eps: float = 1e-6, rope_theta: float = 1e6, stream=None) -> None:
    """tts_attention_decode_kv4 on torch device tensors: qkv fp32
    [(n_q + 2 n_kv) 128], gains bf16 [128], the 4-bit cache as quantize_kv4
    takes it, out fp32 [n_q 128], workspace a uint8 tensor of
    kv4_workspace_bytes zeros (kept between calls), kv_row fp32 [2][n_kv][128]
    or None."""
    heads, max_pos, dev = _kv4_cache("tts_attention_decode_kv4", k4, v4, k_par, v_par)
    f32, _, u8, bf16, _ = _types
    if (heads != n_kv
            or qkv.dtype is not f32 or qkv.numel() != (n_q + 2 * n_kv) * 128
            or qkv.get_device() != dev or not qkv.is_contiguous()
            or q_norm.dtype not in bf16 or q_norm.numel() != 128
            or q_norm.get_device() != dev or not q_norm.is_contiguous()
            or k_norm.dtype not in bf16 or k_norm.numel() != 128
            or k_norm.get_device() != dev or not k_norm.is_contiguous()
            or out.dtype is not f32 or out.numel() != n_q * 128
            or out.get_device() != dev or not out.is_contiguous()
            or kv_row is not None and (kv_row.dtype is not f32 or kv_row.numel() != 2 * n_kv * 128
                                       or kv_row.get_device() != dev or not kv_row.is_contiguous())
            or workspace.dtype is not u8 or workspace.get_device() != dev or not workspace.is_contiguous()):
        raise TtsError("tts_attention_decode_kv4", -1)
    _call("tts_attention_decode_kv4", qkv.data_ptr(), q_norm.data_ptr(), k_norm.data_ptr(), k4.data_ptr(),
          v4.data_ptr(), k_par.data_ptr(), v_par.data_ptr(), out.data_ptr(), _opt(kv_row), n_q, n_kv, max_pos, pos,
          eps, rope_theta, workspace.data_ptr(), workspace.numel(), stream)


def code_logprobs(logits, codes, cb_vocab: int, top: int = 0, temperature: float = 1.0, stream=None):
    """tts_code_logprobs: logits fp32 [rows][ld] (rows may be strided) and codes
    int32 [rows][n_cb]; returns (logprob [rows][n_cb], entropy [rows][n_cb],
    top_codes [rows][n_cb][top], top_logprob [rows][n_cb][top]), made for `stream`
    (None: the default stream, whatever torch's current one is)."""
    f32, i32, _, _, several = _types or _get_types()
    rows, n_cb = codes.shape
    dev = codes.get_device()
    if (codes.dtype is not i32 or not codes.is_contiguous()
            or logits.dtype is not f32 or logits.get_device() != dev or logits.dim() != 2
            or logits.shape[0] != rows or logits.shape[1] < n_cb * cb_vocab or logits.stride(1) != 1
            or _elsewhere(dev, several)):
        raise TtsError("tts_code_logprobs", -1)
    ld = logits.stride(0) if rows > 1 else logits.shape[1]
    empty, device, n = _torch().empty, codes.device, max(top, 0)
    lp, ent, at, at_lp = _fresh(stream, dev, lambda: (
        empty((rows, n_cb), dtype=f32, device=device), empty((rows, n_cb), dtype=f32, device=device),
        empty((rows, n_cb, n), dtype=i32, device=device), empty((rows, n_cb, n), dtype=f32, device=device)))
    _call("tts_code_logprobs", logits.data_ptr(), ld, codes.data_ptr(), rows, n_cb, cb_vocab, temperature, top,
          lp.data_ptr(), ent.data_ptr(), at.data_ptr() if n else None, at_lp.data_ptr() if n else None, stream)
    return lp, ent, at, at_lp


@dataclass
class Dims:
    n_layers: int = 36
    hidden: int = 2560
    n_q: int = 32
    n_kv: int = 8
    head_dim: int = 128
    inter: int = 9728
    n_cb: int = 8
    cb_vocab: int = 1026
    rms_eps: float = 1e-6
    rope_theta: float = 1e6


class DeviceWeights:
    """Device copies of a weight set.  ``host`` is any object with the
    attributes embed, head, final_norm and per-layer lists wqkv, wo, wgu, wd,
    ln_in, ln_post, q_norm, k_norm holding bf16 bit images (uint16 numpy).
    For FP8 the four projection matrices of each layer are quantised on the
    GPU by tts_quantize_fp8_weight and only the E4M3 copies are kept."""

    def __init__(self, host, precision: int = TTS_BF16, device="cuda"):
        torch = _torch()
        self.precision = precision
        d = lambda a: _to_dev_u16(a, device)
        self.embed, self.head, self.final_norm = d(host.embed), d(host.head), d(host.final_norm)
        self.mats = {n: [] for n in ("wqkv", "wo", "wgu", "wd")}
        self.scales = {n: [] for n in ("wqkv", "wo", "wgu", "wd")}
        for name in ("wqkv", "wo", "wgu", "wd"):
            for m in getattr(host, name):
                t = d(m)
                if precision == TTS_FP8:
                    q, s = quantize_fp8_weight(t)
                    del t
                    self.mats[name].append(q)
                    self.scales[name].append(s)
                else:
                    self.mats[name].append(t)
        self.norms = {n: [d(x) for x in getattr(host, n)] for n in ("ln_in", "ln_post", "q_norm", "k_norm")}
        torch.cuda.synchronize()
        self.n_layers = len(self.mats["wqkv"])

    def struct(self) -> tts_weights:
        L = self.n_layers
        keep = []

        def arr(ts):
            a = (ctypes.c_void_p * L)(*[t.data_ptr() for t in ts])
            keep.append(a)
            return ctypes.cast(a, _PP)

        w = tts_weights()
        w.embed, w.head, w.final_norm = self.embed.data_ptr(), self.head.data_ptr(), self.final_norm.data_ptr()
        w.wqkv, w.wo, w.wgu, w.wd = (arr(self.mats[n]) for n in ("wqkv", "wo", "wgu", "wd"))
        if self.precision == TTS_FP8:
            w.sqkv, w.so, w.sgu, w.sd = (arr(self.scales[n]) for n in ("wqkv", "wo", "wgu", "wd"))
        w.ln_in, w.ln_post, w.q_norm, w.k_norm = (arr(self.norms[n]) for n in ("ln_in", "ln_post", "q_norm", "k_norm"))
        self._keep = keep
        return w


# ----------------------------------------------------------------------------
# The decoder context
# ----------------------------------------------------------------------------

class Decoder:
    """One tts_ctx: KV cache, scratch and the captured decode-step graph."""

    def __init__(self, dims, weights: DeviceWeights, max_pos: int, stream=None, options: int = 0):
        self.dims = dims
        self.weights = weights
        cfg = tts_config(dims.n_layers, dims.hidden, dims.n_q, dims.n_kv, dims.head_dim, dims.inter,
                         dims.n_cb, dims.cb_vocab, max_pos, dims.rms_eps, dims.rope_theta,
                         weights.precision, stream, options)
        self._cfg = cfg
        self._w = weights.struct()
        self._ctx = ctypes.c_void_p()
        _call("tts_init", ctypes.byref(cfg), ctypes.byref(self._w), ctypes.byref(self._ctx))
        self.max_pos = max_pos

    @property
    def handle(self):
        return self._ctx

    def close(self):
        if self._ctx:
            _call("tts_shutdown", self._ctx)
            self._ctx = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def reset(self):
        _call("tts_reset", self._ctx)

    def prefill(self, codes: np.ndarray):
        c = np.ascontiguousarray(codes, np.int32)
        _call("tts_prefill", self._ctx, _ptr(c), c.shape[0])

    def decode_step(self, codes_in=None) -> np.ndarray:
        out = np.empty(self.dims.n_cb, np.int32)
        if codes_in is None:
            _call("tts_decode_step", self._ctx, None, _ptr(out))
        else:
            c = np.ascontiguousarray(codes_in, np.int32)
            _call("tts_decode_step", self._ctx, _ptr(c), _ptr(out))
        return out

    def decode_steps(self, n: int) -> np.ndarray:
        out = np.empty((n, self.dims.n_cb), np.int32)
        _call("tts_decode_steps", self._ctx, n, _ptr(out))
        return out

    def set_sampling(self, temperature: float, seed: int = 0):
        """tts_set_sampling: 0 = greedy argmax; > 0 = seeded categorical draws
        from softmax(logits / temperature)."""
        _call("tts_set_sampling", self._ctx, float(temperature), int(seed) & 0xFFFFFFFFFFFFFFFF)

    def decode_until_eoc(self, max_frames: int) -> np.ndarray:
        """tts_decode_until_eoc: free-running frames with one frame of
        lookahead until the last codebook's EOC; returns the codes [n][n_cb]."""
        out = np.empty((max_frames, self.dims.n_cb), np.int32)
        n = ctypes.c_int()
        _call("tts_decode_until_eoc", self._ctx, max_frames, _ptr(out), ctypes.byref(n))
        return out[:n.value]

    def set_fp8_scales(self, scales=None):
        """tts_set_fp8_scales: static activation scales [n_layers][4] (0 =
        dynamic for that site), or None for all dynamic."""
        if scales is None:
            _call("tts_set_fp8_scales", self._ctx, None)
            return
        a = np.ascontiguousarray(scales, np.float32).reshape(self.dims.n_layers, 4)
        _call("tts_set_fp8_scales", self._ctx, _ptr(a))

    def fp8_calibrate(self, n_frames: int) -> np.ndarray:
        """tts_fp8_calibrate: per-site amax [n_layers][4] over n_frames
        discarded free-running frames."""
        out = np.zeros((self.dims.n_layers, 4), np.float32)
        _call("tts_fp8_calibrate", self._ctx, n_frames, _ptr(out))
        return out

    def prefix_save(self):
        """tts_prefix_save: snapshot the cache rows [0, pos) and the state."""
        _call("tts_prefix_save", self._ctx)

    def prefix_restore(self):
        """tts_prefix_restore: back to the saved prefix (cache rows and state)."""
        _call("tts_prefix_restore", self._ctx)

    def set_input(self, codes):
        """tts_set_input: the next step's input frame (host codes [n_cb])."""
        c = np.ascontiguousarray(codes, np.int32)
        _call("tts_set_input", self._ctx, _ptr(c))

    def rewind(self, pos: int, t: int = 0):
        _call("tts_rewind", self._ctx, pos, t)

    def set_kv(self, k_dev, v_dev, length: int, len_stride: int | None = None):
        _call("tts_set_kv", self._ctx, k_dev.data_ptr(), v_dev.data_ptr(), length,
              length if len_stride is None else len_stride)

    def get_kv(self, p0: int, p1: int):
        d = self.dims
        shape = (d.n_layers, d.n_kv, p1 - p0, d.head_dim)
        k = np.empty(shape, np.uint16)
        v = np.empty(shape, np.uint16)
        _call("tts_get_kv", self._ctx, _ptr(k), _ptr(v), p0, p1)
        return k, v

    def get_logits(self) -> np.ndarray:
        out = np.empty((self.dims.n_cb, self.dims.cb_vocab), np.float32)
        _call("tts_get_logits", self._ctx, _ptr(out))
        return out

    def logprobs(self, codes=None, top: int = 0, temperature: float = 1.0):
        """tts_get_logprobs on the last step's logits: (logprob [n_cb] of `codes`
        (default: the codes the last step produced), entropy [n_cb], top codes
        [n_cb][top], their log probabilities [n_cb][top])."""
        n = self.dims.n_cb
        lp, ent = np.empty(n, np.float32), np.empty(n, np.float32)
        at, at_lp = np.empty((n, max(top, 0)), np.int32), np.empty((n, max(top, 0)), np.float32)
        c = None
        if codes is not None:
            c = np.asarray(codes).reshape(n)
            if not ((c >= 0) & (c < self.dims.cb_vocab)).all():  # before a wider integer wraps
                raise TtsError("tts_get_logprobs", -2)
            c = np.ascontiguousarray(c, np.int32)
        _call("tts_get_logprobs", self._ctx, None if c is None else _ptr(c), float(temperature), top, _ptr(lp),
              _ptr(ent), _ptr(at) if top > 0 else None, _ptr(at_lp) if top > 0 else None)
        return lp, ent, at, at_lp

    def get_hidden(self) -> np.ndarray:
        out = np.empty(self.dims.hidden, np.float32)
        _call("tts_get_hidden", self._ctx, _ptr(out))
        return out

    def set_frame(self, t: int, eoc: int = -1):
        _call("tts_set_frame", self._ctx, t, eoc)

    def state(self):
        p, t, e = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
        _call("tts_get_state", self._ctx, ctypes.byref(p), ctypes.byref(t), ctypes.byref(e))
        return p.value, t.value, e.value

    def time_gemv(self, kind: int, reps: int = 1) -> float:
        """Mean device ms of one launch of projection `kind` (0 QKV, 1 O, 2 gate/up, 3 down, 4 head)."""
        ms = ctypes.c_float()
        _call("tts_time_gemv", self._ctx, kind, reps, ctypes.byref(ms))
        return ms.value

    def trace_step(self, n_sms_max: int = 1024):
        """One decode step with the persistent kernel's phase trace: uint64 ns
        stamps shaped [n_cta][stride]."""
        cap = n_sms_max * (8 + 31 * self.dims.n_layers) + 2 * 4 * 2048
        buf = np.zeros(cap, np.uint64)
        st, nc = ctypes.c_int(), ctypes.c_int()
        _call("tts_trace_step", self._ctx, _ptr(buf), cap, ctypes.byref(st), ctypes.byref(nc))
        n = st.value * nc.value
        self.last_stage_trace = buf[n: n + 2 * 4 * 2048].reshape(2, 2048, 4)
        return buf[:n].reshape(nc.value, st.value)

    def layer_states(self, codes_in=None):
        """One decode step (as decode_step) through the traced step kernel,
        returning (codes, hidden states [n_layers + 1][hidden]): the residual
        stream after the embedding and after each layer."""
        n = (self.dims.n_layers + 1) * self.dims.hidden
        buf = np.zeros(n, np.float32)
        out = np.empty(self.dims.n_cb, np.int32)
        c = None if codes_in is None else np.ascontiguousarray(codes_in, np.int32)
        _call("tts_debug_layer_states", self._ctx, None if c is None else _ptr(c), _ptr(out), _ptr(buf), n)
        return out, buf.reshape(self.dims.n_layers + 1, self.dims.hidden)

    def prefill_states(self, codes):
        """prefill(codes) on the batched path, returning the residual stream of
        every row after the embedding and after each layer: [n_layers + 1][P][hidden]."""
        c = np.ascontiguousarray(codes, np.int32)
        P = c.shape[0]
        n = (self.dims.n_layers + 1) * P * self.dims.hidden
        buf = np.zeros(n, np.float32)
        _call("tts_debug_prefill_states", self._ctx, _ptr(c), P, _ptr(buf), n)
        return buf.reshape(self.dims.n_layers + 1, P, self.dims.hidden)

    def debug_expire_wait(self) -> int:
        """tts_debug_expire_wait: one step launch whose first wait (for the
        embedding, never stored) cannot complete and whose waits give up
        after 1 ms; returns the status code (TTS_ERR_DEVICE, -5, when the
        timeout was detected)."""
        return int(load().tts_debug_expire_wait(self._ctx))

    def last_steps_ms(self) -> float:
        ms = ctypes.c_float()
        _call("tts_last_steps_ms", self._ctx, ctypes.byref(ms))
        return ms.value
