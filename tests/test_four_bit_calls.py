"""Calls of the 4-bit operators and the code scoring that their documentation
allows or refuses, found on the host before any device call (no GPU needed)."""
import pytest

ARG = -1
A = [0x1000000 * (i + 1) for i in range(16)]  # far apart, 16-byte aligned stand-ins, never dereferenced


@pytest.fixture(scope="module")
def lib():
    import ar_decode_step_gb300.build as b
    b.build()
    import ar_decode_step_gb300 as m
    return m.load()


SCORE = dict(z=A[0], ld=8208, codes=A[1], rows=4, n_cb=8, V=1026, T=1.0, top=5, lp=A[2], ent=A[3], at=A[4],
             at_lp=A[5], stream=None)


def test_code_logprobs_of_no_rows_wants_no_memory(lib):
    """An empty tensor's address is NULL: with no rows nothing is read or written.
    The sizes are checked all the same."""
    none = dict(SCORE, z=None, codes=None, rows=0, lp=None, ent=None, at=None, at_lp=None)
    assert lib.tts_code_logprobs(*none.values()) == 0
    assert lib.tts_code_logprobs(*dict(none, top=0).values()) == 0
    for bad in (dict(V=1), dict(n_cb=9), dict(top=33), dict(T=0.0), dict(ld=8207)):
        assert lib.tts_code_logprobs(*dict(none, **bad).values()) == ARG, bad


# ---- what the binding checks, on host tensors that claim a device ---------------------

class On:
    """A host tensor that says it is on a device (its address reaches no library here)."""

    def __init__(self, t, device=0):
        self.t, self.device_number = t, device

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.device_number

    @property
    def is_cuda(self):
        return self.device_number >= 0


def calls():
    """Per function: its arguments, and the names of those that are tensors."""
    import torch
    f = lambda *s: torch.zeros(s)
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    u = lambda *s: torch.zeros(s, dtype=torch.uint8)
    cache = lambda: dict(k4=u(2, 9, 64), v4=u(2, 9, 64), k_par=b(2, 9, 2, 2), v_par=b(2, 9, 2, 2))
    return {
        "quantize_w4_weight": dict(w_dev=b(4, 256)),
        "gemv_w4": dict(x_dev=f(3, 256), w4_dev=u(10, 128), s_dev=b(10, 2), y_dev=f(3, 5), epi=2, gamma_dev=b(256)),
        "gemv_w4 ": dict(x_dev=f(3, 256), w4_dev=u(5, 128), s_dev=b(5, 2), y_dev=f(3, 5), epi=1, resid_dev=f(3, 5)),
        "quantize_kv4": dict(k_dev=b(2, 6, 128), v_dev=b(2, 6, 128), **cache(), p0=1, p1=4),
        "dequantize_kv4": dict(**cache(), k_dev=b(2, 6, 128), v_dev=b(2, 6, 128), p0=1, p1=4),
        "attention_decode_kv4": dict(qkv=f(8 * 128), q_norm=b(128), k_norm=b(128), **cache(), out=f(4 * 128), n_q=4,
                                     n_kv=2, pos=3, workspace=u(64), kv_row=f(2, 2, 128)),
        "code_logprobs": dict(logits=f(3, 40), codes=torch.zeros((3, 4), dtype=torch.int32), cb_vocab=10, top=2),
    }


@pytest.fixture
def binding(lib, monkeypatch):
    """The binding on a machine of two devices, device 0 current; what reaches the library is listed."""
    import torch
    import ar_decode_step_gb300 as m
    seen = []
    monkeypatch.setattr(m, "_call", lambda name, *args: seen.append(name))
    monkeypatch.setattr(m, "_types", None, raising=False)
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)
    return m, seen


@pytest.mark.parametrize("name", list(calls()))
def test_binding_checks_every_tensor(binding, name):
    """Another element type, size, layout or device of any one tensor is refused
    before the library is called; bf16 tensors may be their bits."""
    import torch
    m, seen = binding
    f = getattr(m, name.strip())
    good = calls()[name]
    tensors = [n for n, v in good.items() if isinstance(v, torch.Tensor)]

    def call(**change):
        args = {n: On(v) if isinstance(v, torch.Tensor) else v for n, v in good.items()}
        args.update(change)
        f(**args)

    call()
    call(**{n: On(good[n].view(torch.int16)) for n in tensors if good[n].dtype is torch.bfloat16})
    assert len(seen) == 2
    for n in tensors:
        t = good[n]
        shorter = t[:-1] if t.dim() == 1 or n == "codes" else t[..., :-1].contiguous()
        bad = dict(fp16=On(t.to(torch.float16)), wider=On(t.to(torch.float64)), host=On(t, -1), elsewhere=On(t, 1))
        bad["layout"] = On(torch.stack((t, t), -1)[..., 0])
        if t.dtype is torch.int32:
            bad["fp32"] = On(t.view(torch.float32))
        if t.dtype is torch.float32:
            bad["int32"] = On(t.view(torch.int32))
        if n not in ("w_dev", "workspace"):  # their sizes are the library's to check
            bad["size"] = On(shorter)
        for kind, wrong in bad.items():
            with pytest.raises(m.TtsError) as e:
                call(**{n: wrong})
            assert e.value.status == ARG, (n, kind)
    with pytest.raises(m.TtsError):  # all on one device, but not the current one
        call(**{n: On(good[n], 1) for n in tensors})
    assert len(seen) == 2


# ---- what is written over another argument ----------------------------------------------

def test_quantize_w4_refuses_results_over_the_weights(lib):
    """A warp writes its group's codes while others still read W."""
    good = dict(W=A[0], N=16, K=256, W4=A[1], s=A[2], stream=None)
    for bad in (dict(W4=A[0]), dict(W4=A[0] + 16 * 512 - 16), dict(s=A[0] + 4), dict(s=A[1] + 16 * 128 - 4),
                dict(W4=A[2] + 48)):
        assert lib.tts_quantize_w4_weight(*dict(good, **bad).values()) == ARG, bad


def test_kv4_rows_refuse_results_over_one_another(lib):
    """k and v, codes and parameters are written at once."""
    n = 2 * 16
    good = dict(k=A[0], v=A[1], n_kv=2, p0=0, p1=8, stride=16, k4=A[2], v4=A[3], k_par=A[4], v_par=A[5], max_pos=16,
                stream=None)
    for bad in (dict(v4=A[2]), dict(v4=A[2] + n * 64 - 16), dict(v_par=A[4]), dict(k_par=A[2] + 16),
                dict(v_par=A[3] + n * 64 - 16), dict(k4=A[5] + n * 8 - 16)):
        assert lib.tts_quantize_kv4(*dict(good, **bad).values()) == ARG, bad
    order = ("k4", "v4", "k_par", "v_par", "n_kv", "p0", "p1", "max_pos", "k", "v", "stride", "stream")
    for bad in (dict(v=A[0]), dict(v=A[0] + n * 256 - 16)):
        args = dict(good, **bad)
        assert lib.tts_dequantize_kv4(*(args[a] for a in order)) == ARG, bad


def test_code_logprobs_refuses_results_over_the_logits(lib):
    """A row's results are written while others are read."""
    row, rows, n = 4 * 8208, 4, 4 * 8
    for bad in (dict(lp=A[0]), dict(ent=A[0] + rows * row - 4), dict(at=A[0] + row), dict(at_lp=A[0] + 64),
                dict(lp=A[1]), dict(at=A[1] + 4 * n - 4), dict(ent=A[2]), dict(ent=A[4] + 4 * n * 5 - 4),
                dict(at_lp=A[3] + 4), dict(at=A[5])):
        assert lib.tts_code_logprobs(*dict(SCORE, **bad).values()) == ARG, bad
    # rows further apart than any memory is large
    assert lib.tts_code_logprobs(*dict(SCORE, ld=1 << 60).values()) == ARG


def test_code_logprobs_takes_temperatures_that_are_normal_numbers(lib):
    """2 log2(e) / T has to be finite: from the smallest normal number on."""
    none = dict(SCORE, z=None, codes=None, rows=0, lp=None, ent=None, at=None, at_lp=None)
    for T in (2.0 ** -126, 1e-37, 1e38, 3.4e38):
        assert lib.tts_code_logprobs(*dict(none, T=T).values()) == 0
    for T in (1.1e-38, 6e-39, 1e-45, -1e-37):
        assert lib.tts_code_logprobs(*dict(none, T=T).values()) == ARG, T


def test_decoder_logprobs_refuses_codes_that_wrap(lib):
    """A code of 2^32 + 5 is not code 5 (found before the context is looked at)."""
    import numpy as np
    import ar_decode_step_gb300 as m
    dec = object.__new__(m.Decoder)
    dec._ctx, dec.dims = None, m.Dims()
    n, V = dec.dims.n_cb, dec.dims.cb_vocab
    for bad in (2 ** 32 + 5, -2 ** 32, V, -1, float("nan")):
        codes = np.zeros(n, np.float64 if bad != bad else np.int64)
        codes[n - 1] = bad
        with pytest.raises(m.TtsError) as e:
            dec.logprobs(codes)
        assert e.value.status == -2, bad
    with pytest.raises(m.TtsError) as e:
        dec.logprobs(np.full(n, V - 1))
    assert e.value.status == -6  # codes in range: the context is what is missing
