"""Log probabilities, entropy and alternatives of given codes, on the GPU,
against the fp64 restatement."""
import numpy as np
import pytest

import four_bit_ref as ref
import synth

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


def run(ads, z, codes, top, T=1.0, ld=None):
    """z fp32 [rows][n_cb][V] through the library, rows ld apart."""
    import torch
    rows, n_cb, V = z.shape
    ld = ld or n_cb * V
    buf = torch.full((rows, ld), float("nan"), device="cuda")
    buf[:, :n_cb * V] = torch.from_numpy(z.reshape(rows, -1)).cuda()
    got = ads.code_logprobs(buf[:, :n_cb * V] if ld > n_cb * V else buf, torch.from_numpy(codes).cuda(), V, top=top,
                            temperature=T)
    return [t.cpu().numpy() for t in got]


def check(got, z, codes, top, T=1.0):
    lp, ent, at, at_lp, t_lp, t_ent, t_at = ref.code_logprobs(z, codes, top, T)
    for g, w, t in ((got[0], lp, t_lp), (got[1], ent, t_ent), (got[3], at_lp, t_at)):
        fine = np.isfinite(w)
        assert np.array_equal(fine, np.isfinite(g)) and np.array_equal(g[~fine & ~np.isnan(w)], w[~fine & ~np.isnan(w)])
        assert (np.abs(g[fine] - w[fine]) <= t[fine]).all(), np.max(np.abs(g[fine] - w[fine]) / t[fine])
    assert np.array_equal(got[2], at)


def codes_for(rows, n_cb, V, seed):
    return np.random.default_rng(seed).integers(0, V, (rows, n_cb)).astype(np.int32)


@pytest.mark.parametrize("rows,n_cb,V,top,T,pad", [
    (1, 8, 1026, 5, 1.0, 0), (1, 1, 2, 2, 1.0, 0), (3, 8, 2, 1, 0.5, 3), (5, 3, 31, 31, 1.0, 1), (2, 7, 33, 32, 1.3, 0),
    (17, 5, 127, 0, 1.0, 0), (40, 8, 1026, 32, 0.7, 48), (9, 4, 1025, 20, 2.0, 5), (300, 8, 1026, 5, 1.0, 0),
    (2, 2, 2050, 7, 1.0, 1), (3, 1, 4097, 20, 1.0, 0), (2, 1, 16385, 32, 0.8, 2), (3, 1, 131072, 20, 0.8, 0),
    (1, 1, 150001, 32, 1.0, 7), (2, 3, 65537, 1, 1.0, 0), (200, 1, 20000, 5, 1.0, 0), (1, 1, 1 << 20, 32, 1.0, 0)])
def test_code_logprobs(ads, rows, n_cb, V, top, T, pad):
    z = synth.normal_f32(7, V, (rows, n_cb, V), std=2.5)
    if V > 64:
        z[:, :, V - 2] = -np.inf
        z[0, 0, ::7] = -np.inf
    codes = codes_for(rows, n_cb, V, V)
    got = run(ads, z, codes, top, T, n_cb * V + pad)
    check(got, z, codes, top, T)
    again = run(ads, z, codes, top, T, n_cb * V + pad)
    assert all(np.array_equal(a, b, equal_nan=True) for a, b in zip(got, again))


@pytest.mark.parametrize("rows,n_cb,V,top", [(2000, 1, 5300, 20), (600, 1, 17000, 6), (330, 2, 3200, 32), (700, 1, 9000, 1)])
def test_many_long_rows(ads, rows, n_cb, V, top):
    """Rows enough for a warp to take several runs of each: runs that rise, so that
    the alternatives found first are replaced, that fall, and ones of a few values,
    where most entries are equal."""
    z = synth.normal_f32(7, V + top, (rows, n_cb, V), std=2.0)
    z[0::4] += np.linspace(-6.0, 6.0, V, dtype=np.float32)
    z[1::4] -= np.linspace(-6.0, 6.0, V, dtype=np.float32)
    z[2::4] = np.round(z[2::4])
    codes = codes_for(rows, n_cb, V, V)
    check(run(ads, z, codes, top), z, codes, top)


@pytest.mark.parametrize("V", [5, 1026, 9001])
def test_ties_go_to_the_lowest_code(ads, V):
    z = np.round(synth.normal_f32(7, 3, (6, 2, V)) * 2).astype(np.float32)
    z[0] = 1.5                        # every entry equal
    z[1, :, ::2], z[1, :, 1::2] = 0.0, -0.0
    z[2] = -np.inf
    z[2, :, 3] = 0.0                  # one entry left: the rest of the alternatives are -inf
    z[3, :, V - 1] = 50.0             # almost one-hot at the last entry
    top = min(V, 32)
    check(run(ads, z, codes_for(6, 2, V, 1), top), z, codes_for(6, 2, V, 1), top)


@pytest.mark.parametrize("V", [300, 1026, 5000])
@pytest.mark.parametrize("top", [1, 5, 20, 32])
def test_alternatives_of_awkward_values(ads, V, top):
    """Runs of equal values across the last alternative's, values one step apart,
    zeros of both signs, subnormals, the largest and infinite ones."""
    rng = np.random.default_rng(V + top)
    z = synth.normal_f32(7, 4, (8, 2, V))
    z[0] = rng.choice(np.float32([0.0, -0.0, 1e-45, -1e-45, 2e-45]), (2, V))
    z[1] = np.float32(1) + rng.integers(0, 40, (2, V)).astype(np.float32) * np.float32(2 ** -23)
    z[2, :, :200] = 3.0                             # far more than 64 at the maximum
    z[3] = -rng.choice(np.float32([3.4028235e38, 3.4e38, 1.0]), (2, V))
    z[4] = np.where(rng.random((2, V)) < 0.97, -np.inf, z[4])
    z[5] = np.where(rng.random((2, V)) < 0.5, np.float32(-0.0), np.float32(-1))
    z[5, 0, ::9] = 0.0
    z[6] = np.round(z[6] * 30) / 30                 # ties everywhere
    z[7] = np.sort(z[7])                            # all the largest at the end
    codes = codes_for(8, 2, V, top)
    check(run(ads, z, codes, top), z, codes, top)


@pytest.mark.parametrize("V", [4, 1026, 40000])
def test_masked_and_non_finite_rows(ads, V):
    z = synth.normal_f32(7, 9, (6, 1, V), std=2.5)
    z[0] = -np.inf                    # nothing left
    z[1, 0, 2] = np.nan
    z[2, 0, V - 1] = np.inf
    z[3] = -np.inf
    z[3, 0, 1] = np.nan               # nothing but a NaN
    codes = np.array([[0], [0], [1], [0], [V], [-1]], np.int32)
    lp, ent, at, at_lp = run(ads, z, codes, 3)
    assert lp[0, 0] == -np.inf and ent[0, 0] == 0
    assert at[0, 0].tolist() == [0, 1, 2] and (at_lp[0] == -np.inf).all()
    for r in (1, 2, 3):
        assert np.isnan(lp[r]).all() and np.isnan(ent[r]).all() and np.isnan(at_lp[r]).all()
    assert 2 not in at[1] and at[2, 0, 0] == V - 1
    order = np.argsort(-z[1, 0], kind="stable")  # NaN sorts last
    assert at[1, 0].tolist() == order[:3].tolist()
    assert at[3, 0].tolist() == [0, 2, 3]
    assert np.isnan(lp[4:]).all()      # codes outside [0, V)
    _, want_ent, want_at, want_lp, _, t_ent, t_at = ref.code_logprobs(z[4:], np.zeros((2, 1), np.int32), 3, 1.0)
    assert (np.abs(ent[4:] - want_ent) <= t_ent).all() and np.array_equal(at[4:], want_at)
    assert (np.abs(at_lp[4:] - want_lp) <= t_at).all()


@pytest.mark.parametrize("V", [1026, 70000])
def test_large_logits_and_small_temperature(ads, V):
    z = synth.normal_f32(7, 11, (3, 1, V), std=2.5)
    z[0] *= 1e30
    z[1] += 3e6
    z[2] -= 1e3
    codes = codes_for(3, 1, V, 2)
    check(run(ads, z, codes, 4), z, codes, 4)
    check(run(ads, z[2:], codes[2:], 4, 1e-3), z[2:], codes[2:], 4, 1e-3)


def test_optional_outputs_and_capture(ads):
    """Without codes, entropy or alternatives nothing of them is written; a
    captured call replays on new logits."""
    import torch
    V, n_cb, rows = 1026, 8, 4
    z = torch.from_numpy(synth.normal_f32(7, 21, (rows, n_cb * V), std=2.5)).cuda()
    codes = torch.from_numpy(codes_for(rows, n_cb, V, 5)).cuda()
    ent = torch.zeros((rows, n_cb), device="cuda")
    ads._call("tts_code_logprobs", z.data_ptr(), n_cb * V, None, rows, n_cb, V, 1.0, 0, None, ent.data_ptr(), None,
              None, None)
    lp2, ent2, _, _ = ads.code_logprobs(z, codes, V)
    assert torch.equal(ent, ent2)
    lp = torch.zeros_like(ent)
    ads._call("tts_code_logprobs", z.data_ptr(), n_cb * V, codes.data_ptr(), rows, n_cb, V, 1.0, 0, lp.data_ptr(),
              None, None, None, None)
    assert torch.equal(lp, lp2)
    torch.cuda.synchronize()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = ads.code_logprobs(z, codes, V, top=3, stream=s.cuda_stream)
    z.copy_(torch.from_numpy(synth.normal_f32(7, 22, (rows, n_cb * V), std=2.5)))
    g.replay()
    torch.cuda.synchronize()
    check([t.cpu().numpy() for t in got], z.cpu().numpy().reshape(rows, n_cb, V), codes.cpu().numpy(), 3)


def test_context_logprobs(ads):
    """tts_get_logprobs on a decode step: the context's own logits, the codes it
    produced by default, given codes otherwise."""
    from helpers import reduced_dims, to_binding_dims
    d = reduced_dims()
    dec = ads.Decoder(to_binding_dims(d), ads.DeviceWeights(synth.make_weights(d)), 32)
    dec.prefill(synth.delayed_prompt_codes(5))
    dec.set_frame(8)
    got = dec.decode_step(synth.random_codes(1)[0])
    z = dec.get_logits()[None]
    check([a[None] for a in dec.logprobs(top=5)], z, got[None].astype(np.int32), 5)
    assert np.array_equal(dec.logprobs(top=1)[2][:, 0], got)  # greedy: the argmax is the first alternative
    given = np.arange(8, dtype=np.int32) * 100
    check([a[None] for a in dec.logprobs(given, top=0, temperature=0.9)], z, given[None], 0, 0.9)
    for bad in (1026, -1):
        with pytest.raises(ads.TtsError) as e:
            dec.logprobs(np.full(8, bad))
        assert e.value.status == -2
    for kw in (dict(top=33), dict(top=-1), dict(temperature=0.0)):
        with pytest.raises(ads.TtsError) as e:
            dec.logprobs(**kw)
        assert e.value.status == -1
    dec.close()
