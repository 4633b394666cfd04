"""What the 4-bit decode operators and the code scoring are measured on.

Three operators: the matrix-vector product with 4-bit weights (`gemv_w4`),
decode attention over a cache held in 4 bits together with the writing and
reading back of cache rows (`attention_decode_kv4`, `quantize_kv4`,
`dequantize_kv4`), and the log probabilities of given codes with entropy and
top alternatives (`code_logprobs`).  `run` computes each in plain torch
operations, or (where `own` is true) through the library.

Formats (the same on both sides):
  weights  uint8 [rows][K/2], low nibble = even k, value = s * (nibble - 8)
           with one bf16 scale s per row and 128 consecutive k: [rows][K/128].
  cache    uint8 [n_kv][max_pos][64] and bf16 [n_kv][max_pos][2][2]: channels
           0-63 and 64-127 of a row have a (scale, minimum) pair each, value =
           minimum + scale * nibble.  Byte 8r + j of a row holds channels
           8r + 2j (low nibble) and 8r + 2j + 1 for j < 4, and the same
           channels + 64 in bytes 8r + 4 + j.
"""
import math

import torch

own = False

D = 128
EPS, THETA = 1e-6, 1e6


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decoded frame, O projection of the 2560-wide backbone, added to the residual stream
        dict(name="gemv_o_m1", op="gemv", M=1, N=2560, K=4096, epi=1, norm=False),
        # one decoded frame, the largest product of a layer: normalised input, gate and up rows, SwiGLU
        dict(name="gemv_gate_up_m1", op="gemv", M=1, N=9728, K=2560, epi=2, norm=True),
        # eight short-prompt rows (or candidates) through the down projection
        dict(name="gemv_down_m8", op="gemv", M=8, N=2560, K=9728, epi=1, norm=False),
        # the first position of an utterance: no cached row, latency alone
        dict(name="attn_first", op="attn", n_q=32, n_kv=8, pos=0, max_pos=32),
        # a usual context: a 1024-position prefix and some 250 frames
        dict(name="attn_1280", op="attn", n_q=32, n_kv=8, pos=1279, max_pos=2048),
        # eight query heads on each of two key-value heads, an odd length
        dict(name="attn_g8_10007", op="attn", n_q=16, n_kv=2, pos=10007, max_pos=16384),
        # the longest cache a context takes
        dict(name="attn_65536", op="attn", n_q=32, n_kv=8, pos=65535, max_pos=65536),
        # a 13-position prompt moved into a 4-bit cache and read back
        dict(name="store_13", op="store", n_kv=8, p0=0, p1=13, max_pos=141),
        # an idle 8192-position prefix parked in 4 bits and restored
        dict(name="store_8192", op="store", n_kv=8, p0=0, p1=8192, max_pos=8256),
        # one frame's eight codebooks with five alternatives each
        dict(name="score_frame", op="score", rows=1, n_cb=8, V=1026, top=5, T=1.0),
        # a teacher-forced batch of utterances, 4096 frames in all
        dict(name="score_frames_4096", op="score", rows=4096, n_cb=8, V=1026, top=5, T=1.0),
        # one large vocabulary in two rows: long rows, little to spread
        dict(name="score_wide", op="score", rows=2, n_cb=1, V=131072, top=20, T=0.8),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gemv", "attn", "store", "score"])
    if op == "gemv":
        epi = rng.choice([0, 1, 2])
        return dict(op=op, M=rng.randint(1, 8), N=_log_int(rng, 16, 6000 if epi == 2 else 12000),
                    K=128 * _log_int(rng, 1, 96), epi=epi, norm=rng.random() < 0.5)
    if op == "attn":
        n_kv = rng.choice([1, 2, 3, 5, 8])
        pos = _log_int(rng, 1, 65536) - 1
        return dict(op=op, n_q=n_kv * rng.choice([1, 2, 4, 8]), n_kv=n_kv, pos=pos,
                    max_pos=min(65536, pos + 1 + _log_int(rng, 1, 200)))
    if op == "store":
        p0 = rng.choice([0, 0, rng.randint(1, 500)])
        p1 = p0 + _log_int(rng, 1, 20000)
        return dict(op=op, n_kv=rng.choice([1, 2, 3, 8]), p0=p0, p1=p1, max_pos=p1 + rng.randint(0, 99))
    V = _log_int(rng, 2, 150000)
    n_cb = rng.randint(1, 8) if V < 20000 else 1
    return dict(op=op, rows=_log_int(rng, 1, max(1, min(4096, 16000000 // (V * n_cb)))), n_cb=n_cb, V=V,
                top=min(V, rng.choice([0, 1, 5, 20, 32])), T=rng.choice([1.0, 1.0, 0.7, 1.3]))


def work(case):
    c = case
    if c["op"] == "gemv":
        rows = c["N"] * (2 if c["epi"] == 2 else 1)
        b = rows * c["K"] // 2 + 2 * rows * (c["K"] // 128) + 4 * c["M"] * (c["K"] + c["N"])
        b += 4 * c["M"] * c["N"] * (c["epi"] == 1) + 2 * c["K"] * c["norm"]
        return {"bytes": b, "flops": 2 * c["M"] * rows * c["K"]}
    if c["op"] == "attn":
        rows = 2 * c["n_kv"] * (c["pos"] + 1)  # read, the new ones written
        return {"bytes": 72 * rows + 4 * D * (2 * c["n_q"] + 2 * c["n_kv"]) + 4 * D + 8 * D * c["n_kv"],
                "flops": 4 * c["n_q"] * D * (c["pos"] + 1)}
    if c["op"] == "store":
        rows = 2 * c["n_kv"] * (c["p1"] - c["p0"])  # bf16 in, 4 bits out and in again, bf16 out
        return {"bytes": rows * (256 + 72 + 72 + 256), "flops": rows * D * 6}
    n = c["rows"] * c["n_cb"]
    return {"bytes": 4 * n * c["V"] + 4 * n + 8 * n + 8 * n * c["top"], "flops": 5 * n * c["V"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed, at):
    return torch.Generator(device="cuda").manual_seed(1000003 * seed + at)


def _randn(shape, g, std=1.0, mean=0.0):
    return torch.randn(shape, generator=g, device="cuda") * std + mean


def prepare(case, seed):
    c = case
    g = _gen(seed, 1)
    if c["op"] == "gemv":
        rows = c["N"] * (2 if c["epi"] == 2 else 1)
        w = _randn((rows, c["K"] // 128, 128), g, 0.02)
        s = (w.abs().amax(-1) / 7).bfloat16()
        u = (w / s.float().unsqueeze(-1)).round_().clamp_(-8, 7).add_(8).to(torch.uint8).view(rows, c["K"])
        st = dict(case=c, w4=u[:, 0::2] | (u[:, 1::2] << 4), s=s,
                  x=_randn((c["M"], c["K"]), g, 1.5), y=torch.empty((c["M"], c["N"]), device="cuda"))
        st["resid"] = _randn((c["M"], c["N"]), g) if c["epi"] == 1 else None
        st["gamma"] = _randn((c["K"],), g, 0.02, 1.0).bfloat16() if c["norm"] else None
        return st
    if c["op"] == "attn":
        n_q, n_kv = c["n_q"], c["n_kv"]
        k4, kp = _pack(*_to_nibbles(_randn((n_kv, c["max_pos"], D), g).bfloat16()))
        v4, vp = _pack(*_to_nibbles(_randn((n_kv, c["max_pos"], D), g).bfloat16()))
        # scratch that a program allocates once, zeroed: room for the partial results of 160 splits
        ws = torch.zeros(4096 + 4 * n_kv + 520 * n_q * (160 // n_kv + 1), dtype=torch.uint8, device="cuda")
        return dict(case=c, qkv=_randn(((n_q + 2 * n_kv) * D,), g, 1.5), qn=_randn((D,), g, 0.02, 1.0).bfloat16(),
                    kn=_randn((D,), g, 0.02, 1.0).bfloat16(), k4=k4, v4=v4, kp=kp, vp=vp, ws=ws,
                    out=torch.empty(n_q * D, device="cuda"), row=torch.empty((2, n_kv, D), device="cuda"))
    if c["op"] == "store":
        shape = (c["n_kv"], c["max_pos"], D)
        byte = lambda: torch.zeros((c["n_kv"], c["max_pos"], 64), dtype=torch.uint8, device="cuda")
        par = lambda: torch.zeros((c["n_kv"], c["max_pos"], 2, 2), dtype=torch.bfloat16, device="cuda")
        return dict(case=c, k=_randn(shape, g).bfloat16(), v=_randn(shape, g).bfloat16(), k4=byte(), v4=byte(),
                    kp=par(), vp=par(), k_out=torch.zeros(shape, dtype=torch.bfloat16, device="cuda"),
                    v_out=torch.zeros(shape, dtype=torch.bfloat16, device="cuda"))
    z = _randn((c["rows"], c["n_cb"] * c["V"]), g, 2.5)
    if c["V"] > 64:  # the pad entry before the last is forbidden, as a caller's mask leaves it
        z.view(c["rows"], c["n_cb"], c["V"])[:, :, c["V"] - 2] = -math.inf
    codes = torch.randint(0, c["V"] - 2 if c["V"] > 64 else c["V"], (c["rows"], c["n_cb"]), generator=g,
                          device="cuda", dtype=torch.int32)
    return dict(case=c, z=z, codes=codes)


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _to_nibbles(rows):
    """bf16 [..., 128] -> nibbles [..., 2, 64], scale and minimum [..., 2] (bf16 values in fp32)."""
    x = rows.float().unflatten(-1, (2, 64))
    lo, hi = x.amin(-1), x.amax(-1)
    s = ((hi - lo) / 15).bfloat16().float()
    u = ((x - lo.unsqueeze(-1)) / s.unsqueeze(-1)).round().clamp(0, 15)
    return torch.where(s.unsqueeze(-1) > 0, u, torch.zeros_like(u)).to(torch.uint8), s, lo


def _pack(u, s, lo):
    u = u.unflatten(-1, (8, 4, 2))  # [..., half, unit, byte, nibble]
    b = (u[..., 0] | (u[..., 1] << 4)).transpose(-3, -2)  # [..., unit, half, byte]
    return b.flatten(-3).contiguous(), torch.stack((s, lo), -1).bfloat16()


def _from_cache(b, par):
    """[..., 64] bytes and [..., 2, 2] parameters -> the fp32 values [..., 128]."""
    b = b.unflatten(-1, (8, 2, 4)).transpose(-3, -2)
    u = torch.stack((b & 15, b >> 4), -1).flatten(-3).float()  # [..., half, 64]
    p = par.float()
    return (p[..., 1:] + p[..., :1] * u).flatten(-2)


def _plain_gemv(st):
    c = st["case"]
    u = torch.stack((st["w4"] & 15, st["w4"] >> 4), -1).float() - 8
    w = (u.view(-1, c["K"] // 128, 128) * st["s"].float().unsqueeze(-1)).view(-1, c["K"])
    x = st["x"]
    if c["norm"]:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * st["gamma"].float()
    y = x @ w.t()
    if c["epi"] == 1:
        y = st["resid"] + y
    if c["epi"] == 2:
        gate, up = y[:, :c["N"]], y[:, c["N"]:]
        y = gate / (1 + torch.exp(-gate)) * up
    return y


def _norm_rope(x, gain, pos):
    """x [heads][128] in the type that it comes in, normalised and rotated to position pos."""
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * gain.to(x.dtype)
    i = torch.arange(64, dtype=torch.float64, device=x.device)
    ang = pos * THETA ** (-2 * i / D)
    cos, sin = torch.cos(ang).to(x.dtype), torch.sin(ang).to(x.dtype)
    a, b = n[:, :64], n[:, 64:]
    return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)


def _plain_attn(st):
    c = st["case"]
    n_q, n_kv, pos = c["n_q"], c["n_kv"], c["pos"]
    x = st["qkv"].view(-1, D)
    q = _norm_rope(x[:n_q], st["qn"], pos)
    # the new key decides 4-bit codes, which lie next to borders: in 64 bits until it is rounded to bf16
    k_new = _norm_rope(x[n_q:n_q + n_kv].double(), st["kn"], pos).bfloat16()
    v_new = x[n_q + n_kv:].bfloat16()
    for new, b, p in ((k_new, st["k4"], st["kp"]), (v_new, st["v4"], st["vp"])):
        b[:, pos], p[:, pos] = _pack(*_to_nibbles(new))
    k = _from_cache(st["k4"][:, :pos + 1], st["kp"][:, :pos + 1])
    v = _from_cache(st["v4"][:, :pos + 1], st["vp"][:, :pos + 1])
    z = q.view(n_kv, n_q // n_kv, D) @ k.transpose(1, 2) / math.sqrt(D)
    e = torch.exp(z - z.amax(-1, keepdim=True))
    out = (e @ v) / e.sum(-1, keepdim=True)
    return {"out": out.reshape(-1), "row": torch.stack((k[:, pos], v[:, pos]))}


def _plain_store(st):
    c = st["case"]
    res = []
    for src, b, p, dst in ((st["k"], st["k4"], st["kp"], st["k_out"]), (st["v"], st["v4"], st["vp"], st["v_out"])):
        b[:, c["p0"]:c["p1"]], p[:, c["p0"]:c["p1"]] = _pack(*_to_nibbles(src[:, c["p0"]:c["p1"]]))
        dst[:, c["p0"]:c["p1"]] = _from_cache(b[:, c["p0"]:c["p1"]], p[:, c["p0"]:c["p1"]]).bfloat16()
        res.append(dst)
    return res


def _plain_score(st):
    c = st["case"]
    z = st["z"].view(c["rows"], c["n_cb"], c["V"])
    t = z / c["T"]
    m = t.amax(-1, keepdim=True)
    e = torch.exp(t - m)
    total = e.sum(-1, keepdim=True)
    lse = m + torch.log(total)
    lp = t - lse
    ent = -(e / total * torch.where(e > 0, lp, torch.zeros_like(lp))).sum(-1)
    at = torch.sort(z, dim=-1, descending=True, stable=True).indices[..., :c["top"]]
    return {"logprob": lp.gather(-1, st["codes"].long().unsqueeze(-1)).squeeze(-1), "entropy": ent,
            "top": at.int(), "top_logprob": lp.gather(-1, at)}


def run(state):
    st, c = state, state["case"]
    if own:
        import ar_decode_step_gb300 as ads
        if c["op"] == "gemv":
            ads.gemv_w4(st["x"], st["w4"], st["s"], st["y"], epi=c["epi"], resid_dev=st["resid"],
                        gamma_dev=st["gamma"], eps=EPS)
            return st["y"]
        if c["op"] == "attn":
            ads.attention_decode_kv4(st["qkv"], st["qn"], st["kn"], st["k4"], st["v4"], st["kp"], st["vp"],
                                     st["out"], c["n_q"], c["n_kv"], c["pos"], st["ws"], kv_row=st["row"],
                                     eps=EPS, rope_theta=THETA)
            return {"out": st["out"], "row": st["row"]}
        if c["op"] == "store":
            ads.quantize_kv4(st["k"], st["v"], st["k4"], st["v4"], st["kp"], st["vp"], c["p0"], c["p1"])
            ads.dequantize_kv4(st["k4"], st["v4"], st["kp"], st["vp"], st["k_out"], st["v_out"], c["p0"], c["p1"])
            return [st["k_out"], st["v_out"]]
        lp, ent, at, at_lp = ads.code_logprobs(st["z"], st["codes"], c["V"], top=c["top"], temperature=c["T"])
        return {"logprob": lp, "entropy": ent, "top": at, "top_logprob": at_lp}
    return {"gemv": _plain_gemv, "attn": _plain_attn, "store": _plain_store, "score": _plain_score}[c["op"]](st)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_row(x):
    """One half row [..., 64] of bf16 values (held in fp64) as its 4-bit code stands for it."""
    lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    s = ((hi - lo) / 15).to(torch.bfloat16).double()
    u = torch.clamp(torch.round((x - lo) / torch.where(s > 0, s, torch.ones_like(s))), 0, 15)
    return lo + torch.where(s > 0, u * s, torch.zeros_like(u))


def _exact_rows(rows):
    x = rows.double()
    return torch.cat((_exact_row(x[..., :64]), _exact_row(x[..., 64:])), -1)


def _exact_cached(b, par):
    """Cache rows channel by channel: channel c of half h sits in byte 8 (c // 8) + 4 h + (c % 8) // 2."""
    ch = torch.arange(D, device=b.device)
    h, i = ch // 64, ch % 64
    byte = b[..., 8 * (i // 8) + 4 * h + (i % 8) // 2].int()
    u = (byte >> (4 * (i % 2)).int()) & 15
    return par[..., 1].double()[..., h] + par[..., 0].double()[..., h] * u.double()


def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["op"] == "gemv":
        x = st["x"].double()
        if c["norm"]:
            x = x * torch.rsqrt(x.pow(2).sum(-1, keepdim=True) / c["K"] + EPS) * st["gamma"].double()
        acc = torch.empty((c["M"], st["w4"].shape[0]), dtype=torch.float64, device="cuda")
        for r in range(0, st["w4"].shape[0], 4096):  # a block of rows at a time
            b, s = st["w4"][r:r + 4096], st["s"][r:r + 4096].double().repeat_interleave(64, dim=1)
            even, odd = (b % 16).double() - 8, (b // 16).double() - 8
            acc[:, r:r + 4096] = x[:, 0::2] @ (even * s).t() + x[:, 1::2] @ (odd * s).t()
        if c["epi"] == 1:
            return acc + st["resid"].double()
        if c["epi"] == 2:
            gate, up = acc[:, :c["N"]], acc[:, c["N"]:]
            return gate * torch.sigmoid(gate) * up
        return acc
    if c["op"] == "attn":
        n_q, n_kv, pos = c["n_q"], c["n_kv"], c["pos"]
        x = st["qkv"].double().view(-1, D)
        j = torch.arange(64, dtype=torch.float64, device="cuda")
        rot = torch.polar(torch.ones_like(j), pos * torch.exp(-(j / 64) * math.log(THETA)))

        def turned(rows, gain):
            y = rows * torch.rsqrt(rows.pow(2).sum(-1, keepdim=True) / D + EPS) * gain.double()
            z = torch.complex(y[:, :64].contiguous(), y[:, 64:].contiguous()) * rot
            return torch.cat((z.real, z.imag), -1)

        q = turned(x[:n_q], st["qn"])
        k1 = _exact_rows(turned(x[n_q:n_q + n_kv], st["kn"]).to(torch.bfloat16))
        v1 = _exact_rows(x[n_q + n_kv:].float().to(torch.bfloat16))
        outs = []
        for h in range(n_kv):
            k = torch.cat((_exact_cached(st["k4"][h, :pos], st["kp"][h, :pos]), k1[h:h + 1]))
            v = torch.cat((_exact_cached(st["v4"][h, :pos], st["vp"][h, :pos]), v1[h:h + 1]))
            g = n_q // n_kv
            outs.append(torch.softmax(q[h * g:(h + 1) * g] @ k.t() / math.sqrt(D), -1) @ v)
        return {"out": torch.cat(outs).reshape(-1), "row": torch.stack((k1, v1))}
    if c["op"] == "store":
        res = []
        for src in (st["k"], st["v"]):
            y = torch.zeros(src.shape, dtype=torch.float64, device="cuda")
            y[:, c["p0"]:c["p1"]] = _exact_rows(src[:, c["p0"]:c["p1"]])
            res.append(y)
        return res
    z = st["z"].double().view(c["rows"], c["n_cb"], c["V"])
    lp = torch.log_softmax(z / c["T"], -1)
    p = lp.exp()
    ent = torch.where(p > 0, -p * lp, torch.zeros_like(p)).sum(-1)
    best = torch.sort(z, dim=-1, descending=True, stable=True).indices[..., :c["top"]]
    return {"logprob": lp.gather(-1, st["codes"].long().unsqueeze(-1)).squeeze(-1), "entropy": ent,
            "top": best.int(), "top_logprob": lp.gather(-1, best)}
