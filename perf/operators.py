"""Measured cases of three operators of the layer around the attention.

norm_rope     RMS norm of every query and key head, with the position rotation in the same pass: forward
              (`sagesla_qk_norm_rope`) and backward (`sagesla_qk_norm_rope_bwd`).
w8a8_token    linear layer in 8-bit integers, one scale per token of x and per output channel of W
              (`sagesla_w8a8_token_linear`; the weight is quantised once by `sagesla_w8a8_token_quant`).
linear_decay  causal linear attention with a decay for each head: whole prompts (`sagesla_linear_decay`) and single
              tokens (`sagesla_linear_decay_step`).
"""
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6
POSITIONS = ("index", "tokens")  # the token index itself, or a position of each token (negative: padding)


def _rope(name, back, dtype, B, N, Hq, Hk, d, rot, interleaved, pos, T, head_major):
    return {"name": name, "op": "norm_rope_bwd" if back else "norm_rope", "dtype": dtype, "B": B, "N": N, "Hq": Hq,
            "Hk": Hk, "d": d, "rot": rot, "interleaved": interleaved, "pos": pos, "T": T, "head_major": head_major}


def _w8a8(name, dtype, M, N, K, bias):
    return {"name": name, "op": "w8a8_token", "dtype": dtype, "M": M, "N": N, "K": K, "bias": bias}


def _decay(name, step, B, N, H, Hk, d, padded, head_major):
    return {"name": name, "op": "linear_decay_step" if step else "linear_decay", "dtype": "bf16", "B": B, "N": N, "H": H,
            "Hk": Hk, "d": d, "padded": padded, "head_major": head_major}


def listed():
    return [
        # one new token of four sequences, anywhere in a long context, grouped key heads
        _rope("rope_step_b4_h40_8", False, "bf16", 4, 1, 40, 8, 128, 128, False, "tokens", 131072, False),
        # two prompts, one of them padded, a quarter of the channels rotated, fp16
        _rope("rope_prompt_b2_n1000_d64_fp16", False, "fp16", 2, 1000, 16, 4, 64, 16, False, "tokens", 4096, False),
        # the 14B video model at 720p, the token-major form
        _rope("rope_720p_h40", False, "bf16", 1, 75600, 40, 40, 128, 128, True, "index", 75600, False),
        # training of the 1.3B video model at 480p
        _rope("rope_bwd_480p_h12", True, "bf16", 1, 32760, 12, 12, 128, 128, True, "index", 32760, True),
        # one token (a timestep's embedding through a projection of the 14B model)
        _w8a8("w8a8_m1_5120", "bf16", 1, 5120, 5120, True),
        # odd sizes: an output width that is no multiple of anything
        _w8a8("w8a8_m333_n1001_k1280_fp16", "fp16", 333, 1001, 1280, True),
        # a small clip's tokens through a projection of the 14B model
        _w8a8("w8a8_m1024_5120", "bf16", 1024, 5120, 5120, False),
        # 720p tokens at the 14B model's width
        _w8a8("w8a8_720p_5120", "bf16", 75600, 5120, 5120, False),
        # one new token of one sequence, and of a batch of 64
        _decay("decay_step_b1_h40", True, 1, 1, 40, 40, 128, False, False),
        _decay("decay_step_b64_h40", True, 64, 1, 40, 40, 128, False, False),
        # three prompts of different lengths behind an earlier state, grouped key heads
        _decay("decay_prompt_b3_n1000_d64", False, 3, 1000, 16, 4, 64, True, False),
        # a 480p clip's tokens as one causal sequence, the attention's head-major tensors
        _decay("decay_480p_h12", False, 1, 32760, 12, 12, 128, False, True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm_rope", "w8a8_token", "linear_decay"])
    if op == "norm_rope":
        d = rng.choice([32, 64, 80, 128, 128, 256])
        rot = rng.choice([d, d, d // 32 * 16, 16])
        Hk = rng.choice([1, 2, 4, 8, 12])
        Hq = Hk * rng.choice([1, 1, 2, 5])
        B = rng.randint(1, 4)
        most = 75600 * 80 * 128 // (B * (Hq + Hk) * d * 4)
        N = _log(rng, 1, min(32760, most))
        pos = rng.choice(POSITIONS)
        T = N if pos == "index" else _log(rng, max(N, 64), 131072)
        return _rope("", rng.random() < 0.5, rng.choice(sorted(DTYPES)), B, N, Hq, Hk, d, rot, rng.random() < 0.5,
                     pos, T, rng.random() < 0.5)
    if op == "linear_decay":
        d = rng.choice([64, 128, 128])
        Hk = rng.choice([1, 2, 4, 8, 12])
        H = Hk * rng.choice([1, 1, 1, 4])
        step = rng.random() < 0.4
        B = _log(rng, 1, 64) if step else rng.randint(1, 4)
        N = 1 if step else _log(rng, 1, int(32760 * min(1.0, (12 / (B * H)) ** 0.5)))
        return _decay("", step, B, N, H, Hk, d, not step and rng.random() < 0.5, rng.random() < 0.5)
    N, K = _log(rng, 64, 13824), 16 * _log(rng, 8, 320)
    M = _log(rng, 1, min(32760, 75600 * 5120 * 5120 // (N * K)))
    return _w8a8("", rng.choice(["bf16", "fp16"]), M, N, K, rng.random() < 0.5)


# ------------------------------------------------------------------- inputs --
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _table(T, rot):
    """cos and sin of t * 10000^(-2c/rot), angles in 64 bits, kept in fp32."""
    f = torch.pow(10000.0, -torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    a = torch.arange(T, device="cuda", dtype=torch.float64)[:, None] * f[None]
    return a.cos().float(), a.sin().float()


def _prepare_rope(c, seed):
    g = _gen(seed)
    t = DTYPES[c["dtype"]]
    B, N, Hq, Hk, d = c["B"], c["N"], c["Hq"], c["Hk"], c["d"]
    width = (Hq + 2 * Hk) * d
    qkv = torch.randn(B, N, width, device="cuda", generator=g, dtype=t)  # rows of a fused projection
    qkv *= torch.rand(width, device="cuda", generator=g).mul_(2).add_(0.1).to(t)
    s = {"q": qkv[..., :Hq * d].unflatten(-1, (Hq, d)), "k": qkv[..., Hq * d:(Hq + Hk) * d].unflatten(-1, (Hk, d))}
    s["gq"] = (1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(t)
    s["gk"] = (1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(t)
    s["cos"], s["sin"] = _table(c["T"], c["rot"])
    s["pos"] = None
    if c["pos"] == "tokens":  # consecutive positions from an offset; a padded tail in every second sequence
        first = torch.randint(0, c["T"] - N + 1, (B, 1), device="cuda", generator=g)
        n = torch.arange(N, device="cuda")
        length = torch.full((B, 1), N, device="cuda")
        length[1::2] = max(1, N * 3 // 4)
        s["pos"] = torch.where(n < length, first + n, -1).to(torch.int32)
    if c["op"] == "norm_rope_bwd":
        def grad(H):
            if c["head_major"]:
                return torch.randn(B, H, N, d, device="cuda", generator=g, dtype=t).transpose(1, 2)
            return torch.randn(B, N, H, d, device="cuda", generator=g, dtype=t)
        s["dqo"], s["dko"] = grad(Hq), grad(Hk)
    return s


def _quant_rows(w):
    """Codes (int8) and fp32 scales of the rows of w: scale amax/127, code RNE(x * (127/amax)); a row without a
    value of at least 2^-100 has scale 1 and codes 0."""
    x = w.float()
    amax = x.abs().amax(1)
    some = amax >= 2.0 ** -100
    mult = torch.where(some, 127.0 / amax, 0.0)
    scale = torch.where(some, amax / 127.0, 1.0)
    return (x * mult[:, None]).round_().clamp_(-127, 127), scale


def _prepare_w8a8(c, seed):
    g = _gen(seed)
    t = DTYPES[c["dtype"]]
    M, N, K = c["M"], c["N"], c["K"]
    x = torch.randn(M, K, device="cuda", generator=g, dtype=t)
    x *= torch.rand(K, device="cuda", generator=g).mul_(3).add_(0.1).to(t)  # channels of different ranges
    codes, sw = _quant_rows(torch.randn(N, K, device="cuda", generator=g) / K ** 0.5)
    bias = torch.randn(N, device="cuda", generator=g).to(t) if c["bias"] else None
    return {"x": x, "wq": codes.to(torch.int8), "sw": sw, "bias": bias}


def _prepare_decay(c, seed):
    g = _gen(seed)
    B, N, H, Hk, d = c["B"], c["N"], c["H"], c["Hk"], c["d"]

    def rows(heads):  # normalised rows, as a norm of each head leaves them
        if c["head_major"]:
            return torch.randn(B, heads, N, d, device="cuda", generator=g, dtype=torch.bfloat16).transpose(1, 2)
        return torch.randn(B, N, heads, d, device="cuda", generator=g, dtype=torch.bfloat16)
    s = {"q": rows(H), "k": rows(Hk), "v": rows(Hk)}
    # slopes from 2^(-8/H) per token (the last tokens alone) to 2^-8 (hundreds of tokens)
    s["log_decay"] = -torch.pow(2.0, -8.0 * torch.arange(1, H + 1, device="cuda", dtype=torch.float32) / H)
    s["scale"] = d ** -0.5
    s["state"] = 3 * torch.randn(B, H, d, d, device="cuda", generator=g)
    s["state_out"] = torch.empty_like(s["state"])  # a user keeps two states, or gives the same one twice
    s["lens"] = None
    if c["padded"]:
        s["lens"] = torch.tensor([N] + [max(0, N * 3 // 4 - 100 * i) for i in range(1, B)], device="cuda", dtype=torch.int32)
    if c["op"] == "linear_decay_step":
        s.update({n: s[n][:, 0] for n in "qkv"})
    return s


def prepare(case, seed):
    make = {"w8a8_token": _prepare_w8a8, "linear_decay": _prepare_decay, "linear_decay_step": _prepare_decay}
    s = make.get(case["op"], _prepare_rope)(case, seed)
    s["case"] = case
    return s


# ----------------------------------------------------------------- one pass --
def _token_tables(c, s):
    """cos, sin [B or 1, N, 1, rot/2] and, with padding, which tokens are real [B, N, 1, 1]."""
    if s["pos"] is None:
        return s["cos"][None, :c["N"], None], s["sin"][None, :c["N"], None], None
    p = s["pos"].clamp(min=0).long()
    return s["cos"][p][:, :, None], s["sin"][p][:, :, None], (s["pos"] >= 0)[:, :, None, None]


def _pairs(x, rot, interleaved):
    r = x[..., :rot]
    return (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])


def _unpair(a, b, rest, interleaved):
    r = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((r, rest), -1)


def _rope_plain(c, x, gamma, cos, sin, real):
    f = x.float()
    y = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS) * gamma.float()
    a, b = _pairs(y, c["rot"], c["interleaved"])
    y = _unpair(a * cos - b * sin, a * sin + b * cos, y[..., c["rot"]:], c["interleaved"])
    if real is not None:
        y = torch.where(real, y, 0.0)
    y = y.to(x.dtype)
    return y.transpose(1, 2).contiguous() if c["head_major"] else y


def _rope_bwd_plain(c, dy, x, gamma, cos, sin, real):
    f, g = x.float(), dy.float()
    if real is not None:
        g = torch.where(real, g, 0.0)
    a, b = _pairs(g, c["rot"], c["interleaved"])
    g = _unpair(a * cos + b * sin, b * cos - a * sin, g[..., c["rot"]:], c["interleaved"])
    r = torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS)
    xh = f * r
    dgamma = (g * xh).sum((0, 1, 2), dtype=torch.float64).float()
    u = g * gamma.float()
    return (r * (u - xh * (u * xh).mean(-1, keepdim=True))).to(x.dtype), dgamma


def _run_rope(s):
    c = s["case"]
    if own:
        import sparse_bit_attention_smoothing_b200 as sg
        if c["op"] == "norm_rope":
            return sg.sagesla_qk_norm_rope(s["q"], s["k"], s["gq"], s["gk"], s["cos"], s["sin"], pos=s["pos"], eps=EPS,
                                           interleaved=c["interleaved"], head_major=c["head_major"])
        return sg.sagesla_qk_norm_rope_bwd(s["dqo"], s["dko"], s["q"], s["k"], s["gq"], s["gk"], s["cos"], s["sin"],
                                           pos=s["pos"], eps=EPS, interleaved=c["interleaved"])
    t = _token_tables(c, s)
    if c["op"] == "norm_rope":
        return _rope_plain(c, s["q"], s["gq"], *t), _rope_plain(c, s["k"], s["gk"], *t)
    dq, dgq = _rope_bwd_plain(c, s["dqo"], s["q"], s["gq"], *t)
    dk, dgk = _rope_bwd_plain(c, s["dko"], s["k"], s["gk"], *t)
    return dq, dk, dgq, dgk


def _run_w8a8(s):
    if own:
        import sparse_bit_attention_smoothing_b200 as sg
        return sg.sagesla_w8a8_token_linear(s["x"], s["wq"], s["sw"], bias=s["bias"])
    codes, sx = _quant_rows(s["x"])
    y = (codes @ s["wq"].float().t()) * sx[:, None] * s["sw"]
    if s["bias"] is not None:
        y += s["bias"].float()
    return y.to(s["x"].dtype)


CHUNK = 128  # tokens that the plain form takes together


def _step_plain(c, s):
    G = c["H"] // c["Hk"]
    q, k, v = s["q"].float(), s["k"].float().repeat_interleave(G, 1), s["v"].float().repeat_interleave(G, 1)
    state = s["state"] * torch.exp(s["log_decay"])[:, None, None] + k[..., :, None] * v[..., None, :]
    out = s["scale"] * (q[..., None, :] @ state)[..., 0, :]
    return out.to(s["q"].dtype), state


def _decay_plain(c, s):
    """Chunks of 128 tokens: products within a chunk, and the sums of earlier chunks by one product over chunks."""
    B, N, H, d, G = c["B"], c["N"], c["H"], c["d"], c["H"] // c["Hk"]
    C, nc = CHUNK, -(-N // CHUNK)
    lens = s["lens"].long() if s["lens"] is not None else torch.full((B,), N, device="cuda")
    real = (torch.arange(nc * C, device="cuda") < lens[:, None])[:, None, :, None]

    def chunks(x, heads):  # [B, H, nc, C, d] in 32 bits, rows past a sequence's end 0
        x = x.float().transpose(1, 2).repeat_interleave(heads, 1)
        return torch.where(real, torch.nn.functional.pad(x, (0, 0, 0, nc * C - N)), 0.0).unflatten(2, (nc, C))
    q, k, v = chunks(s["q"], 1), chunks(s["k"], G), chunks(s["v"], G)
    g = s["log_decay"].double()[:, None, None]
    i = torch.arange(C, device="cuda", dtype=torch.float64)
    j = torch.arange(nc, device="cuda", dtype=torch.float64)
    diff = i[:, None] - i[None]
    within = torch.where(diff >= 0, torch.exp(g * diff.clamp(min=0)), 0.0).float()[:, None]  # [H, 1, C, C]
    out = ((q @ k.transpose(-1, -2)) * within) @ v
    to_end = torch.exp(g[..., 0] * (C - 1 - i)).float()[:, None, :, None]
    sums = ((k * to_end).transpose(-1, -2) @ v).flatten(3)  # what each chunk adds to the state, [B, H, nc, d*d]
    gap = j[:, None] - j[None] - 1
    across = torch.where(gap >= 0, torch.exp(g * C * gap.clamp(min=0)), 0.0).float()  # [H, nc, nc]
    state = across @ sums + torch.exp(g[..., 0] * C * j).float()[..., None] * s["state"].flatten(2)[:, :, None]
    out += (q * torch.exp(g[..., 0] * (i + 1)).float()[:, None, :, None]) @ state.unflatten(3, (d, d))
    out = (s["scale"] * out).flatten(2, 3)[:, :, :N].to(s["q"].dtype)
    # the state behind a sequence's last token: its chunk's start, and the chunk's own tokens decayed to that token
    last = torch.div(lens.clamp(min=1) - 1, C, rounding_mode="floor")
    n = (lens - last * C).double()[:, None, None]  # tokens of the last chunk
    b = torch.arange(B, device="cuda")
    weight = torch.where(i < n, torch.exp(g[..., 0] * (n - 1 - i).clamp(min=0)), 0.0).float()  # [B, H, C]
    end = torch.exp(g[..., 0] * n).float()[..., None] * state.unflatten(3, (d, d))[b, :, last]
    end = end + (k[b, :, last] * weight[..., None]).transpose(-1, -2) @ v[b, :, last]
    return (out if c["head_major"] else out.transpose(1, 2)), end


def _run_decay(s):
    c = s["case"]
    if own:
        import sparse_bit_attention_smoothing_b200 as sg
        if c["op"] == "linear_decay_step":
            return sg.sagesla_linear_decay_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], scale=s["scale"],
                                                state_out=s["state_out"])
        return sg.sagesla_linear_decay(s["q"], s["k"], s["v"], s["log_decay"], s["state"], lens=s["lens"],
                                       scale=s["scale"], state_out=s["state_out"], head_major=c["head_major"])
    return _step_plain(c, s) if c["op"] == "linear_decay_step" else _decay_plain(c, s)


def run(state):
    op = state["case"]["op"]
    return _run_w8a8(state) if op == "w8a8_token" else _run_decay(state) if op.startswith("linear") else _run_rope(state)


def work(case):
    c, e = case, SIZE[case["dtype"]]
    if c["op"] == "w8a8_token":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": M * K * e + N * K + 4 * N + (e * N if c["bias"] else 0) + M * N * e, "flops": 2 * M * N * K}
    tokens = c["B"] * c["N"]
    if c["op"].startswith("linear"):
        d, H = c["d"], c["H"]
        moved = tokens * (2 * H + 2 * c["Hk"]) * d * e + 2 * c["B"] * H * d * d * 4 + 4 * H
        # a token: its product with the state and its outer product, 2 d^2 each
        return {"bytes": moved, "flops": 4 * tokens * H * d * d}
    rows = tokens * (c["Hq"] + c["Hk"])
    back = c["op"] == "norm_rope_bwd"
    table = min(c["T"], tokens) * c["rot"] * 4
    small = 2 * c["d"] * (e + (4 if back else 0)) + (4 * tokens if c["pos"] == "tokens" else 0)
    return {"bytes": rows * c["d"] * e * (3 if back else 2) + table + small, "flops": rows * c["d"] * (20 if back else 10)}


# ------------------------------------------------------------------ 64 bits --
def _turn(c, s, x, sign):
    """x (64 bits, [B, N, H, d]) with its first rot channels turned by the tokens' angles (sign -1: back)."""
    B, N, H = x.shape[:3]
    half, rot = c["rot"] // 2, c["rot"]
    w = torch.complex(s["cos"].double(), sign * s["sin"].double())
    w = w[:N].expand(B, N, half) if s["pos"] is None else w[s["pos"].clamp(min=0).long()]
    z = x[..., :rot].reshape(B, N, H, half, 2) if c["interleaved"] else x[..., :rot].reshape(B, N, H, 2, half).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * w[:, :, None])
    z = z if c["interleaved"] else z.transpose(-1, -2)
    return torch.cat((z.reshape(B, N, H, rot), x[..., rot:]), -1)


def _exact_rope(c, s):
    out, grads = [], []
    for x, gamma, dy in ((s["q"], s["gq"], s.get("dqo")), (s["k"], s["gk"], s.get("dko"))):
        x, gamma = x.double(), gamma.double()
        rms = (x.pow(2).sum(-1, keepdim=True) / c["d"] + EPS).sqrt()
        pad = None if s["pos"] is None else (s["pos"] < 0)[:, :, None, None]
        if dy is None:
            y = _turn(c, s, x / rms * gamma, 1)
            y = y if pad is None else y.masked_fill(pad, 0)
            out.append(y.transpose(1, 2).contiguous() if c["head_major"] else y)
            continue
        g = _turn(c, s, dy.double(), -1)
        g = g if pad is None else g.masked_fill(pad, 0)
        n = x / rms
        grads.append((g * n).sum((0, 1, 2)))
        g = g * gamma
        out.append((g - n * ((g * n).sum(-1, keepdim=True) / c["d"])) / rms)
    return tuple(out + grads)


def _exact_w8a8(s):
    x = s["x"].double()
    amax = x.abs().amax(1, keepdim=True)
    none = amax < 2.0 ** -100
    # the operator's definition rounds the multiplier, the product and the scale to fp32
    mult = (127.0 / amax).masked_fill(none, 0.0).float().double()
    codes = (x * mult).float().double().round().clamp(-127, 127)
    y = codes @ s["wq"].double().t()
    y *= (amax / 127.0).float().double().masked_fill(none, 1.0)
    y *= s["sw"].double()
    return y if s["bias"] is None else y + s["bias"].double()


def _exact_decay(c, s):
    """The sum over all earlier tokens, a block of queries at a time (quadratic in the length)."""
    step = c["op"] == "linear_decay_step"
    q, k, v = (s[n].double() if step else s[n].double().transpose(1, 2) for n in "qkv")
    if step:
        q, k, v = q[:, :, None], k[:, :, None], v[:, :, None]
    B, N, H, G = c["B"], c["N"], c["H"], c["H"] // c["Hk"]
    k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    g, S0 = s["log_decay"].double(), s["state"].double()
    out, end = torch.zeros_like(q), torch.empty_like(S0)
    for b in range(B):
        n = N if s["lens"] is None else int(s["lens"][b])
        t = torch.arange(n, device="cuda", dtype=torch.float64)
        for i in range(0, n, 512):
            e = min(n, i + 512)
            age = t[i:e, None] - t[None, :e]
            w = q[b, :, i:e] @ k[b, :, :e].transpose(-1, -2)
            w *= torch.exp(g[:, None, None] * age.clamp(min=0)).masked_fill_(age < 0, 0)
            old = torch.exp(g[:, None] * (t[i:e] + 1))[..., None] * (q[b, :, i:e] @ S0[b])
            out[b, :, i:e] = s["scale"] * (w @ v[b, :, :e] + old)
        left = torch.exp(g[:, None] * (n - 1 - t))[..., None] * k[b, :, :n]
        end[b] = left.transpose(-1, -2) @ v[b, :, :n] + torch.exp(g * n)[:, None, None] * S0[b]
    return (out[:, :, 0] if step else out if c["head_major"] else out.transpose(1, 2)), end


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("linear"):
        return _exact_decay(case, s)
    return _exact_w8a8(s) if case["op"] == "w8a8_token" else _exact_rope(case, s)
