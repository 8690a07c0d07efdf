"""Measured cases of two operators of the layer around the attention.

norm_rope   RMS norm of every query and key head, with the position rotation in the same pass: forward
            (`sagesla_qk_norm_rope`) and backward (`sagesla_qk_norm_rope_bwd`).
w8a8_token  linear layer in 8-bit integers, one scale per token of x and per output channel of W
            (`sagesla_w8a8_token_linear`; the weight is quantised once by `sagesla_w8a8_token_quant`).
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


def listed():
    return [
        # one new token of four sequences, anywhere in a long context, grouped key heads
        _rope("rope_step_b4_h40_8", False, "bf16", 4, 1, 40, 8, 128, 128, False, "tokens", 131072, False),
        # two padded prompts, a quarter of the channels rotated, fp16
        _rope("rope_prompt_b2_n1000_d64_fp16", False, "fp16", 2, 1000, 16, 4, 64, 16, False, "tokens", 4096, False),
        # the 1.3B video model at 480p: from the fused projection's rows to the attention's head-major tensors
        _rope("rope_480p_h12", False, "bf16", 1, 32760, 12, 12, 128, 128, True, "index", 32760, True),
        # the 14B video model at 720p, the token-major form
        _rope("rope_720p_h40", False, "bf16", 1, 75600, 40, 40, 128, 128, True, "index", 75600, False),
        # training in fp32: odd length, wide heads, grouped key heads, padded rows
        _rope("rope_bwd_b3_n577_d256_fp32", True, "fp32", 3, 577, 8, 2, 256, 128, False, "tokens", 1024, False),
        # training of the 1.3B video model at 480p
        _rope("rope_bwd_480p_h12", True, "bf16", 1, 32760, 12, 12, 128, 128, True, "index", 32760, True),
        # one token (a timestep's embedding through a projection of the 14B model)
        _w8a8("w8a8_m1_5120", "bf16", 1, 5120, 5120, True),
        # a few tokens into the feed-forward width of the 14B model
        _w8a8("w8a8_m24_ffn_fp16", "fp16", 24, 13824, 5120, True),
        # odd sizes: an output width that is no multiple of anything
        _w8a8("w8a8_m333_n1001_k1280", "fp16", 333, 1001, 1280, True),
        # a small clip's tokens through a projection of the 14B model
        _w8a8("w8a8_m1024_5120", "bf16", 1024, 5120, 5120, False),
        # 480p tokens at the 1.3B model's width
        _w8a8("w8a8_480p_1536", "bf16", 32760, 1536, 1536, True),
        # 720p tokens at the 14B model's width
        _w8a8("w8a8_720p_5120", "bf16", 75600, 5120, 5120, False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    if rng.random() < 0.5:
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


def prepare(case, seed):
    s = _prepare_w8a8(case, seed) if case["op"] == "w8a8_token" else _prepare_rope(case, seed)
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


def run(state):
    return _run_w8a8(state) if state["case"]["op"] == "w8a8_token" else _run_rope(state)


def work(case):
    c, e = case, SIZE[case["dtype"]]
    if c["op"] == "w8a8_token":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": M * K * e + N * K + 4 * N + (e * N if c["bias"] else 0) + M * N * e, "flops": 2 * M * N * K}
    tokens = c["B"] * c["N"]
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


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_w8a8(s) if case["op"] == "w8a8_token" else _exact_rope(case, s)
