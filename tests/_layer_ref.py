"""Plain 64-bit implementations of the operators around the attention (norm
and rotation of query and key heads, W8A8 with a scale per token and channel,
linear attention with a decay), and what their tests compare by."""
import numpy as np
import torch

U32 = 2.0 ** -24  # a rounding in fp32 is off by at most this, relative


def half_step(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    """Half of the type's smallest step (what a rounding may be off near zero)."""
    return torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2


def inside(got, ref, tol, what=""):
    got, ref, tol = got.double().cpu(), ref.double().cpu(), tol.double().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    off = torch.where(torch.isnan(ref), 0.0, (got - ref).abs() - tol)
    worst = float(off.max())
    assert worst <= 0, f"{what}: {int((off > 0).sum())} of {off.numel()} beyond the bound, worst by {worst:.3e}"


# ------------------------------------------------------- norm and rotation --
def _split(x, rot, il):
    r = x[..., :rot]
    return (r[..., 0::2], r[..., 1::2]) if il else (r[..., :rot // 2], r[..., rot // 2:])


def _join(a, b, x, rot, il):
    r = torch.stack((a, b), -1).flatten(-2) if il else torch.cat((a, b), -1)
    return torch.cat((r, x[..., rot:]), -1)


def turn(x, cos, sin, rot, il, sign=1.0):
    """x [B, N, H, d] turned by cos/sin [B, N, rot/2]; sign -1: turned back."""
    if rot == 0:
        return x
    c, s = cos[:, :, None], sign * sin[:, :, None]
    a, b = _split(x, rot, il)
    return _join(a * c - b * s, a * s + b * c, x, rot, il)


def pair_size(x, rot, il):
    """|a| + |b| at both channels of a pair, |x| at the rest."""
    x = x.abs()
    if rot == 0:
        return x
    a, b = _split(x, rot, il)
    return _join(a + b, a + b, x, rot, il)


def rows_of_table(table, pos, B, N):
    t = table.double().cpu()
    if pos is None:
        return t[:N].expand(B, N, -1)
    p = pos.cpu().long()
    r = t[p.clamp(0, t.shape[0] - 1)]
    return torch.where((p >= t.shape[0])[..., None], torch.nan, r)


def norm_rope(x, gamma, cos, sin, pos, eps, il):
    """(y, tolerance) in 64 bits."""
    B, N, H, d = x.shape
    rot = 2 * cos.shape[1]
    f = x.double().cpu()
    far = None if pos is None else (pos.cpu() >= cos.shape[0])[:, :, None, None]
    pad = None if pos is None else (pos.cpu() < 0)[:, :, None, None]
    c, s = rows_of_table(cos, pos, B, N), rows_of_table(sin, pos, B, N)
    n = f / (f.pow(2).mean(-1, keepdim=True) + eps).sqrt() * gamma.double().cpu()
    if far is not None:
        n = torch.where(far, torch.nan, n)
    y = turn(n, c, s, rot, il)
    if pad is not None:
        y = torch.where(pad, 0.0, y)
    # fp32 steps: d squares summed by 8 and a tree of 5 (13 steps, halved by the root), mean, root, reciprocal, two
    # products, two products and a sum of the rotation: under 20 roundings of the pair's size; then the type's own
    tol = half_step(x.dtype) * y.abs() + 20 * U32 * pair_size(n, rot, il) + tiny(x.dtype)
    return y, tol


def norm_rope_bwd(dy, x, gamma, cos, sin, pos, eps, il):
    """((dx, tolerance), (dgamma, tolerance of one rounding of its terms' sizes))."""
    B, N, H, d = x.shape
    rot = 2 * cos.shape[1]
    f, gm = x.double().cpu(), gamma.double().cpu()
    c, s = rows_of_table(cos, pos, B, N), rows_of_table(sin, pos, B, N)
    g = dy.double().cpu()
    if pos is not None:
        p = pos.cpu()
        g = torch.where((p < 0)[:, :, None, None], 0.0, g)
        f = torch.where((p >= cos.shape[0])[:, :, None, None], torch.nan, f)
    r = 1 / (f.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    size = pair_size(g, rot, il)
    g = turn(g, c, s, rot, il, -1.0)
    xh = f * r
    dgamma = (g * xh).sum((0, 1, 2))
    u, us = g * gm, size * gm.abs()
    dx = r * (u - xh * (u * xh).mean(-1, keepdim=True))
    if pos is not None:
        dx = torch.where((p < 0)[:, :, None, None], 0.0, dx)
    dots = xh.abs() * (us * xh.abs()).mean(-1, keepdim=True)
    tol = half_step(x.dtype) * dx.abs() + 48 * U32 * r * (us + dots) + tiny(x.dtype)
    return (dx, tol), (dgamma, (size * xh.abs()).sum((0, 1, 2)) * U32)


# -------------------------------------------------------------------- W8A8 --
def token_quant(a):
    """Codes (float64 whole numbers) and fp32 scales of the rows of a, by the definition in 64 bits with the three
    fp32 roundings it names."""
    x = a.double().cpu()
    amax = x.abs().amax(1, keepdim=True)
    bad = ~torch.isfinite(x).all(1, keepdim=True)
    some = (amax >= 2.0 ** -100) & ~bad
    mult = (127.0 / torch.where(some, amax, 1.0)).float().double()
    codes = torch.where(some, (torch.where(some, x, 0.0) * mult).float().double().round().clamp(-127, 127), 0.0)
    scale = torch.where(bad, torch.nan, torch.where(some, (amax / 127.0).float().double(), 1.0))
    return codes, scale[:, 0]


def token_linear(xq, sx, wq, sw, bias, dtype):
    """(y, tolerance): the fp32 steps are the dot's conversion, two products and a sum."""
    dot = xq.double().cpu() @ wq.double().cpu().t()
    y0 = dot * sx.double().cpu()[:, None] * sw.double().cpu()
    b = 0.0 if bias is None else bias.double().cpu()
    y = y0 + b
    size = y0.abs() + (0.0 if bias is None else b.abs())
    return y, half_step(dtype) * y.abs() + 4 * U32 * (1 + half_step(dtype)) * size + tiny(dtype)


# ------------------------------------------- linear attention with a decay --
def decay(q, k, v, log_decay, state, lens, scale):
    """(out, size, state, size) by the recurrence in 64 bits; a size is the same sum over magnitudes."""
    q, k, v = (t.double().cpu().transpose(1, 2) for t in (q, k, v))
    B, H, N, d = q.shape
    G = H // k.shape[1]
    k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    lam = torch.exp(log_decay.double().cpu())[None, :, None, None]
    S = torch.zeros(B, H, d, d, dtype=torch.float64) if state is None else state.double().cpu().clone()
    A = S.abs()
    out, size = torch.zeros(B, H, N, d, dtype=torch.float64), torch.zeros(B, H, N, d, dtype=torch.float64)
    n_of = [N] * B if lens is None else [max(0, min(N, int(n))) for n in lens]
    for t in range(N):
        on = torch.tensor([t < n for n in n_of])[:, None, None, None]
        kv = k[:, :, t, :, None] * v[:, :, t, None, :]
        S = torch.where(on, lam * S + kv, S)
        A = torch.where(on, lam * A + kv.abs(), A)
        live = on[..., 0]
        out[:, :, t] = torch.where(live, scale * (q[:, :, t, None] @ S)[:, :, 0], 0.0)
        size[:, :, t] = torch.where(live, abs(scale) * (q[:, :, t, None].abs() @ A)[:, :, 0], 0.0)
    return out.transpose(1, 2), size.transpose(1, 2), S, A


def as_numpy(t):
    return np.asarray(t.detach().double().cpu())
