"""The per-head QK norm with the position rotation, forward and backward,
against a plain implementation in 64 bits: types, head layouts, partial
rotation, both pairings, positions with padding and out of the tables, views
of a fused projection, in place, one row, other streams, captured graphs."""
import pytest
import torch

from tests import _layer_ref as ref

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-6


@pytest.fixture(scope="module")
def sg():
    from sparse_bit_attention_smoothing_b200 import build
    build.build()
    import sparse_bit_attention_smoothing_b200 as s
    assert torch.cuda.is_available()
    return s


def tables(T, rot, seed=0):
    f = torch.pow(10000.0, -torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    a = torch.arange(T, dtype=torch.float64)[:, None] * f[None]
    return a.cos().float().cuda(), a.sin().float().cuda()


def fused(B, N, Hq, Hk, d, dtype, seed):
    """q, k as views of the rows of a fused projection, channels of different ranges."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = (Hq + 2 * Hk) * d
    x = torch.randn(B, N, w, generator=g, device="cuda") * (0.1 + 4 * torch.rand(w, generator=g, device="cuda"))
    x = x.to(dtype)
    gq, gk = ((1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(dtype) for _ in range(2))
    return x[..., :Hq * d].unflatten(-1, (Hq, d)), x[..., Hq * d:(Hq + Hk) * d].unflatten(-1, (Hk, d)), gq, gk


def grads(q, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return tuple(torch.randn(t.shape, generator=g, device="cuda").to(t.dtype) for t in (q, k))


def positions(B, N, T, seed):
    g = torch.Generator().manual_seed(seed)
    p = torch.randint(0, T, (B, N), generator=g, dtype=torch.int32)
    p[torch.rand(B, N, generator=g) < 0.2] = -1
    return p.cuda()


def check_forward(got, q, k, gq, gk, cos, sin, pos, il):
    for o, x, g, w in ((got[0], q, gq, "q"), (got[1], k, gk, "k")):
        y, tol = ref.norm_rope(x, g, cos, sin, pos, EPS, il)
        ref.inside(o, y, tol, w)


def check_backward(got, dyq, dyk, q, k, gq, gk, cos, sin, pos, il):
    for dx, dg, dy, x, g, w in ((got[0], got[2], dyq, q, gq, "q"), (got[1], got[3], dyk, k, gk, "k")):
        (rx, tx), (rg, tg) = ref.norm_rope_bwd(dy, x, g, cos, sin, pos, EPS, il)
        ref.inside(dx, rx, tx, "d" + w)
        # a term has under 48 roundings; a lane adds at most 2 rows of each of its tokens in fp32, the rest is a tree
        rows = x.shape[0] * x.shape[1] * x.shape[2]
        ref.inside(dg, rg, (60 + rows) * tg if rows < 256 else 316 * tg, "dgamma " + w)


CASES = [  # B, N, Hq, Hk, d, rot, interleaved, dtype
    (1, 1, 1, 1, 128, 128, True, BF), (1, 1, 40, 8, 128, 128, False, BF), (2, 7, 3, 1, 16, 16, False, HF),
    (1, 33, 5, 5, 32, 16, True, FP), (3, 50, 16, 4, 64, 32, False, HF), (2, 19, 9, 3, 80, 48, False, BF),
    (2, 21, 2, 2, 96, 96, True, FP), (1, 130, 12, 12, 128, 128, True, BF), (1, 65, 7, 2, 256, 256, False, FP),
    (2, 40, 6, 6, 240, 0, True, BF), (1, 300, 4, 1, 256, 64, True, HF), (4, 17, 33, 11, 48, 48, False, FP),
]


@pytest.mark.parametrize("B,N,Hq,Hk,d,rot,il,dtype", CASES)
@pytest.mark.parametrize("placed", [False, True])
def test_forward(sg, B, N, Hq, Hk, d, rot, il, dtype, placed):
    q, k, gq, gk = fused(B, N, Hq, Hk, d, dtype, B * N + d)
    cos, sin = tables(N + 3 if not placed else 500, rot)
    pos = positions(B, N, 500, N) if placed else None
    for head_major in (False, True):
        got = sg.sagesla_qk_norm_rope(q, k, gq, gk, cos, sin, pos=pos, eps=EPS, interleaved=il, head_major=head_major)
        if head_major:
            assert all(t.is_contiguous() for t in got) and got[0].shape == (B, Hq, N, d)
            got = [t.transpose(1, 2) for t in got]
        check_forward(got, q, k, gq, gk, cos, sin, pos, il)


@pytest.mark.parametrize("B,N,Hq,Hk,d,rot,il,dtype", CASES)
@pytest.mark.parametrize("placed", [False, True])
def test_backward(sg, B, N, Hq, Hk, d, rot, il, dtype, placed):
    q, k, gq, gk = fused(B, N, Hq, Hk, d, dtype, B + N + d)
    dyq, dyk = grads(q, k, d)
    cos, sin = tables(N if not placed else 500, rot)
    pos = positions(B, N, 500, N) if placed else None
    got = sg.sagesla_qk_norm_rope_bwd(dyq, dyk, q, k, gq, gk, cos, sin, pos=pos, eps=EPS, interleaved=il)
    check_backward(got, dyq, dyk, q, k, gq, gk, cos, sin, pos, il)


def test_backward_long_and_repeatable(sg):
    """Every warp walks many tokens; the sums have the same bits every time."""
    q, k, gq, gk = fused(1, 5003, 12, 4, 128, BF, 9)
    dyq, dyk = grads(q, k, 3)
    cos, sin = tables(5003, 128)
    a = sg.sagesla_qk_norm_rope_bwd(dyq, dyk, q, k, gq, gk, cos, sin)
    b = sg.sagesla_qk_norm_rope_bwd(dyq, dyk, q, k, gq, gk, cos, sin)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    check_backward(a, dyq, dyk, q, k, gq, gk, cos, sin, None, True)


@pytest.mark.parametrize("il", [False, True])
def test_backward_against_differences(sg, il):
    """<gradient, direction> against central differences of the 64-bit forward."""
    q, k, gq, gk = fused(1, 6, 2, 1, 32, FP, 4)
    dyq, dyk = grads(q, k, 5)
    cos, sin = tables(6, 16)
    got = sg.sagesla_qk_norm_rope_bwd(dyq, dyk, q, k, gq, gk, cos, sin, eps=EPS, interleaved=il)
    gen = torch.Generator().manual_seed(1)
    h = 1e-6
    for x, gm, dy, dx, dg in ((q, gq, dyq, got[0], got[2]), (k, gk, dyk, got[1], got[3])):
        x64, g64 = x.double().cpu(), gm.double().cpu()
        ex, eg = torch.randn(x.shape, generator=gen, dtype=torch.float64), torch.randn(gm.shape, generator=gen, dtype=torch.float64)

        def loss(s):
            y, _ = ref.norm_rope(x64 + s * ex, g64 + s * eg, cos, sin, None, EPS, il)
            return float((y * dy.double().cpu()).sum())
        want = (loss(h) - loss(-h)) / (2 * h)
        have = float((dx.double().cpu() * ex).sum() + (dg.double().cpu() * eg).sum())
        # differences: h^2 of the third derivative and 1e-16 |loss| / h; the fp32 gradient: 1e-5 of its size
        assert abs(want - have) <= 1e-5 * float(dx.double().norm() * ex.norm() + dg.double().norm() * eg.norm()) + 1e-6


def test_positions_out_of_the_tables_and_padding(sg):
    q, k, gq, gk = fused(1, 4, 2, 1, 64, BF, 2)
    cos, sin = tables(10, 64)
    pos = torch.tensor([[9, 10, -5, 2147483647]], dtype=torch.int32, device="cuda")
    q2 = q.clone()
    q2[0, 2] = float("nan")  # padding is not read
    got = sg.sagesla_qk_norm_rope(q2, k, gq, gk, cos, sin, pos=pos)
    check_forward(got, q, k, gq, gk, cos, sin, pos, True)
    assert torch.isnan(got[0][0, 1]).all() and torch.isnan(got[1][0, 3]).all() and not got[0][0, 2].any()
    dyq, dyk = grads(q, k, 1)
    pos = torch.tensor([[0, 3, -1, 2]], dtype=torch.int32, device="cuda")
    dyq[0, 2] = float("inf")
    dg = sg.sagesla_qk_norm_rope_bwd(dyq, dyk, q2, k, gq, gk, cos, sin, pos=pos)
    dyq[0, 2] = 0
    check_backward(dg, dyq, dyk, q, k, gq, gk, cos, sin, pos, True)
    dg = sg.sagesla_qk_norm_rope_bwd(dyq, dyk, q, k, gq, gk, cos, sin, pos=torch.full_like(pos, -1))
    assert not any(t.any() for t in dg)  # nothing but padding
    dg = sg.sagesla_qk_norm_rope_bwd(dyq, dyk, q, k, gq, gk, cos, sin, pos=torch.full_like(pos, 10))
    assert all(torch.isnan(t).all() for t in dg)


def test_zero_and_special_rows(sg):
    q, k, gq, gk = fused(1, 5, 1, 1, 128, FP, 8)
    q = q.clone()
    q[0, 0] = 0
    q[0, 1, 0, 3] = float("inf")
    q[0, 2, 0, 5] = float("nan")
    q[0, 3] *= 2.0 ** 50
    q[0, 4] *= 2.0 ** -60
    cos, sin = tables(5, 128)
    got, _ = sg.sagesla_qk_norm_rope(q, None, gq, None, cos, sin, eps=EPS)
    assert not got[0, 0].any()
    assert torch.isnan(got[0, 1]).any() and torch.isnan(got[0, 2]).all()
    y, tol = ref.norm_rope(q[:, 3:], gq, cos[3:], sin[3:], None, EPS, True)
    ref.inside(got[:, 3:], y, tol, "scaled rows")


def test_query_alone_in_place_and_broadcast(sg):
    q, k, gq, gk = fused(2, 30, 4, 2, 64, BF, 6)
    cos, sin = tables(30, 64)
    want = sg.sagesla_qk_norm_rope(q, k, gq, gk, cos, sin)
    alone, none = sg.sagesla_qk_norm_rope(q, None, gq, None, cos, sin)
    assert none is None and torch.equal(alone, want[0])
    q2, k2, _, _ = fused(2, 30, 4, 2, 64, BF, 6)
    whole = q2._base.clone()
    sg.sagesla_qk_norm_rope(q2, k2, gq, gk, cos, sin, q_out=q2, k_out=k2)  # into the fused rows themselves
    assert torch.equal(q2, want[0]) and torch.equal(k2, want[1])
    assert torch.equal(q2._base[..., 6 * 64:], whole[..., 6 * 64:])  # v's rows as they were
    shared = k[:, :, :1].expand(2, 30, 4, 64)  # one head read four times (stride 0)
    got, _ = sg.sagesla_qk_norm_rope(shared, None, gq, None, cos, sin)
    one, _ = sg.sagesla_qk_norm_rope(k[:, :, :1], None, gq, None, cos, sin)
    assert torch.equal(got, one.expand_as(got))
    dyq, dyk = grads(q, k, 2)
    want = sg.sagesla_qk_norm_rope_bwd(dyq, dyk, q, k, gq, gk, cos, sin)
    a = sg.sagesla_qk_norm_rope_bwd(dyq, None, q, None, gq, None, cos, sin)
    assert torch.equal(a[0], want[0]) and a[1] is None and a[3] is None
    # the warps share the tokens out differently without k, so dgamma's sums run in another order
    _, (rg, tg) = ref.norm_rope_bwd(dyq, q, gq, cos, sin, None, EPS, True)
    ref.inside(a[2], rg, 300 * tg, "dgamma alone")
    g2 = dyq.clone()
    sg.sagesla_qk_norm_rope_bwd(g2, dyk, q, k, gq, gk, cos, sin, dq=g2)  # into the incoming gradient
    assert torch.equal(g2, want[0])


def test_offsets_past_32_bits(sg):
    """Rows more than 2^31 elements apart."""
    far = 2 ** 31 + 64
    buf = torch.zeros(far + 64 * 8, dtype=BF, device="cuda")
    x = buf.as_strided((2, 2, 4, 64), (far, 256, 64, 1))
    x.copy_(torch.randn(2, 2, 4, 64, device="cuda"))
    q, _, gq, _ = fused(1, 1, 1, 1, 64, BF, 0)
    cos, sin = tables(2, 64)
    got, _ = sg.sagesla_qk_norm_rope(x, None, gq, None, cos, sin)
    want, _ = sg.sagesla_qk_norm_rope(x.contiguous(), None, gq, None, cos, sin)
    assert torch.equal(got, want)
    sg.sagesla_qk_norm_rope(x.contiguous(), None, gq, None, cos, sin, q_out=x)
    assert torch.equal(x, want)


def test_other_stream_and_captured(sg):
    q, k, gq, gk = fused(1, 200, 8, 2, 128, BF, 5)
    dyq, dyk = grads(q, k, 7)
    cos, sin = tables(200, 128)
    torch.cuda.synchronize()
    want = sg.sagesla_qk_norm_rope(q, k, gq, gk, cos, sin) + sg.sagesla_qk_norm_rope_bwd(dyq, dyk, q, k, gq, gk, cos, sin)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = (sg.sagesla_qk_norm_rope(q, k, gq, gk, cos, sin, stream=s)
           + sg.sagesla_qk_norm_rope_bwd(dyq, dyk, q, k, gq, gk, cos, sin, stream=s))
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(sg.sagesla_qk_norm_rope(q, k, gq, gk, cos, sin)
                        + sg.sagesla_qk_norm_rope_bwd(dyq, dyk, q, k, gq, gk, cos, sin))
        graphs.append(g)
    q.copy_(torch.randn_like(q))
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):  # both at once
        for g, s in zip(graphs, side):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    want = sg.sagesla_qk_norm_rope(q, k, gq, gk, cos, sin) + sg.sagesla_qk_norm_rope_bwd(dyq, dyk, q, k, gq, gk, cos, sin)
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, want))
