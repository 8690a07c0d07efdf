"""dgamma of the norm and rotation: sums over rows that a group leaves out."""
import pytest
import torch

from tests import _layer_ref as ref

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def sg():
    from sparse_bit_attention_smoothing_b200 import build
    build.build()
    import sparse_bit_attention_smoothing_b200 as s
    assert torch.cuda.is_available()
    return s


HEADS = [(1, 0), (1, 1), (2, 1), (3, 3), (5, 1), (12, 4), (40, 5)]


@pytest.mark.parametrize("Hq,Hk", HEADS)
@pytest.mark.parametrize("d", [16, 48, 64, 128, 256])
@pytest.mark.parametrize("il", [True, False])
@pytest.mark.parametrize("dtype", [BF, HF, FP])
def test_no_eps_and_groups_that_heads_do_not_fill(sg, Hq, Hk, d, il, dtype):
    """eps = 0 and rows that are not zero: places of a group without a head add nothing (they have no norm)."""
    N = 700 if Hq < 12 else 300  # enough tokens for groups of several heads
    g = torch.Generator().manual_seed(Hq + d)
    rows = lambda H: (0.5 + torch.rand(1, N, H, d, generator=g)).mul_(torch.randint(0, 2, (1, N, H, d), generator=g) * 2 - 1).to(dtype).cuda()
    cos, sin = (torch.randn(N, d // 2 // 8 * 8, generator=g).cuda() for _ in range(2))
    pos = torch.arange(N, dtype=torch.int32)[None].clone()
    pos[:, ::7] = -1
    q, dyq, gq = rows(Hq), rows(Hq), torch.rand(d, generator=g).to(dtype).cuda()
    k, dyk, gk = (rows(Hk), rows(Hk), torch.rand(d, generator=g).to(dtype).cuda()) if Hk else (None, None, None)
    for p in (None, pos.cuda()):
        got = sg.sagesla_qk_norm_rope_bwd(dyq, dyk, q, k, gq, gk, cos, sin, pos=p, eps=0.0, interleaved=il)
        for dx, dg, dy, x, gm in ((got[0], got[2], dyq, q, gq), (got[1], got[3], dyk, k, gk)):
            if x is None:
                assert dx is None and dg is None
                continue
            (rx, tx), (rg, tg) = ref.norm_rope_bwd(dy, x, gm, cos, sin, p, 0.0, il)
            ref.inside(dx, rx, tx, "dx")
            # a term has under 48 roundings; no sum of terms in fp32 is longer than all of them
            ref.inside(dg, rg, (60 + N * x.shape[2]) * tg, "dgamma")


def test_error_does_not_grow_with_the_tokens(sg):
    """Terms of one sign over 2.4 million tokens: many that are each less than half a step of one long fp32 sum of them
    (they would all be lost: 2^-13 of the sum)."""
    N, H, d = 2400000, 8, 128
    x = torch.ones(1, 1, 1, d, dtype=BF, device="cuda").expand(1, N, H, d)
    dy = torch.full((1, N, 1, d), 2.0 ** -19, dtype=BF, device="cuda")
    dy[:, :N // 64] = 1.0
    no = torch.empty(N, 0, device="cuda")
    _, _, dg, _ = sg.sagesla_qk_norm_rope_bwd(dy.expand(1, N, H, d), None, x, None, torch.ones(d, dtype=BF, device="cuda"),
                                              None, no, no, eps=0.0)
    want = torch.full((d,), H * (N // 64 + (N - N // 64) * 2.0 ** -19), dtype=torch.float64)
    # a term has under 48 roundings; then at most 128 tokens of 4 rows in one fp32 sum, 4 lanes' and 8 warps' sums in
    # fp32, one rounding behind the fp64 sum
    ref.inside(dg, want, (48 + 512 + 4 + 8 + 1) * ref.U32 * want, "dgamma")


@pytest.mark.parametrize("il", [True, False])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_rounds_of_blocks(sg, il, dtype):
    """More tokens than one round of blocks walks: both tensors, padding, the same bits every time."""
    N, Hq, Hk, d = 330000, 3, 1, 16
    g = torch.Generator(device="cuda").manual_seed(4)
    q, dyq = (torch.randn(1, N, Hq, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    k, dyk = (torch.randn(1, N, Hk, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    gq, gk = (torch.rand(d, generator=g, device="cuda").to(dtype) for _ in range(2))
    cos, sin = (torch.randn(N, d // 2, generator=g, device="cuda") for _ in range(2))
    pos = torch.arange(N, dtype=torch.int32, device="cuda")[None].clone()
    pos[:, 5::9] = -1
    args = (dyq, dyk, q, k, gq, gk, cos, sin)
    got = sg.sagesla_qk_norm_rope_bwd(*args, pos=pos, interleaved=il)
    for dx, dg, dy, x, gm in ((got[0], got[2], dyq, q, gq), (got[1], got[3], dyk, k, gk)):
        (rx, tx), (rg, tg) = ref.norm_rope_bwd(dy, x, gm, cos, sin, pos, 1e-6, il)
        ref.inside(dx, rx, tx, "dx")
        ref.inside(dg, rg, (48 + 512 + 16 + 8 + 1) * tg, "dgamma")
    again = sg.sagesla_qk_norm_rope_bwd(*args, pos=pos, interleaved=il)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
