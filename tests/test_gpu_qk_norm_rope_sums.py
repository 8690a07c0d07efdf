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
