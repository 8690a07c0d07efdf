"""The state that a prompt leaves, to the fp32 roundings it may have: one token alone in it, so that no sum of many terms hides
how many bits of the decayed v are kept."""
import math

import pytest
import torch

from tests import _layer_ref as ref

BF = torch.bfloat16


def bound(N, at):
    """Of the state's size, for a token at `at`.  The power l^m and its product with v: 2^-24 each.  Three bf16 parts of it
    leave 2^-27.  Their three products with k are exact and added in fp32 by the tensor core, which may cut instead of
    round: 2^-23 each of two sums.  Every chunk (or segment) behind the token's multiplies by a rounded power and rounds:
    2^-23."""
    later = (N - 1) // 64 - at // 64
    return (2 + 2 + later) * 2.0 ** -23


def parts_left(x, n):
    """What n bf16 parts leave of fp32 values, relative."""
    left = x.clone()
    for _ in range(n):
        left = left - left.to(BF).float()
    return (left.abs() / x.abs()).max()


def test_bound_tells_two_parts_from_three():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(128, generator=g).to(BF).float() * math.exp(-0.37)
    assert parts_left(x, 3) <= 2.0 ** -27 < bound(64, 0) < parts_left(x, 2)


CASES = [  # B, N, H, d: one segment, two and three that the walk carries itself, many with a carry of their own
    (1, 50, 3, 64), (2, 64, 2, 128), (1, 200, 2, 128), (40, 130, 4, 64), (3, 1000, 16, 64), (6, 1100, 12, 128), (4, 1500, 10, 128),
    (1, 4100, 3, 64), (2, 3000, 4, 128), (5, 150, 40, 64), (1, 20000, 1, 128),
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,H,d", CASES)
def test_one_token_in_the_state(B, N, H, d):
    import sparse_bit_attention_smoothing_b200 as sg
    g = torch.Generator().manual_seed(N + d)
    q, v = (torch.randn(B, N, H, d, generator=g).to(BF) for _ in range(2))
    row = torch.randn(B, H, d, generator=g).to(BF)
    ld = -0.6 * torch.rand(H, generator=g) / 40  # l^m of any m, none of them below 2^-100 for the places here
    for at in sorted({0, 1, N // 3, N // 2, max(0, N - 65), N - 2, N - 1}):
        at = max(at, N - 2500)
        k = torch.zeros(B, N, H, d, dtype=BF)
        k[:, at] = row
        _, s = sg.sagesla_linear_decay(q.cuda(), k.cuda(), v.cuda(), ld.cuda())
        want = (row.double()[..., :, None] * v[:, at].double()[..., None, :]
                * torch.exp(ld.double() * (N - 1 - at))[None, :, None, None])
        ref.inside(s, want, bound(N, at) * want.abs() + 2.0 ** -140, f"state of token {at}")
    assert sg.sync_status() == 0
