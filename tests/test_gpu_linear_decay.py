"""Causal linear attention with a decay for each head against the recurrence
in 64 bits: chunk edges, lengths of zero and one, grouped key heads, strides,
states carried from call to call, extreme decays, streams and graphs."""
import pytest
import torch

from tests import _layer_ref as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
# of the sums' magnitudes: the prompt form holds the scores and the carried state in two bf16 parts (2^-16), the
# keys of the state in three (2^-23); decay factors are exp2 of an fp32 product (|x| 2^-24 and two steps)
OUT, STATE = 2.0 ** -14, 2.0 ** -18


@pytest.fixture(scope="module")
def sg():
    from sparse_bit_attention_smoothing_b200 import build
    build.build()
    import sparse_bit_attention_smoothing_b200 as s
    assert torch.cuda.is_available()
    return s


def inputs(B, N, H, Hk, d, seed, fused=False):
    g = torch.Generator().manual_seed(seed)
    if fused:
        x = torch.randn(B, N, (H + 2 * Hk) * d, generator=g).to(BF).cuda()
        q, k, v = (t.unflatten(-1, (-1, d)) for t in x.split([H * d, Hk * d, Hk * d], -1))
    else:
        q, k, v = (torch.randn(B, N, h, d, generator=g).to(BF).cuda() for h in (H, Hk, Hk))
    ld = -torch.pow(2.0, -8.0 * torch.arange(1, H + 1, dtype=torch.float32) / H).cuda()
    s = torch.randn(B, H, d, d, generator=g).cuda()
    return q, k, v, ld, s


def check(got, q, k, v, ld, s, lens, scale):
    o, os, S, Ss = ref.decay(q, k, v, ld, s, lens, scale)
    ref.inside(got[0], o, ref.half_step(BF) * o.abs() + OUT * os + ref.tiny(BF), "out")
    ref.inside(got[1], S, STATE * Ss, "state")


CASES = [  # B, N, H, Hk, d
    (1, 1, 1, 1, 64), (1, 1, 3, 1, 128), (2, 2, 2, 2, 128), (1, 31, 2, 1, 64), (1, 63, 2, 2, 128), (2, 64, 4, 2, 64),
    (1, 65, 2, 1, 128), (1, 127, 1, 1, 128), (1, 128, 2, 2, 128), (3, 129, 6, 3, 64), (1, 300, 4, 1, 128),
    (2, 513, 3, 3, 64), (1, 1000, 2, 1, 128), (1, 2111, 2, 2, 64),
]


@pytest.mark.parametrize("B,N,H,Hk,d", CASES)
@pytest.mark.parametrize("with_state", [True, False])
def test_prompt(sg, B, N, H, Hk, d, with_state):
    q, k, v, ld, s = inputs(B, N, H, Hk, d, N + d, fused=N % 2 == 1)
    s = s if with_state else None
    for head_major in (False, True):
        out, st = sg.sagesla_linear_decay(q, k, v, ld, s, scale=d ** -0.5, head_major=head_major)
        out = out.transpose(1, 2) if head_major else out
        check((out, st), q, k, v, ld, s, None, d ** -0.5)
    assert sg.sync_status() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_lengths(sg, d):
    """Sequences of different lengths, none and one among them, out of range ones taken into [0, N]."""
    B, N = 8, 200
    q, k, v, ld, s = inputs(B, N, 2, 1, d, 5)
    lens = torch.tensor([0, 1, 64, 65, 128, 199, 1000, -3], dtype=torch.int32, device="cuda")
    for b, n in enumerate(lens.tolist()):  # padding is not read
        for t in (q, k, v):
            t[b, max(0, n):] = float("nan")
    out = torch.full((B, N, 2, d), float("nan"), dtype=BF, device="cuda")
    got = sg.sagesla_linear_decay(q, k, v, ld, s, lens=lens, scale=0.1, out=out)
    clean = [torch.nan_to_num(t) for t in (q, k, v)]
    check(got, *clean, ld, s, lens, 0.1)
    assert torch.equal(got[1][0], s[0]) and torch.equal(got[1][7], s[7])
    st = s.clone()
    sg.sagesla_linear_decay(q, k, v, ld, st, lens=lens, scale=0.1, state_out=st)  # in place
    assert torch.equal(st, got[1])


def test_many_chunks_and_heads(sg):
    """More (sequence, head) pairs than SMs, and few with many chunks."""
    for B, N, H, Hk, d in ((5, 150, 40, 40, 64), (1, 4100, 1, 1, 128), (1, 4100, 3, 3, 64)):
        q, k, v, ld, s = inputs(B, N, H, Hk, d, 7)
        check(sg.sagesla_linear_decay(q, k, v, ld, s, scale=0.2), q, k, v, ld, s, None, 0.2)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [100, 700])
def test_extreme_decays(sg, d, N):
    """No decay at all, and decays that leave only the token itself."""
    q, k, v, _, s = inputs(1, N, 6, 2, d, 3)
    ld = torch.tensor([0.0, -1e-7, -0.5, -30.0, -1e30, float("-inf")], device="cuda")
    got = sg.sagesla_linear_decay(q, k, v, ld, s, scale=0.3)
    check(got, q, k, v, ld, s, None, 0.3)
    own = (0.3 * torch.einsum("bnhd,bnhd->bnh", q[:, :, 5].double()[:, :, None], k[:, :, 1].double()[:, :, None])[..., None]
           * v[:, :, 1].double()[:, :, None])[:, :, 0]
    ref.inside(got[0][:, :, 5], own, ref.half_step(BF) * own.abs() + OUT * own.abs().amax(-1, keepdim=True) * 40 + 1e-30, "alone")


def test_prompt_in_pieces_and_single_tokens(sg):
    """A prompt in pieces, then token by token, is the whole prompt."""
    B, N, H, Hk, d = 2, 333, 4, 2, 128
    q, k, v, ld, s = inputs(B, N, H, Hk, d, 21)
    st, outs = s, []
    for a, b in ((0, 1), (1, 130), (130, 320)):
        o, st = sg.sagesla_linear_decay(q[:, a:b], k[:, a:b], v[:, a:b], ld, st, scale=0.1)
        outs.append(o)
    for n in range(320, N):
        o, st2 = sg.sagesla_linear_decay_step(q[:, n], k[:, n], v[:, n], ld, st, scale=0.1)
        assert st2 is st
        outs.append(o[:, None])
    check((torch.cat(outs, 1), st), q, k, v, ld, s, None, 0.1)


@pytest.mark.parametrize("B,H,Hk,d", [(1, 1, 1, 64), (1, 40, 40, 128), (3, 6, 2, 64), (64, 12, 4, 128), (200, 2, 1, 128)])
def test_step(sg, B, H, Hk, d):
    q, k, v, ld, s = inputs(B, 1, H, Hk, d, B + H, fused=True)
    q, k, v = q[:, 0], k[:, 0], v[:, 0]
    keep = s.clone()
    out, st = sg.sagesla_linear_decay_step(q, k, v, ld, s, scale=0.25, state_out=torch.empty_like(s))
    assert torch.equal(s, keep)
    check((out[:, None], st), q[:, None], k[:, None], v[:, None], ld, s, None, 0.25)
    out2, st2 = sg.sagesla_linear_decay_step(q, k, v, ld, s, scale=0.25)
    assert st2 is s and torch.equal(s, st) and torch.equal(out, out2)


def test_special_values_stay_in_their_rows(sg):
    """NaN of one head or sequence reaches no other; an infinite state only what it feeds."""
    q, k, v, ld, s = inputs(2, 150, 4, 4, 64, 4)
    want = sg.sagesla_linear_decay(q, k, v, ld, s)
    k[1, 70, 2] = float("nan")
    got = sg.sagesla_linear_decay(q, k, v, ld, s)
    assert torch.equal(got[0][0], want[0][0]) and torch.equal(got[1][0], want[1][0])
    keep = [0, 1, 3]
    assert torch.equal(got[0][1][:, keep], want[0][1][:, keep]) and torch.equal(got[1][1][keep], want[1][1][keep])
    assert torch.equal(got[0][1][:64, 2], want[0][1][:64, 2]) and torch.isnan(got[0][1][70:, 2]).all()


def test_offsets_past_32_bits(sg):
    """Sequences more than 2^31 elements apart."""
    far, N, d = 2 ** 31 + 64, 70, 64
    buf = torch.zeros(far + N * 2 * d + 64, dtype=BF, device="cuda")
    x = buf.as_strided((2, N, 2, d), (far, 2 * d, d, 1))
    q, k, v, ld, s = inputs(2, N, 2, 2, d, 1)
    x.copy_(q)
    want = sg.sagesla_linear_decay(q, k, v, ld, s)
    got = sg.sagesla_linear_decay(x, k, v, ld, s)
    assert torch.equal(got[0], want[0])
    sg.sagesla_linear_decay(q, k, v, ld, s, out=x)
    assert torch.equal(x, want[0])


@pytest.mark.parametrize("N", [100, 1500])
def test_other_stream_and_captured(sg, N):
    q, k, v, ld, s = inputs(1, N, 2, 1, 128, 8)
    step = [t[:, 0] for t in (q, k, v)]
    want = sg.sagesla_linear_decay(q, k, v, ld, s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = sg.sagesla_linear_decay(q, k, v, ld, s, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, outs, states = [], [], [s.clone(), s.clone()]
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = sg.sagesla_linear_decay(q, k, v, ld, states[i])
            outs.append(o + sg.sagesla_linear_decay_step(*step, ld, o[1], state_out=torch.empty_like(s)))
        graphs.append(g)
    states[1].mul_(2)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(10):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for o, st in zip(outs, states):
        w = sg.sagesla_linear_decay(q, k, v, ld, st)
        w = w + sg.sagesla_linear_decay_step(*step, ld, w[1], state_out=torch.empty_like(s))
        assert all(torch.equal(a, b) for a, b in zip(o, w))
    assert sg.sync_status() == 0


@pytest.mark.parametrize("B,N,H,Hk,d,segments", [(3, 1000, 16, 4, 64, 3), (6, 1100, 12, 6, 128, 2), (4, 1500, 10, 10, 128, 3)])
def test_few_segments(sg, B, N, H, Hk, d, segments):
    """Two and three segments, whose states the walk joins itself: with and without a state, in place, lengths that end in
    every segment, a v that is not finite."""
    assert sg.sagesla_linear_decay_workspace(B, N, H, d) == 4 * B * H * (segments + 1) * d * d
    q, k, v, ld, s = inputs(B, N, H, Hk, d, 17)
    for state in (s, None):
        check(sg.sagesla_linear_decay(q, k, v, ld, state, scale=0.1), q, k, v, ld, state, None, 0.1)
    lens = torch.tensor([0, 1, N // 2, N - 1, N // 4, N][:B], dtype=torch.int32, device="cuda")
    for b, n in enumerate(lens.tolist()):
        for t in (q, k, v):
            t[b, n:] = float("nan")
    got = sg.sagesla_linear_decay(q, k, v, ld, s, lens=lens, scale=0.1)
    check(got, *(torch.nan_to_num(t) for t in (q, k, v)), ld, s, lens, 0.1)
    assert torch.equal(got[1][0], s[0])
    st = s.clone()
    o, _ = sg.sagesla_linear_decay(q, k, v, ld, st, lens=lens, scale=0.1, state_out=st)
    assert torch.equal(st, got[1]) and torch.equal(o, got[0])
    v[2, N // 2 - 40, 0, 5] = float("inf")
    o, st = sg.sagesla_linear_decay(q, k, v, ld, s, lens=lens, scale=0.1)
    of, bad = got[0].clone(), torch.zeros_like(got[0], dtype=torch.bool)
    bad[2, N // 2 - 40:N // 2, :H // Hk, 5] = True
    assert torch.isnan(o[bad]).all() and torch.equal(o[~bad], of[~bad])
    worst = torch.zeros_like(st, dtype=torch.bool)
    worst[2, :H // Hk, :, 5] = True
    assert torch.isnan(st[worst]).all() and torch.equal(st[~worst], got[1][~worst])


@pytest.mark.parametrize("B,N,H,d", [(3, 700, 16, 64), (1, 2000, 60, 128), (1, 900, 9, 128)])
def test_segments_captured_in_place(sg, B, N, H, d):
    """Calls one after another in one graph, each from the state that the one before left in place, replayed on new
    inputs while another graph of the same calls runs."""
    q, k, v, ld, s = inputs(B, N, H, H, d, 31)
    lens = torch.tensor([N, N // 2, 3][:B], dtype=torch.int32, device="cuda")
    sets = []
    for i in range(2):
        qi, st = q.clone(), s.clone()
        sg.sagesla_linear_decay(qi, k, v, ld, st, lens=lens, state_out=st)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = [sg.sagesla_linear_decay(qi, k, v, ld, st, lens=lens, scale=0.1, state_out=st)[0] for _ in range(3)]
        sets.append((g, qi, st, outs))
    for i, (g, qi, st, outs) in enumerate(sets):
        qi.copy_(q.flip(1) if i else q * 2)
        st.copy_(s)
    torch.cuda.synchronize()
    for g, *_ in sets:
        with torch.cuda.stream(torch.cuda.Stream()):
            g.replay()
    torch.cuda.synchronize()
    for g, qi, st, outs in sets:
        w = s
        for o in outs:
            want, w = sg.sagesla_linear_decay(qi, k, v, ld, w, lens=lens, scale=0.1)
            assert torch.equal(o, want)
        assert torch.equal(st, w)
    assert sg.sync_status() == 0
