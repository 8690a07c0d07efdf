"""The barrier protocols of the linear attention with a decay, on the CPU, with
the scheduler and the conditions of test_protocols.py.

A product that an MMA-issuing warp serves is a role of its own here (the warp
takes whichever is ready, so the products of one warp meet in any order), and
what the warp signals when two of its products are over is a role that waits
for both.  The warp tests all barriers of a product at once, again and again
until all are there: `turn` puts another one of them last.  Buffers of which
each warp has its own part are modelled by parts.
"""
from collections import defaultdict

import pytest

from test_protocols import _caught, simulate

STATE, OUT = 2, 2  # warps of the state and of the outputs (fewer than the kernel's: the same protocol)


def _reads(bufs, tag):
    return [("rbeg", b, tag) for b in bufs], [("rend", b) for b in bufs]


def _writes(bufs, tag):
    return [("wbeg", b, tag) for b in bufs], [("wend", b) for b in bufs]


def _copies(n, stages, tensors):
    p = []
    for c in range(n):
        st = c % stages
        if c >= stages:
            p.append(("wait", ("empty", st), c // stages - 1))
        for t in tensors:
            p += [("wbeg", (t, st), c), ("wend", (t, st))]
        p.append(("arrive", ("full", st)))
    return p


def _turned(waits, turn):
    k = turn % len(waits)
    return waits[k:] + waits[:k]


def walk_programs(n, stages=3, nparts=2, nscore=2, turn=0):
    """linear_decay_kernel with outputs: n chunks."""
    P, C = {"copies": _copies(n, stages, "qkv")}, defaultdict(lambda: 1)
    area = lambda i: [("area", i & 1, w) for w in range(STATE)]
    pbuf = lambda i: [("pbuf", i & 1, w) for w in range(OUT)]
    U, S, OS, OI = [], [], [], []
    for c in range(n):
        st, b = c % stages, c & 1
        full = ("wait", ("full", st), c // stages)
        # the chunk's own state, into the area of the state before the last chunk
        waits = [("wait", ("vp_full",), c), full]
        if c >= 1:
            waits.append(("wait", ("s_read", b ^ 1), (c - 1) // 2))
        r, re = _reads([("k", st), ("vp",)], c)
        w, we = _writes(area(c + 1), ("U", c))
        U += _turned(waits, turn) + r + w + re + we + [("arrive", ("u_full", b)), ("arrive", ("U", c))]
        # the scores
        waits = [full]
        if c >= 2:
            waits.append(("wait", ("o_empty", b), (c - 2) // 2))
        r, re = _reads([("q", st), ("k", st)], c)
        S += _turned(waits, turn) + r + [("wbeg", ("oi", b), ("P", c))] + re + [("wend", ("oi", b)), ("arrive", ("p_full", b)), ("arrive", ("S", c))]
        # S^T q
        waits = [("wait", ("s_full", b), c // 2), full]
        if c >= 1:
            waits.append(("wait", ("o_empty", b ^ 1), (c - 1) // 2))
        r, re = _reads(area(c), ("TS", c))
        OS += _turned(waits, turn) + [("rbeg", ("q", st), c)] + r + [("wbeg", ("os",), c)] + re + \
              [("rend", ("q", st)), ("wend", ("os",)), ("arrive", ("s_read", b)), ("arrive", ("OS", c))]
        # V^T P'
        r, re = _reads(pbuf(c), ("P'", c))
        waits = [("wait", ("pp_full", b), c // 2), ("wait", ("u_full", b), c // 2)]
        OI += _turned(waits, turn) + [("rbeg", ("v", st), c)] + r + \
              [("wbeg", ("oi", b), ("O", c)), ("rend", ("v", st))] + re + [("wend", ("oi", b)), ("arrive", ("OI", c))]
    P.update(U=U, S=S, OS=OS, OI=OI)
    P["read1"] = [s for c in range(n) for s in (("wait", ("U", c), 0), ("wait", ("S", c), 0), ("arrive", ("empty", c % stages)))]
    P["read2"] = [s for c in range(n) for s in (("wait", ("OS", c), 0), ("wait", ("OI", c), 0), ("arrive", ("empty", c % stages)))]
    P["o_full"] = [s for c in range(n) for s in (("wait", ("OS", c), 0), ("wait", ("OI", c), 0), ("arrive", ("o_full",)))]
    for b in range(stages):
        C[("empty", b)] = 2
    for w in range(nparts):
        p = []
        for c in range(n):
            st = c % stages
            p += [("wait", ("full", st), c // stages), ("rbeg", ("v", st), c)]
            if c >= 1:
                p.append(("wait", ("u_full", (c + 1) & 1), (c - 1) // 2))
            p += [("wbeg", ("vp",), c), ("rend", ("v", st)), ("wend", ("vp",)), ("arrive", ("vp_full",))]
        P[f"parts{w}"] = p
    C[("vp_full",)] = nparts
    for w in range(nscore):
        p = []
        for c in range(n):
            b = c & 1
            p += [("wait", ("p_full", b), c // 2), ("rbeg", ("oi", b), ("P", c))]
            if c >= 2:
                p.append(("wait", ("pp_empty", b), (c - 2) // 2))
            wr, we = _writes(pbuf(c), ("P'", c))
            p += wr + [("rend", ("oi", b))] + we + [("arrive", ("pp_full", b))]
        P[f"score{w}"] = p
    for w in range(STATE):
        p = [("wbeg", ("area", 0, w), ("TS", 0)), ("wend", ("area", 0, w)), ("arrive", ("s_full", 0))]
        for c in range(n):
            mine = ("area", (c + 1) & 1, w)
            p += [("wait", ("u_full", c & 1), c // 2), ("rbeg", mine, ("U", c)), ("rend", mine)]
            if c + 1 < n:
                p += [("wbeg", mine, ("TS", c + 1)), ("wend", mine), ("arrive", ("s_full", (c + 1) & 1))]
        P[f"state{w}"] = p
    for w in range(OUT):
        p = []
        for c in range(n):
            b, mine = c & 1, ("pbuf", c & 1, w)
            p += [("wait", ("o_full",), c), ("rbeg", ("oi", b), ("O", c)), ("rbeg", ("os",), c),
                  ("wbeg", mine, ("out", c)), ("rend", ("oi", b)), ("rend", ("os",)), ("arrive", ("o_empty", b)),
                  ("wend", mine), ("rbeg", mine, ("out", c)), ("rend", mine), ("arrive", ("pp_empty", b))]
        P[f"out{w}"] = p
    for b in range(2):
        C[("pp_full", b)], C[("s_full", b)], C[("o_empty", b)], C[("pp_empty", b)] = nscore, STATE, OUT, OUT
    return P, C


def own_state_programs(n, stages=5, groups=2, nparts=2, turn=0):
    """linear_decay_kernel without outputs: a segment's own state, the parts of
    v by two warpgroups in turn."""
    P, C = {"copies": _copies(n, stages, "kv")}, defaultdict(lambda: 1)
    U = []
    for c in range(n):
        st, b = c % stages, c & 1
        waits = [("wait", ("vp_full", b), c // 2), ("wait", ("full", st), c // stages)]
        if c >= 2:
            waits.append(("wait", ("u_read", b), (c - 2) // 2))
        U += _turned(waits, turn) + [("rbeg", ("k", st), c), ("rbeg", ("vp", b), c), ("wbeg", ("u", b), c),
              ("rend", ("k", st)), ("rend", ("vp", b)), ("wend", ("u", b)), ("arrive", ("empty", st)), ("arrive", ("u_full", b))]
    P["U"] = U
    for g in range(groups):
        for w in range(nparts):
            p = []
            for c in range(g, n, groups):
                st, b = c % stages, c & 1
                p += [("wait", ("full", st), c // stages), ("rbeg", ("v", st), c)]
                if c >= 2:
                    p.append(("wait", ("u_full", b), (c - 2) // 2))
                p += [("wbeg", ("vp", b), c), ("rend", ("v", st)), ("wend", ("vp", b)), ("arrive", ("vp_full", b))]
            P[f"parts{g}.{w}"] = p
    for w in range(STATE):
        p = []
        for c in range(n):
            b = c & 1
            p += [("wait", ("u_full", b), c // 2), ("rbeg", ("u", b), c), ("rend", ("u", b)), ("arrive", ("u_read", b))]
        P[f"state{w}"] = p
    for b in range(2):
        C[("vp_full", b)], C[("u_read", b)] = nparts, STATE
    return P, C


@pytest.mark.parametrize("turn", [0, 1, 2])
@pytest.mark.parametrize("n,stages", [(1, 3), (2, 3), (3, 3), (9, 3), (14, 6)])
def test_walk_protocol(n, stages, turn):
    P, C = walk_programs(n, stages, turn=turn)
    for seed in range(60):
        simulate(P, C, seed)


@pytest.mark.parametrize("turn", [0, 1, 2])
@pytest.mark.parametrize("n,stages", [(1, 5), (2, 5), (12, 5), (17, 8)])
def test_own_state_protocol(n, stages, turn):
    P, C = own_state_programs(n, stages, turn=turn)
    for seed in range(60):
        simulate(P, C, seed)


def test_the_model_catches_three_warpgroups_for_the_parts():
    # a third warpgroup may stand two phases before the product it waits for
    P, C = own_state_programs(12, groups=3)
    assert _caught(P, C)


def test_the_model_catches_an_area_that_is_still_read():
    # the chunk's own state written before S^T q has read the area
    P, C = walk_programs(6)
    P["U"] = [s for s in P["U"] if not (s[0] == "wait" and s[1][0] == "s_read")]
    assert _caught(P, C)


def test_the_model_catches_scores_over_unread_outputs():
    P, C = walk_programs(6)
    P["S"] = [s for s in P["S"] if not (s[0] == "wait" and s[1][0] == "o_empty")]
    assert _caught(P, C)


def test_the_model_catches_a_single_state_barrier():
    # one barrier for the state of every chunk: it may be two completions ahead
    P, C = walk_programs(8, turn=1)
    for r, prog in P.items():
        for i, s in enumerate(prog):
            if s[1][0] == "s_full":
                prog[i] = ("arrive", ("s_full", 0)) if s[0] == "arrive" else ("wait", ("s_full", 0), -1)
    k = 0
    for i, s in enumerate(P["OS"]):
        if s[0] == "wait" and s[1][0] == "s_full":
            P["OS"][i] = ("wait", ("s_full", 0), k)
            k += 1
    assert _caught(P, C)
