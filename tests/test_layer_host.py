"""Host side of the operators around the attention, on the fake CUDA runtime (an sm_100 device whose launches do not run)."""
import subprocess
import sys

from tests._fake import ROOT, fake  # noqa: F401

HEAD = """
import ctypes, sys
sys.path.insert(0, %r)
fake = ctypes.CDLL(%r, mode=ctypes.RTLD_GLOBAL)
import sparse_bit_attention_smoothing_b200 as sg
L, P, F, LL = sg.lib(), ctypes.c_void_p, ctypes.c_float, ctypes.c_longlong
A = P(0x10000)
"""


def run(fake, body):  # noqa: F811
    r = subprocess.run([sys.executable, "-c", HEAD % (ROOT, fake) + body], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.stdout, r.stderr[-2000:])


WORKSPACE = """
def need(B, N, Hq, Hk, d):
    n = LL(-1)
    assert L.sagesla_qk_norm_rope_bwd_workspace(B, N, Hq, Hk, d, ctypes.byref(n)) == 0
    return n.value
for d in (16, 128, 256):
    row = 2 * d * 4  # a block's partial sums of q and k
    assert need(1, 1, 1, 0, d) == row
    last = 0
    for N in (1, 100, 32760, 75600, 10 ** 6, 10 ** 8, 2 ** 31 - 1):
        for H in (1, 40, 5000, 65535):
            n = need(1, N, H, H, d)
            most = -(-N * 2 * H // 8)  # blocks of 8 warps, a (token, head) each
            assert 0 < n <= row * max(most, 1) and n % row == 0
            # no warp walks more than 128 tokens (and its share of a group)
            assert n // row * 8 * 128 >= N * 2 * H
            assert n >= need(1, N, H, 0, d)
"""

IGNORED = """
i64 = ctypes.c_int64
odd = P(0x10001)  # what an argument that is not used may be
s12, s18 = (i64 * 12)(*[1024, 128, 64] * 4), (i64 * 18)(*[1024, 128, 64] * 6)
def fwd(gk, cos, sin, k, ko, Hk, rot):
    return L.sagesla_qk_norm_rope(A, k, A, gk, F(1e-6), cos, sin, None, A, ko, 0, 1, 8, 2, Hk, 64, rot, 8, 1, s12, None)
def bwd(gk, cos, sin, k, dk, dgk, Hk, rot):
    return L.sagesla_qk_norm_rope_bwd(A, k, A, k, A, gk, F(1e-6), cos, sin, None, A, dk, A, dgk, 0, 1, 8, 2, Hk, 64, rot, 8, 1,
                                      s18, A, LL(1 << 20), None)
assert fwd(A, A, A, A, A, 2, 64) == 0 and bwd(A, A, A, A, A, A, 2, 64) == 0
# used: refused
assert fwd(odd, A, A, A, A, 2, 64) == -2 and fwd(A, odd, A, A, A, 2, 64) == -2 and fwd(A, A, A, odd, A, 2, 64) == -2
assert bwd(A, A, A, A, A, odd, 2, 64) == -2
# not used: whatever they are
n = fake.fake_launches()
assert fwd(odd, A, A, odd, odd, 0, 64) == 0 and fwd(A, odd, odd, A, A, 2, 0) == 0
assert bwd(odd, A, A, odd, odd, odd, 0, 64) == 0 and bwd(A, odd, odd, A, A, A, 2, 0) == 0
assert fake.fake_launches() == n + 6
"""


def test_unused_arguments_are_ignored(fake):  # noqa: F811
    """Hk = 0: no k and nothing of it; rot = 0: no tables."""
    run(fake, IGNORED)


def test_backward_workspace_over_all_sizes(fake):  # noqa: F811
    run(fake, WORKSPACE)
