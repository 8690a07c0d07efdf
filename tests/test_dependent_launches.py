"""Kernels that may be resident before the one whose results they read has ended: those buffers are read by ordinary loads
behind the wait, never by the read-only path (which is for memory that nobody writes while the kernel is resident)."""
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_bit_attention_smoothing_b200", "csrc")

# kernel: what the launch before it writes (a parameter, or a member of its argument struct)
WRITTEN_BEFORE = {
    "w8a8_token_gemm_kernel": ["sx"],
    "w8a8_token_few_kernel": ["sx"],
    "dgamma_kernel": ["part"],
    "linear_decay_kernel": ["ws"],
    "linear_decay_carry_kernel": ["ws"],
}


def kernels():
    """name: (parameters, body) of every kernel of the library."""
    out = {}
    for f in sorted(os.listdir(CSRC)):
        if not f.endswith(".cu"):
            continue
        s = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, f)).read())
        for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\([^)]*\)\s*)?(\w+)\s*\(", s):
            depth, i = 1, m.end()
            while depth:
                depth += {"(": 1, ")": -1}.get(s[i], 0)
                i += 1
            b = s.index("{", i)
            depth, j = 1, b + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(s[j], 0)
                j += 1
            out[m.group(1)] = (s[m.end():i - 1], s[b:j])
    return out


def test_every_waiting_kernel_is_listed():
    waiting = {n for n, (_, body) in kernels().items() if "wait_previous()" in body}
    assert waiting == set(WRITTEN_BEFORE)


@pytest.mark.parametrize("kernel", sorted(WRITTEN_BEFORE))
def test_no_read_only_loads_of_what_the_launch_before_writes(kernel):
    params, body = kernels()[kernel]
    for name in WRITTEN_BEFORE[kernel]:
        assert not re.search(r"__restrict__\s+%s\b" % name, params), name
        for call in re.findall(r"__ldg\(([^()]*(?:\([^()]*\)[^()]*)*)\)", body):
            assert not re.search(r"\b%s\b" % name, call), call


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 640, 1280), (33, 257, 5120), (300, 1001, 256), (2000, 512, 512)])
def test_calls_back_to_back_with_other_scales(M, N, K):
    """The layer called again and again in one workspace, each time with rows of another size: the same bits as the
    quantiser and the product one after another."""
    import sparse_bit_attention_smoothing_b200 as sg
    g = torch.Generator(device="cuda").manual_seed(M)
    w = torch.randn(N, K, generator=g, device="cuda").bfloat16()
    wq, sw = sg.sagesla_w8a8_token_quant(w)
    x = [(torch.randn(M, K, generator=g, device="cuda") * 4.0 ** (i % 7 - 3)).bfloat16() for i in range(40)]
    torch.cuda.synchronize()
    got = [sg.sagesla_w8a8_token_linear(t, wq, sw) for t in x]
    torch.cuda.synchronize()
    for t, y in zip(x, got):
        q, s = sg.sagesla_w8a8_token_quant(t)
        assert torch.equal(y, sg.sagesla_w8a8_token_gemm(q, s, wq, sw))
    assert sg.sync_status() == 0
