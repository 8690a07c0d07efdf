"""Addresses that are no memory of a device never reach a launch.  On the CPU the library runs on a fake CUDA runtime (one
sm_100 device, launches counted and not run); on a GPU the same calls are made with host memory."""
import ctypes
import os
import subprocess
import sys

import pytest

from tests._fake import ROOT, fake  # noqa: F401


CALLS = """
import ctypes, sys
sys.path.insert(0, %r)
fake = ctypes.CDLL(%r, mode=ctypes.RTLD_GLOBAL)
import sparse_bit_attention_smoothing_b200 as sg
L, F, P = sg.lib(), ctypes.c_float, ctypes.c_void_p
A, BAD = P(0x10000), P(0x900000)
attn = lambda a: (a, a, a, a, a)
calls = {
    "attn": lambda a: L.sagesla_attn(a[0], a[1], a[2], a[3], a[4], 1, 1, 256, 128, 64, F(0.3), None),
    "opts": lambda a: L.sagesla_attn_opts(a[0], a[1], a[2], a[3], a[4], 1, 1, 256, 128, 64, F(0.3), 4, 1, None),
    "qknorm": lambda a: L.sagesla_attn_qknorm(a[0], a[1], A, a[2], a[3], F(1e-6), None, a[4], 1, 1, 256, 128, 64, F(0.3), None),
    "bnhd": lambda a: L.sagesla_attn_bnhd(a[0], a[1], A, a[2], a[3], F(1e-6), A, a[4], 1, 256, 1, 128, 64, F(0.3), None),
    "dense": lambda a: L.dense_int8_attn(a[0], a[1], a[2], a[3], 1, 1, 256, 128, None),
    "mask": lambda a: L.sagesla_get_mask(a[0], a[1], 1, 1, 256, 128, 64, F(0.3), a[2], a[3], a[4], None, None),
    "quant": lambda a: L.sagesla_get_quant(a[0], a[1], a[2], 1, 1, 256, 128, a[3], A, A, a[4], A, A, A, None),
    "w8a8_quant": lambda a: L.sagesla_w8a8_quant(a[0], 128, 128, a[1], a[2], None),
    "w8a8_gemm": lambda a: L.sagesla_w8a8_gemm(a[0], a[1], a[2], a[3], a[4], 128, 128, 128, None),
    "w8a8_linear": lambda a: L.sagesla_w8a8_linear(a[0], a[1], a[2], a[3], 128, 128, 128, None),
}
used = {"dense": 4, "w8a8_quant": 3, "w8a8_linear": 4}
fake.fake_known(ctypes.c_size_t(0x10000), ctypes.c_size_t(0x20000))
for name, f in calls.items():
    n = fake.fake_launches()
    for i in range(used.get(name, 5)):
        rc = f([BAD if j == i else A for j in range(5)])
        assert rc == -7, (name, i, rc)
    assert fake.fake_launches() == n, name
    if name in ("attn", "dense", "mask", "w8a8_quant"):  # with memory everywhere the same calls launch
        assert f([A] * 5) == 0 and fake.fake_launches() > n, name
print("ok", fake.fake_launches())
"""


def test_no_launch_on_unknown_addresses(fake):  # noqa: F811
    r = subprocess.run([sys.executable, "-c", CALLS % (ROOT, fake)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("ok"), (r.stdout, r.stderr[-2000:])


PLUGIN = """
import ctypes
fake = ctypes.CDLL({fake!r}, mode=ctypes.RTLD_GLOBAL)
def pytest_sessionfinish(session):
    print("\\nlaunches", fake.fake_launches())
"""


@pytest.mark.parametrize("only", ["test_abi.py -k rejects", "test_abi_layer.py"])
def test_argument_checks_launch_nothing(fake, only):  # noqa: F811
    """The tests of refused arguments, whose pointers are not memory, on a machine that has the device: they pass and launch
    nothing."""
    work = os.path.join(ROOT, "_build")
    with open(os.path.join(work, "fake_runtime_plugin.py"), "w") as f:
        f.write(PLUGIN.format(fake=fake))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([work, os.environ.get("PYTHONPATH", "")]))
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-s", "-p", "fake_runtime_plugin",
                        *os.path.join(ROOT, "tests", only).split()], capture_output=True, text=True, timeout=300, env=env, cwd=ROOT)
    assert r.returncode == 0 and " passed" in r.stdout and "launches 0\n" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]


@pytest.mark.gpu
def test_host_memory_is_refused_on_the_device():
    """Tensors in host memory: an error, and the context stays usable."""
    import torch
    import sparse_bit_attention_smoothing_b200 as sg
    host = torch.zeros(1, 1, 256, 128, dtype=torch.bfloat16)
    dev = torch.randn(1, 1, 256, 128, device="cuda").to(torch.bfloat16)
    want = sg.sagesla_attn(dev, dev, dev)
    for i in range(4):
        t = [host if i == j else dev for j in range(4)]
        with pytest.raises(sg.SageSLAError) as e:
            sg.sagesla_attn(t[0], t[1], t[2], out=t[3])
        assert e.value.code == -7
    with pytest.raises(sg.SageSLAError) as e:
        sg.sagesla_w8a8_linear(torch.zeros(128, 128, dtype=torch.bfloat16), dev, dev, N=128, y=dev)
    assert e.value.code == -7
    lim, a = 786432, ctypes.c_void_p(host.data_ptr() // 16 * 16)
    assert sg.lib().sagesla_attn(a, a, a, None, a, 1, 1, lim, 128, 64, ctypes.c_float(0.1), None) == -7
    side = torch.cuda.Stream()
    sg.sagesla_attn(dev, dev, dev, stream=side)  # the stream's workspace
    torch.cuda.synchronize()
    g, got = torch.cuda.CUDAGraph(), torch.empty_like(dev)
    with torch.cuda.graph(g, stream=side):  # the checks are open to a capture
        sg.sagesla_attn(dev, dev, dev, out=got, stream=side)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and sg.sync_status() == 0


ALLOCATOR = """
import torch, sparse_bit_attention_smoothing_b200 as sg
x = torch.randn(1, 2, 300, 128, device="cuda").bfloat16()
w = torch.randn(128, 128, device="cuda").bfloat16()
out = sg.sagesla_attn(x, x[:, :1].expand_as(x).contiguous(), x, w, topk=0.3)
torch.cuda.synchronize()
assert torch.isfinite(out).all() and sg.sync_status() == 0
print("taken")
"""


@pytest.mark.gpu
@pytest.mark.parametrize("conf", ["expandable_segments:True", "backend:cudaMallocAsync", "backend:native"])
def test_memory_of_every_allocator_is_known(conf):
    env = dict(os.environ, PYTORCH_CUDA_ALLOC_CONF=conf, PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", ALLOCATOR], capture_output=True, text=True, timeout=300, env=env, cwd=ROOT)
    assert r.returncode == 0 and "taken" in r.stdout, r.stderr[-2000:]
