"""The fake CUDA runtime of fake_runtime.c, for programs that load it before the library."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = os.path.join(ROOT, "_build", "libfake_runtime.so")


@pytest.fixture(scope="module")
def fake():
    from sparse_bit_attention_smoothing_b200 import build
    build.build()
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    os.makedirs(os.path.dirname(FAKE), exist_ok=True)
    subprocess.run([cc, "-O1", "-shared", "-fPIC", os.path.join(ROOT, "tests", "fake_runtime.c"), "-o", FAKE], check=True)
    return FAKE
