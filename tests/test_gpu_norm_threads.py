"""The norm from several host threads at once (a C++ program: Python's lock would keep the calls apart)."""
import os
import subprocess

import pytest

from preference_alignment_b200 import build as B

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def test_threads_with_different_lengths(tmp_path):
    lib = B.build()
    exe = str(tmp_path / "norm_threads")
    subprocess.run([B._nvcc(), *B.ARCH, "-std=c++17", "-O1", "-I", B.INCLUDE, os.path.join(HERE, "c", "norm_threads.cu"),
                    lib, "-Xlinker", "-rpath," + os.path.dirname(lib), "-lpthread", "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout + out.stderr
