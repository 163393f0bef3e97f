"""The index arithmetic of the streaming statistics' lists, compiled for the host and run there."""
import os
import subprocess

from preference_alignment_b200 import build as B

HERE = os.path.dirname(os.path.abspath(__file__))


def test_every_id_names_a_list_within_bounds(tmp_path):
    exe = str(tmp_path / "stream_lists")
    subprocess.run([B._nvcc(), *B.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", B.CSRC, "-I", B.INCLUDE,
                    os.path.join(HERE, "c", "stream_lists.cu"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout
