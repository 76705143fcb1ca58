"""The scratch of the attention over a cache: the library's own rule for its
chunks against the sizes that the library asks for."""
import os
import subprocess

from learnable_butterfly_rotation_amd import build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_the_chunks_lie_in_the_workspace_and_the_grid(tmp_path):
    exe = str(tmp_path / "attend_cut")
    subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-Wall", "-Werror",
                    "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I" + build.CSRC,
                    os.path.join(HERE, "san", "attend_cut.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and "cuts hold" in r.stdout, r.stdout + r.stderr
