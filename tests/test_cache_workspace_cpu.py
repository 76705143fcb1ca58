"""The scratch of the attention over a cache: the library's own rule for its
chunks against the sizes that the library asks for."""
import os
import subprocess

import pytest

import learnable_butterfly_rotation_amd as B
from learnable_butterfly_rotation_amd import build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_the_chunks_lie_in_the_workspace_and_the_grid(tmp_path):
    exe = str(tmp_path / "attend_cut")
    subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-Wall", "-Werror",
                    "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I" + build.CSRC,
                    os.path.join(HERE, "san", "attend_cut.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and "cuts hold" in r.stdout, r.stdout + r.stderr


def test_the_size_never_falls_while_the_key_value_heads_stay():
    if not os.path.exists(B.library_path):
        pytest.skip("libbfly.so not built")
    size = B.bfly_cache_attention_workspace_bytes
    for kv in (1, 3, 8, 40):
        for rows in (1, 3, 70):
            for d in (64, 128, 256):
                for most in (513, 1000, 8192, 1 << 20):
                    # past 16 and 32 query heads to a key-value head, and one more row
                    sizes = [size(rows, kv * i, kv, d, most) for i in range(1, 41)]
                    assert all(a <= b for a, b in zip(sizes, sizes[1:])), (kv, rows, d, most)
                    assert sizes[0] > 0 and all(
                        s <= size(rows + 1, kv * i, kv, d, most) for i, s in enumerate(sizes, 1))
    # with more key-value heads it may fall: layers that differ in them take the larger
    assert size(1, 64, 64, 128, 1 << 20) < size(1, 32, 8, 128, 1 << 20)
