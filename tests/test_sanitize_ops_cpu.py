"""The host layer of the norm, the adapters and the clipping (bfly_api.hip:
argument validation, size queries) under AddressSanitizer and
UndefinedBehaviorSanitizer, driven by tests/san/ops_san.c through calls that
are rejected, or are pure size queries, before any HIP call.  The device code
is not instrumented."""
import os

import pytest

from learnable_butterfly_rotation_amd import build as B
from test_sanitize_cpu import CLANG, ROOT, SAN, run


def test_ops_host_layer_under_sanitizers(tmp_path):
    objs = [os.path.join(B.OBJ, o) for src, o, _ in B.SOURCES if src != "bfly_api.hip"]
    if not all(os.path.exists(o) for o in objs):
        pytest.skip("the library's objects are not built")
    if not (os.path.exists(B.HIPCC) and os.path.exists(CLANG)):
        pytest.skip("the ROCm compilers are not installed")
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined"]
    api, lib = str(tmp_path / "bfly_api_san.o"), str(tmp_path / "libbfly_san.so")
    flags = [f for f in B.FLAGS if f != "-O3"]
    run([B.HIPCC, "-O1", "-g", *flags, *san, "-Xarch_host", "-fno-sanitize-recover=all",
         "-Xarch_host", "-fno-omit-frame-pointer", "-c",
         os.path.join(B.CSRC, "bfly_api.hip"), "-o", api])
    run([B.HIPCC, "-shared", "-fPIC", "--offload-arch=gfx950", *san, "-shared-libsan", api, *objs,
         "-o", lib])
    rt = os.path.dirname(run([CLANG, "-print-file-name=libclang_rt.asan-x86_64.so"]).stdout.strip())
    exe = str(tmp_path / "ops_san")
    run([CLANG + "++", "-x", "c", "-O1", "-g", "-fsanitize=address,undefined",
         "-fno-sanitize-recover=all", "-shared-libsan", "-I" + os.path.join(ROOT, "include"),
         os.path.join(SAN, "ops_san.c"), "-L" + str(tmp_path), "-lbfly_san",
         "-Wl,-rpath," + str(tmp_path), "-Wl,-rpath," + rt, "-o", exe])
    r = run([exe], env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    assert "all checks passed" in r.stdout
