"""The host side of the layer's C ABI under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only): workspace sizes and argument checks over
a sweep of shapes (tests/sanitize/layer_driver.cpp). Only the host pass of
csrc/layer.hip is built, with the device code of an empty source in its place,
since nothing is launched."""
import os
import subprocess
from pathlib import Path

import pytest

from tests.test_sanitizers import SAN, SAN_FLAGS, _run


def test_layer_host_code_under_asan_ubsan(tmp_path):
    from nonlinear_rnn_solve_newton_amd import build

    clang = Path(os.environ.get("ROCM_PATH", "/opt/rocm")) / "lib" / "llvm" / "bin" / "clang++"
    if not clang.exists() or not Path(build.hipcc()).exists():
        pytest.skip("ROCm compilers not available")
    empty, fatbin, lib = tmp_path / "empty.hip", tmp_path / "empty.hipfb", tmp_path / "libpararnn_layer_san.so"
    empty.write_text("#include <hip/hip_runtime.h>\n__global__ void empty_kernel() {}\n")
    subprocess.run([build.hipcc(), *build.COMMON_FLAGS, *build.DEVICE_FLAGS, str(empty), "-o", str(fatbin)], check=True)
    host = []
    for f in SAN_FLAGS:  # each sanitizer flag goes to the host pass only
        host += ["-Xarch_host", f]
    subprocess.run([build.hipcc(), *build.COMMON_FLAGS, *build.HOST_FLAGS, *host, "-Xclang", "-fcuda-include-gpubinary",
                    "-Xclang", str(fatbin), str(build.CSRC / "layer.hip"), "-o", str(lib)], check=True)
    exe = tmp_path / "layer_driver"
    subprocess.run([str(clang), "-std=c++17", *SAN_FLAGS, str(SAN / "layer_driver.cpp"), f"-L{tmp_path}",
                    "-lpararnn_layer_san", f"-Wl,-rpath,{tmp_path}", "-o", str(exe)], check=True)
    # the HIP runtime the library links keeps allocations until exit: no leak report
    out = _run(exe, ASAN_OPTIONS="detect_leaks=0")
    assert "all checks passed" in out
