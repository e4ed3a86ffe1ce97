"""The host code of the operators around the linear log-prob under the address and
undefined-behaviour sanitizers (CPU only): llp_api.cpp and llp_api_ops.cpp against stand-in
launchers that touch the ends of every array, driven by tests/sanitize/ops_cases.cpp."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "lm_head_linear_logp_amd", "csrc")
SAN = os.path.join(ROOT, "tests", "sanitize")
SRC = [os.path.join(CSRC, "llp_api.cpp"), os.path.join(CSRC, "llp_api_ops.cpp"),
       os.path.join(SAN, "hip_stub.cpp"), os.path.join(SAN, "ops_stub.cpp"),
       os.path.join(SAN, "ops_cases.cpp")]
HIP_INCLUDE = "/opt/rocm/include"


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(HIP_INCLUDE),
                    reason="needs g++ and the HIP headers")
def test_ops_host_code_under_asan_ubsan(tmp_path):
    exe = str(tmp_path / "ops_cases")
    cmd = ["g++", "-std=c++17", "-g", "-O1", "-fno-omit-frame-pointer",
           "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__",
           f"-I{ROOT}/include", f"-I{CSRC}", f"-I{HIP_INCLUDE}", *SRC, "-o", exe]
    b = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert b.returncode == 0, b.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-6000:]
    assert "Sanitizer" not in out and "runtime error" not in out, out[-6000:]
    assert " 0 failed" in out, out[-2000:]
