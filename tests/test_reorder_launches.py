"""The launches of beam_reorder at every size (CPU only): llp_api.cpp and llp_api_gen.cpp against a stand-in
launcher that counts threads and states (tests/sanitize/reorder_launches.cpp)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "lm_head_linear_logp_amd", "csrc")
SAN = os.path.join(ROOT, "tests", "sanitize")
SRC = [os.path.join(CSRC, "llp_api.cpp"), os.path.join(CSRC, "llp_api_gen.cpp"),
       os.path.join(SAN, "hip_stub.cpp"), os.path.join(SAN, "reorder_launches.cpp")]
HIP_INCLUDE = "/opt/rocm/include"


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(HIP_INCLUDE),
                    reason="needs g++ and the HIP headers")
def test_no_reorder_launch_holds_2_to_32_threads(tmp_path):
    exe = str(tmp_path / "reorder_launches")
    cmd = ["g++", "-std=c++17", "-g", "-O1", "-D__HIP_PLATFORM_AMD__", f"-I{ROOT}/include", f"-I{CSRC}",
           f"-I{HIP_INCLUDE}", *SRC, "-o", exe]
    b = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert b.returncode == 0, b.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
