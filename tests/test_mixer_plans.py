"""How attention calls are planned on the host (tests/native/mixer_plans.cpp), without a GPU."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(os.path.join(ROCM, "include")),
                    reason="g++ or the HIP headers are not available")
def test_plans(tmp_path):
    exe = str(tmp_path / "mixer_plans")
    r = subprocess.run(["g++", "-g", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-std=c++17",
                        "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROCM, "include"),
                        os.path.join(ROOT, "quantized_delta_rule_decode_amd", "csrc", "qdr_mixer.cpp"),
                        os.path.join(ROOT, "tests", "native", "mixer_plans.cpp"), "-o", exe],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and r.stdout.startswith("ok "), out
    assert "runtime error" not in out, out
