"""The C ABI around the paged cache (include/qdr_cache.h) without a GPU: exported
names, null handles, frequencies, and every refusal of the host side under
AddressSanitizer / UBSan (tests/native/cache_sanitize.cpp)."""
import ctypes
import math
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

from quantized_delta_rule_decode_amd import qdr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(qdr.LIB_PATH):
        from quantized_delta_rule_decode_amd import build
        build.build()
    return qdr.load()


def test_exports_every_declared_symbol(lib):
    text = open(os.path.join(ROOT, "include", "qdr_cache.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\bqdr_status\s+(qdr_[a-z0-9_]+)\s*\(", text)))
    assert names == sorted(qdr.CACHE_EXPORTS)
    for n in names:
        assert hasattr(lib, n), n


def test_null_handles_rejected(lib):
    n = ctypes.c_size_t(0)
    assert lib.qdr_rotary_create(None, None) == -1
    assert lib.qdr_rotary_destroy(None) == 0
    assert lib.qdr_rotate(None, None, 0, 1, None, 128, None, 128, None) == -1
    assert lib.qdr_rotate_bf16(None, None, 0, 1, None, 128, None, 128, None) == -1
    assert lib.qdr_kv_write_rotary(None, None, None, 0, None, None, 0, 0, None, 0, 0, None, None, 128, None, 128, None) == -1
    assert lib.qdr_kv_copy(None, None, None, None, 0, None) == -1
    assert lib.qdr_slot_copy(None, None, None, 0, None) == -1
    assert lib.qdr_kv_assign_workspace(None, 1, ctypes.byref(n)) == -1
    assert lib.qdr_kv_assign(None, None, None, 0, 0, None, None, 0, None, None, None, None, None, 0, None) == -1
    assert lib.qdr_kv_compact_workspace(None, ctypes.byref(n)) == -1
    assert lib.qdr_kv_compact(None, None, None, 0, 0, None, None, None, None, 0, None) == -1
    assert lib.qdr_kv_attend_shared_workspace(None, 1, 1, 1, 1, 1, ctypes.byref(n)) == -1
    assert lib.qdr_kv_attend_shared(None, None, 0, None, None, 0, 0, None, None, 0, 1, None, 1.0, None, None, 0, None) == -1
    assert lib.qdr_last_error() != b""


@pytest.mark.parametrize("channels", [16, 64, 128])
def test_frequencies(lib, channels):
    """The four rules against their definitions."""
    base, factor, context = 10000.0, 8.0, 4096.0
    f = np.array([base ** (-2 * i / channels) for i in range(channels // 2)])
    plain, one = qdr.qdr_rotary_frequencies(qdr.ROTARY_PLAIN, channels, base)
    assert np.allclose(plain, f, rtol=4e-16) and one == 1
    linear, one = qdr.qdr_rotary_frequencies(qdr.ROTARY_LINEAR, channels, base, factor)
    assert np.allclose(linear, f / factor, rtol=4e-16) and one == 1
    turns, one = qdr.qdr_rotary_frequencies(qdr.ROTARY_TURNS, channels, base, factor, context, 1.0, 4.0)
    k = np.clip((context * f / (2 * math.pi) - 1) / 3, 0, 1)
    assert np.allclose(turns, k * f + (1 - k) * f / factor, rtol=1e-14) and one == 1
    index, amplitude = qdr.qdr_rotary_frequencies(qdr.ROTARY_INDEX, channels, base, factor, context, 1.0, 32.0)
    at = [channels * math.log(context / (2 * math.pi * w)) / (2 * math.log(base)) for w in (32, 1)]
    a, b = max(math.floor(at[0]), 0), min(math.ceil(at[1]), channels - 1)
    k = 1 - np.clip((np.arange(channels // 2) - a) / max(b - a, 0.001), 0, 1)
    assert np.allclose(index, k * f + (1 - k) * f / factor, rtol=1e-14) and abs(amplitude - (0.1 * math.log(factor) + 1)) < 1e-15
    for bad in (dict(channels=24), dict(base=1.0), dict(factor=0.0), dict(context=-1.0), dict(low=5.0, high=4.0)):
        with pytest.raises(qdr.QdrError):
            qdr.qdr_rotary_frequencies(qdr.ROTARY_TURNS, **{**dict(channels=channels, factor=2.0), **bad})


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(os.path.join(ROCM, "include")),
                    reason="g++ or the HIP headers are not available")
def test_host_side_under_asan_ubsan(tmp_path):
    exe = str(tmp_path / "cache_sanitize")
    build = ["g++", "-g", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-std=c++17",
             "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROCM, "include"),
             os.path.join(ROOT, "quantized_delta_rule_decode_amd", "csrc", "qdr_cache.cpp"),
             os.path.join(ROOT, "tests", "native", "cache_sanitize.cpp"), "-o", exe]
    r = subprocess.run(build, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and r.stdout.startswith("ok "), out
    assert "runtime error" not in out, out
