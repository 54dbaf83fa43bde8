"""The token mixers' part of the C ABI (include/qdr_mixer.h) without a GPU:
exported names, null handles, sizes, and every refusal of the host side under
AddressSanitizer / UBSan (tests/native/mixer_sanitize.cpp)."""
import ctypes
import os
import re
import shutil
import subprocess

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
    text = open(os.path.join(ROOT, "include", "qdr_mixer.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\bqdr_status\s+(qdr_[a-z0-9_]+)\s*\(", text)))
    assert names == sorted(qdr.MIXER_EXPORTS)
    for n in names:
        assert hasattr(lib, n), n


def test_null_handles_rejected(lib):
    n = ctypes.c_size_t(0)
    assert lib.qdr_prompt(None, 0, None, None, None, 0, 0, None, None, None, None, None, None, None, 0, None) == -1
    assert lib.qdr_prompt_workspace(None, 1, 1, ctypes.byref(n)) == -1
    assert lib.qdr_linear_step(None, None, 0, None, None, None, None, None, None) == -1
    assert lib.qdr_linear_step_bf16(None, None, 0, None, None, None, None, None, None) == -1
    assert lib.qdr_kv_bytes(None, ctypes.byref(n)) == -1
    assert lib.qdr_kv_create(None, None, 0, None) == -1
    assert lib.qdr_kv_destroy(None) == 0
    assert lib.qdr_kv_write(None, None, 0, None, None, 0, 0, None, None, None) == -1
    assert lib.qdr_kv_read(None, None, 0, None, None, 0, 0, None, None, None) == -1
    assert lib.qdr_kv_attend(None, None, 0, None, None, 0, 0, 1, None, 1.0, None, None, 0, None) == -1
    assert lib.qdr_kv_attend_workspace(None, 1, 1, 1, 1, ctypes.byref(n)) == -1
    assert lib.qdr_kv_poll_device_error(None, None) == -1
    assert lib.qdr_last_error() != b""


@pytest.mark.parametrize("page", [32, 64, 128, 256, 512, 1024])
@pytest.mark.parametrize("kind,token", [(8, 2 * (128 + 4)), (16, 2 * 256)])
def test_cache_bytes(lib, page, kind, token):
    """Codes (or values) of every token and head, and two scales for 8 bits."""
    assert qdr.qdr_kv_bytes(7, page, 3, kind) == 7 * page * 3 * token


@pytest.mark.parametrize("bad", [dict(num_pages=0), dict(page_tokens=16), dict(page_tokens=96), dict(num_heads=-1), dict(kind=4)])
def test_cache_descriptor_errors(lib, bad):
    kw = dict(num_pages=2, page_tokens=64, num_heads=2, kind=8)
    kw.update(bad)
    with pytest.raises(qdr.QdrError) as ei:
        qdr.qdr_kv_bytes(**kw)
    assert ei.value.status == -1 and str(ei.value)


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(os.path.join(ROCM, "include")),
                    reason="g++ or the HIP headers are not available")
def test_host_side_under_asan_ubsan(tmp_path):
    exe = str(tmp_path / "mixer_sanitize")
    build = ["g++", "-g", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-std=c++17",
             "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROCM, "include"),
             os.path.join(ROOT, "quantized_delta_rule_decode_amd", "csrc", "qdr_mixer.cpp"),
             os.path.join(ROOT, "tests", "native", "mixer_sanitize.cpp"), "-o", exe]
    r = subprocess.run(build, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and r.stdout.startswith("ok "), out
    assert "runtime error" not in out, out
