"""The serving half of the C API (serve_api.cpp) under AddressSanitizer and UndefinedBehaviorSanitizer, on the CPU:
extreme sizes, random cache descriptions and rotary plans, and the workspace division of the attention checked by
a stand-in for its launcher (tests/host_sanitize/serve_driver.cpp)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HERE = os.path.join(ROOT, "tests", "host_sanitize")


def _hipcc():
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    return None


def test_serving_entry_points_are_clean_under_asan_and_ubsan(tmp_path):
    hipcc = _hipcc()
    if hipcc is None:
        pytest.skip("hipcc not found")
    common = ["-O1", "-g", "-std=c++17", "--offload-arch=gfx950", f"-I{ROOT}/include",
              f"-I{ROOT}/tile_gemm_amd/csrc", f"-I{HERE}"]
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]
    objs = []
    for src in (f"{ROOT}/tile_gemm_amd/csrc/hts_api.cpp", f"{ROOT}/tile_gemm_amd/csrc/serve_api.cpp", f"{HERE}/launch_stubs.cpp",
                f"{HERE}/serve_driver.cpp"):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        r = subprocess.run([hipcc, *common, *san, "-x", "hip", "-c", src, "-o", obj], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]
        objs.append(obj)
    exe = str(tmp_path / "serve_asan")
    r = subprocess.run([hipcc, "-fsanitize=address,undefined", "-fno-gpu-sanitize", "--offload-arch=gfx950", *objs,
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=600)
    text = r.stdout + r.stderr
    assert "AddressSanitizer" not in text and "runtime error" not in text, text[-4000:]
    assert r.returncode == 0, text[-4000:]
    assert "expectations failed: 0, stub checks failed: 0" in r.stdout
