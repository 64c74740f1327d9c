"""The block-scaled half of the C API (scaled_api.cpp) under AddressSanitizer and UndefinedBehaviorSanitizer, on the CPU:
random and extreme sizes, the workspaces' division and the launches' limits checked by stand-ins for the launchers
(tests/host_sanitize/scaled_driver.cpp), and which kernel the sizes of the GPU tests reach."""
import os
import shutil
import subprocess

import pytest

from scaled_cases import GATED8, SHAPES

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HERE = os.path.join(ROOT, "tests", "host_sanitize")


def _hipcc():
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    return None


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    hipcc = _hipcc()
    if hipcc is None:
        pytest.skip("hipcc not found")
    out = tmp_path_factory.mktemp("scaled")
    common = ["-O1", "-g", "-std=c++17", "--offload-arch=gfx950", f"-I{ROOT}/include",
              f"-I{ROOT}/tile_gemm_amd/csrc", f"-I{HERE}"]
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]
    objs = []
    for src in (f"{ROOT}/tile_gemm_amd/csrc/hts_api.cpp", f"{ROOT}/tile_gemm_amd/csrc/scaled_api.cpp",
                f"{HERE}/launch_stubs.cpp", f"{HERE}/scaled_driver.cpp"):
        obj = str(out / (os.path.basename(src) + ".o"))
        r = subprocess.run([hipcc, *common, *san, "-x", "hip", "-c", src, "-o", obj], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]
        objs.append(obj)
    exe = str(out / "scaled_asan")
    r = subprocess.run([hipcc, "-fsanitize=address,undefined", "-fno-gpu-sanitize", "--offload-arch=gfx950", *objs,
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    return exe


def _run(exe, *args):
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe, *map(str, args)], capture_output=True, text=True, env=env, timeout=600)
    text = r.stdout + r.stderr
    assert "AddressSanitizer" not in text and "runtime error" not in text, text[-4000:]
    assert r.returncode == 0, text[-4000:]
    return r.stdout


def test_scaled_entry_points_are_clean_under_asan_and_ubsan(driver):
    assert "expectations failed: 0, stub checks failed: 0" in _run(driver)


def test_the_gpu_tests_reach_every_kernel(driver):
    names = ["stream", "ring 32x16", "ring 64x16", "ring 32x32", "ring 64x32", "ring 64x64", "ring 128x64", "ring 128x128",
             "tile 128x128", "tile 256x128", "tile 256x256"]
    for gated, out8, shapes in ((0, 0, SHAPES), (1, 0, SHAPES), (1, 1, GATED8)):
        args = [v for s in shapes for v in (*s, gated, out8)]
        got = [tuple(map(int, line.split())) for line in _run(driver, "--kernels", *args).splitlines()]
        reached = {names[k] for k, _ in got}
        if not out8:
            assert reached == set(names), (gated, sorted(set(names) - reached), list(zip(shapes, got)))
        assert any(s > 1 for _, s in got) and any(s == 1 for _, s in got)
