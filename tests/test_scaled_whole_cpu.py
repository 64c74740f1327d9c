"""Which kernels the sizes of tests/scaled_whole_cases.py reach, and the host code of 32-bit outputs under sanitizers, on the CPU."""
import subprocess

import pytest

from scaled_cases import SHAPES
from scaled_whole_cases import E4M3_ROWS, ONCE, PARTS_OF_BATCHES
from test_host_sanitize_scaled import HERE, ROOT, _hipcc, _run, driver  # noqa: F401

NAMES = ["stream", "ring 32x16", "ring 64x16", "ring 32x32", "ring 64x32", "ring 64x64", "ring 128x64", "ring 128x128",
         "tile 128x128", "tile 256x128"]


def _kernels(exe, args):
    return [tuple(map(int, line.split())) for line in _run(exe, "--kernels", *args).splitlines()]


def test_the_gpu_tests_reach_every_kernel_of_e4m3_rows(driver):  # noqa: F811
    got = _kernels(driver, [v for s in E4M3_ROWS for v in (*s, 1, 1)])
    reached = {NAMES[k] for k, _ in got}
    assert reached == set(NAMES), (sorted(set(NAMES) - reached), list(zip(E4M3_ROWS, got)))
    assert any(s > 1 for _, s in got) and any(s == 1 for _, s in got)


@pytest.fixture(scope="module")
def f32_driver(driver, tmp_path_factory):  # noqa: F811
    """The same objects with another main (the first driver's is part of it)."""
    import os
    built, out = os.path.dirname(driver), tmp_path_factory.mktemp("scaled_f32")
    obj, exe = str(out / "driver.o"), str(out / "scaled_f32")
    cmd = [_hipcc(), "-O1", "-g", "-std=c++17", "--offload-arch=gfx950", f"-I{ROOT}/include", f"-I{ROOT}/tile_gemm_amd/csrc", f"-I{HERE}",
           "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=all",
           "-Xarch_host", "-fno-omit-frame-pointer", "-x", "hip", "-c", f"{HERE}/scaled_f32_driver.cpp", "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    objs = [os.path.join(built, n + ".o") for n in ("hts_api.cpp", "scaled_api.cpp", "launch_stubs.cpp")]
    r = subprocess.run([_hipcc(), "-fsanitize=address,undefined", "-fno-gpu-sanitize", "--offload-arch=gfx950", *objs, obj, "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    return exe


def test_32_bit_outputs_are_clean_under_asan_and_ubsan(f32_driver):
    assert "expectations failed: 0, stub checks failed: 0" in _run(f32_driver)


def test_the_gpu_tests_reach_every_kernel_of_32_bit_outputs(f32_driver):
    for gated in (0, 1):
        got = _kernels(f32_driver, [v for s in SHAPES for v in (*s, gated)])
        reached = {NAMES[k] for k, _ in got}
        assert reached == set(NAMES), (gated, sorted(set(NAMES) - reached), list(zip(SHAPES, got)))
        assert any(s > 1 for _, s in got) and any(s == 1 for _, s in got)


def test_the_gpu_tests_reach_every_ring_on_weights_read_once(driver, f32_driver):  # noqa: F811
    rows = {"ring 32x16": 16, "ring 64x16": 16, "ring 32x32": 32, "ring 64x32": 32, "ring 64x64": 64, "ring 128x64": 64, "ring 128x128": 128}
    for (op, out), shapes in ONCE.items():
        gated = int(op == "gated")
        if out == "32":
            got = _kernels(f32_driver, [v for s in shapes for v in (*s, gated)])
        else:
            got = _kernels(driver, [v for s in shapes for v in (*s, gated, int(out == "8"))])
        names = [NAMES[k] for k, _ in got]
        assert set(names) == set(rows) - ({"ring 128x128"} if out != "16" else set()), (op, out, names)
        assert all(M <= rows[n] and N * K * (1 + gated) >= 64 << 20 for n, (M, N, K) in zip(names, shapes))


def test_parts_of_batches_share_their_kernel(driver):  # noqa: F811
    for rows, part, N, K in PARTS_OF_BATCHES:
        a, b = _kernels(driver, [rows, N, K, 0, 0, part, N, K, 0, 0])
        assert a == b, (rows, part, N, K, a, b)
