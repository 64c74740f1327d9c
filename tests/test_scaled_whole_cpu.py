"""Which kernels the sizes of tests/scaled_whole_cases.py reach, on the CPU."""
from scaled_whole_cases import E4M3_ROWS
from test_host_sanitize_scaled import _run, driver  # noqa: F401

NAMES = ["stream", "ring 32x16", "ring 64x16", "ring 32x32", "ring 64x32", "ring 64x64", "ring 128x64", "ring 128x128",
         "tile 128x128", "tile 256x128"]


def test_the_gpu_tests_reach_every_kernel_of_e4m3_rows(driver):  # noqa: F811
    got = [tuple(map(int, line.split())) for line in
           _run(driver, "--kernels", *[v for s in E4M3_ROWS for v in (*s, 1, 1)]).splitlines()]
    reached = {NAMES[k] for k, _ in got}
    assert reached == set(NAMES), (sorted(set(NAMES) - reached), list(zip(E4M3_ROWS, got)))
    assert any(s > 1 for _, s in got) and any(s == 1 for _, s in got)
