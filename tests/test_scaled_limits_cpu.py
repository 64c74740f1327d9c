"""The sizes that the block-scaled products take, at the limits that hts.h states: M and N below 2^26 and ceil(M / 128) *
ceil(N / 128) below 2^22."""
import ctypes

import pytest

import tile_gemm_amd as hts

TOP = (1 << 26) - 1


@pytest.mark.parametrize("M,N,ok", [
    (896, TOP, True), (897, TOP, False), (TOP, 896, True), (TOP, 897, False),                # 7 and 8 times 2^19
    (128 * 2048, 128 * 2047, True), (128 * 2048, 128 * 2047 + 1, False), (128 * 2047 + 1, 128 * 2048, False),
    (1, TOP, True), (1, TOP + 1, False), (TOP, 1, True), (TOP + 1, 1, False),
])
def test_limits(M, N, ok):
    n = ctypes.c_size_t(0)
    by = ctypes.byref(n)
    want = 0 if ok else 7
    assert hts.lib().hts_scaled_gemm_workspace(M, N, 128, by) == want
    assert hts.lib().hts_scaled_gated_workspace(M, N, 128, hts.HTS_BF16, by) == want
    text = hts.lib().hts_last_error().decode()
    assert ok or "2^22" in text
