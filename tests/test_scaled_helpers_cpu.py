"""What the tensor helpers of the 8-bit layers refuse, on tensors of the host (their data is never read here)."""
import pytest
import torch

import tile_gemm_amd as hts
import tile_gemm_amd.scaled as scaled


@pytest.fixture(autouse=True)
def host_tensors(monkeypatch):
    monkeypatch.setattr(scaled, "_gpu", lambda t, name: t.get_device())


def values(N, K):
    return torch.zeros((N, K), dtype=torch.uint8).view(torch.float8_e4m3fn)


@pytest.mark.parametrize("N,K,scale", [
    (256, 256, lambda: torch.ones((1, 2)).expand(2, 2)),            # one row of scales for all blocks: strides (0, 1)
    (300, 1024, lambda: torch.ones((1, 8)).expand(3, 8)),
    (256, 128, lambda: torch.ones((1, 1)).expand(2, 1)),            # strides (0, 0)
    (256, 64, lambda: torch.ones(1).expand(2, 1)),
    (256, 512, lambda: torch.ones(8).as_strided((2, 4), (2, 1))),   # rows that overlap
])
def test_scales_whose_rows_overlap_are_refused(N, K, scale):
    with pytest.raises(hts.HTSError) as e:
        hts.ScaledWeight(values(N, K), scale())
    assert e.value.status == 3


@pytest.mark.parametrize("N,K,scale,lead", [
    (256, 256, lambda: torch.ones((2, 2)), 2),
    (256, 256, lambda: torch.ones((2, 6))[:, 1:3], 6),
    (256, 128, lambda: torch.ones((1, 2)).t(), 1),                  # [2, 1] of strides (1, 2)
    (256, 100 * 16, lambda: torch.ones((2, 13)), 13),
])
def test_the_rows_own_distance_is_kept(N, K, scale, lead):
    assert hts.ScaledWeight(values(N, K), scale()).desc.ld_scale == lead


@pytest.mark.parametrize("scale", [lambda: torch.ones((1, 3)), lambda: torch.ones((1, 3)).expand(1, 3), lambda: torch.ones((5, 3))[2:3],
                                   lambda: torch.ones(3).as_strided((1, 3), (1, 1))])
def test_a_single_row_may_have_any_distance(scale):
    assert hts.ScaledWeight(values(100, 384), scale()).desc.ld_scale >= 3
