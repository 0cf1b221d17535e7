"""Types that the block-sparse binding does not take are refused as such (no GPU)."""
import pytest
import torch

import paged_kv_cache_406_b200 as P


def test_workspace_size_of_unsupported_pools(native):
    for dtype in (torch.float64, torch.int32, torch.float8_e5m2):
        with pytest.raises(TypeError):
            P.pkv_sparse_workspace_size(2, 8, 2, 128, 16, 16, dtype)
    assert P.pkv_sparse_workspace_size(2, 8, 2, 128, 16, 16, torch.uint8) == 0


@pytest.mark.gpu
def test_select_over_unsupported_bounds(native):
    q, bounds = torch.zeros(1, 2, 64, device="cuda").double(), torch.zeros(4, 1, 2, 64, device="cuda").double()
    t, n = torch.zeros(1, 4, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        P.pkv_block_select(q, bounds, t, n, 2, 16)
