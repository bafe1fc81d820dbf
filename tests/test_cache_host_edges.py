"""What the paged-cache entry points refuse at the edges of their ranges, on the host (no GPU
needed: only calls that fail validation are made)."""

import pytest
import torch

import kv_cache_eviction_scores_b200 as dk
from test_cache_host import _attend, _attn, _cache


@pytest.mark.parametrize("scale", [1e-46, 1e39, 0.0, -1.0, float("nan"), float("inf")])
def test_scales_that_fp32_does_not_hold_are_refused(scale):
    # 1e-46 is 0 in fp32, which means the default to the library
    pages, x = torch.zeros(4, 2, 16, 8), torch.zeros(1, 2, 5, 8)
    table, n = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="scale"):
        dk.dropkv_cache_attention(x, pages, pages, table, n, scale=scale)


def test_a_scale_that_overflows_in_units_of_log2_is_refused():
    assert _attend(_cache(), _attn(scale=2.5e38)) == dk.ERR_ARG
    if not torch.cuda.is_available():
        for fine in (2.3e38, 1e-45):
            assert _attend(_cache(), _attn(scale=fine)) == dk.ERR_UNSUPPORTED
