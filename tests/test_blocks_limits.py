"""What attention over blocks refuses as too much for a launch: in words, before any CUDA call."""
import pytest

import nvfp4_activation_quantize_gb300 as h3q
from nvfp4_activation_quantize_gb300 import build as libbuild


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return h3q.library()


@pytest.mark.parametrize("batch, rows_q, heads, kv_heads, dim, block_q", [
    (1 << 24, 1 << 24, 128, 128, 64, 64),          # a token of each sequence, each head a pair of tiles
    (1, 1 << 30, 1 << 9, 1 << 9, 64, 128),         # 2^30 / 256 pairs of each head
    (1, 1 << 30, 1 << 17, 1 << 10, 128, 256),      # 128 heads a tile, a token each
])
def test_more_units_than_a_launch_has_blocks(lib, batch, rows_q, heads, kv_heads, dim, block_q):
    ld_q, ld_k = heads * dim, kv_heads * dim
    args = [1 << 60, ld_q, 1 << 40, ld_k, 1 << 41, ld_k, 1 << 42, 1 << 43, batch, rows_q, 500, heads, kv_heads, dim, block_q, 64,
            1 << 44, 8, 1, 0.1, 1 << 61, None, None]
    assert lib.h3q_attention_blocks(*args) == h3q.H3Q_ERR_INVALID_ARGUMENT
    assert "2^31" in h3q.h3q_last_error()
