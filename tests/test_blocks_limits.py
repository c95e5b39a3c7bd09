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


def test_workspace_of_many_key_blocks(lib, tmp_path):
    """The binding's bytes are the header's below and above 16,000 key blocks, and one byte less is refused."""
    import os
    import subprocess

    shapes = [(1000, 16_000 * 64 + 63, 3, 8, 128, 64, 64), (16, 16_001 * 64, 16, 8, 128, 64, 64),
              (90_000, 1 << 25, 7, 4, 64, 128, 256), (16, 1 << 25, 16, 2, 64, 64, 64)]
    lines = "".join('printf("%lld\\n", (long long)h3q_select_blocks_workspace_bytes(' + ", ".join(map(str, s)) + "));"
                    for s in shapes)
    src = tmp_path / "w.c"
    src.write_text('#include "h3q.h"\n#include <stdio.h>\nint main(void) { ' + lines + " return 0; }\n")
    exe = str(tmp_path / "w")
    subprocess.run(["gcc", "-I", os.path.dirname(libbuild.HEADER), str(src), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in out] == [h3q.select_blocks_workspace_bytes(*s) for s in shapes]
    for (rows_q, rows_k, batch, kv_heads, dim, block_q, block_k), need in zip(shapes, map(int, out)):
        ld = kv_heads * dim
        args = [1 << 40, ld, 1 << 41, ld, 1 << 42, (1 << 42) + (1 << 30), batch, rows_q, rows_k, kv_heads, kv_heads, dim, block_q,
                block_k, 8, 0, 1, 1 << 43, None, 1 << 44, need - 1, None]
        assert lib.h3q_select_blocks(*args) == h3q.H3Q_ERR_INVALID_ARGUMENT
        assert "workspace_bytes" in h3q.h3q_last_error()
        assert ("16,000" in h3q.h3q_last_error()) == (rows_k // block_k > 16_000)
