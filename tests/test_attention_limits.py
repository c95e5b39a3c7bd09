"""Limits of the cache and attention calls that are refused on the host."""
import pytest

import nvfp4_activation_quantize_gb300 as h3q
from nvfp4_activation_quantize_gb300 import build as libbuild


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return h3q.library()


LISTS = (0x1200000, 0x1201000, 0x1202000)   # (addresses of no memory: every call here is refused)
CACHE = (0x2000000, 0x2100000, 0x2200000, 0x2300000)
SCALES = (0x1203000, 0x1203004)


def _calls(lib, batch):
    return {
        "write": lambda: lib.h3q_kv_cache_write_nvfp4(0x1000000, 256, 0x1100000, 256, 10, *LISTS, batch, 4, *SCALES,
                                                      *CACHE, 16, 16, 2, 128, None),
        "read": lambda: lib.h3q_kv_cache_read_nvfp4(*CACHE, 16, 16, 2, 128, *SCALES, 10, *LISTS, batch, 4, 0x1000000,
                                                    0x1100000, None),
        "cached": lambda: lib.h3q_attention_cache_nvfp4(
            0x1000000, 1024, 10, 8, 4, *LISTS, batch, 4, None, *CACHE, 16, 16, 2, 128, *SCALES, 0.1, 0x3000000, None,
            0x10000000, h3q.attention_cache_workspace_bytes(4, 8, 2, 128), None),
        "varlen": lambda: lib.h3q_attention_varlen(0x1000000, 1024, 0x1100000, 256, 0x1200000, 256, 0x1300000, 0x1301000,
                                                   batch, 10, 12, 8, 2, 128, 1, 0.1, 0x2000000, None, None),
    }


@pytest.mark.parametrize("call", ["write", "read", "cached", "varlen"])
@pytest.mark.parametrize("batch", [2 ** 24 + 1, 2 ** 31 - 1, 2 ** 31, 2 ** 40])
def test_more_sequences_than_the_kernels_count(lib, call, batch):
    """The kernels count sequences in 32 bits, up to a thousand past the last, and a prompt's lookup of its unit
    has to stay far inside the bounded waits."""
    assert _calls(lib, batch)[call]() == h3q.H3Q_ERR_INVALID_ARGUMENT
    assert "batch must be" in h3q.h3q_last_error()
