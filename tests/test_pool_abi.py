"""The page pool's entry points without a GPU."""
import ctypes

import pytest

from fp8_scaled_gemm_sm_gb300 import binding, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


def test_null_handles_are_refused(lib):
    pool = binding.PagePoolArgs()
    p = ctypes.byref(pool)
    assert lib.scaled_attn_pool_release(None, p, None, 0, None) == 1
    assert lib.scaled_attn_pool_grow(None, p, None, None, 0, None, None) == 1
    assert lib.scaled_attn_pool_fork(None, p, None, 0, None, None, 0, None, None) == 1
    assert lib.scaled_attn_pool_compact(None, p, None, 0, None, None) == 1


def test_scratch(lib):
    size = binding.scaled_attn_pool_scratch_bytes
    assert size(-1, 4) == 0 and size(4, -1) == 0 and size(1 << 31, 1) == 0
    for rows, pages in ((0, 0), (1, 1), (7, 1000), (1000, 7)):
        # counters, two words a row, one a page, and a move of two words for each row or page
        assert size(rows, pages) >= 16 + 8 * rows + 4 * pages + 8 * max(rows, pages)


def test_rows_and_pages_counted_in_32_bits(lib):
    most = (1 << 31) - 1 - 65536
    size = binding.scaled_attn_pool_scratch_bytes
    assert size(most, 1) > 0 and size(1, most) > 0
    assert size(most + 1, 1) == 0 and size(1, most + 1) == 0
