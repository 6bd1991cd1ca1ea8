"""The size limit of the 4-bit cache's attention that depends on several
arguments together (no GPU needed)."""
import ctypes

import pytest

from attention_forward_gb300 import _build, fa

PAGE = 1024


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fa.load()


def call(lib, B, H, Hkv, Sq, max_pages):
    return lib.fa_fwd_cache(256, 256, 256, 256, 256, 256, 256, 256, 256, B, H, Hkv, Sq, 64, 4, PAGE,
                            max_pages, ctypes.c_float(0.125), 1, ctypes.c_float(0.0), None, None, 0,
                            None)


LIMIT = 2 ** 31 - 256


@pytest.mark.parametrize("B,H,Hkv,Sq,row_blocks", [
    (64, 64, 8, 256, 64 * 8 * 128), (9000, 4, 1, 2, 9000), (12000, 5, 1, 2, 12000),
    (20000, 3, 1, 3, 20000), (32, 256, 16, 64, 32 * 16 * 64)])
def test_more_chunks_than_are_counted(lib, B, H, Hkv, Sq, row_blocks):
    """Refused with the arguments, before any device call."""
    most = LIMIT // (row_blocks * (PAGE // 64))  # pages
    assert (most + 1) * PAGE <= 1 << 24  # within the table's own limit
    assert fa.fa_cache_workspace_bytes(B, H, Hkv, Sq, 64, PAGE, most) > 0
    assert fa.fa_cache_workspace_bytes(B, H, Hkv, Sq, 64, PAGE, most + 1) == 0
    assert call(lib, B, H, Hkv, Sq, most + 1) == fa.FA_ERR_INVALID_ARG


def test_the_largest_table_has_room_for_8191_row_blocks(lib):
    assert fa.fa_cache_workspace_bytes(8191, 1, 1, 1, 64, PAGE, 16384) > 0
    assert fa.fa_cache_workspace_bytes(8192, 1, 1, 1, 64, PAGE, 16384) == 0
    assert call(lib, 8192, 1, 1, 1, 16384) == fa.FA_ERR_INVALID_ARG
