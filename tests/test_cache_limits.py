"""Sizes at the ends of the cache calls' ranges are refused before any launch (CPU, pointers that
nothing follows)."""
import ctypes

import pytest

from diffusion_long_context_b200 import build as focus_build

UNSUPPORTED, INVALID = -2, -1


@pytest.fixture(scope="module")
def F():
    focus_build.build()
    from diffusion_long_context_b200 import focus
    return focus


P = ctypes.c_void_p(4096)


def cache_of(F, n_mat=1, n_pages=4, Hkv=1, page=16, d=64, fmt=0):
    return ctypes.byref(F._CacheStruct(4096, 4096, 4096, 4096, n_mat, n_pages, Hkv, page, d, fmt))


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_attention_over_tables_of_about_2_31_positions(F, page):
    """Positions, page slots and sinks are counted in 32 bits, tiles of 128 at a time."""
    before = F.launch_count()
    for cols in (2 ** 31 // page - 1, (2 ** 31 - 2 ** 18) // page + 1):
        st = F.lib.focus_cache_attention(P, None, cache_of(F, page=page), P, cols, P, 1, 1, 1, 0.1, P, P, 1 << 30, None)
        assert st == INVALID and "positions" in F.last_error()
        st = F.lib.focus_cache_sparse_attention(P, None, cache_of(F, page=page), P, cols, P, P, 16, None, 0, P, 1, 1, 1, 1, 0.1,
                                                P, P, 1 << 30, None)
        assert st == INVALID and "positions" in F.last_error()
    assert F.launch_count() == before


@pytest.mark.parametrize("n_mat,cap", [(1, (2 ** 31 - 1) // 3), (3, (2 ** 31 - 1) // 9), (1, (2 ** 31 - 1) // 3 - 300)])
def test_copies_of_nearly_2_31_pieces(F, n_mat, cap):
    """The pieces are walked in steps of the grid in 32 bits: the last step must not pass 2^31."""
    before = F.launch_count()
    assert F.lib.focus_pages_copy(cache_of(F, n_mat=n_mat), P, P, cap, None) == UNSUPPORTED
    assert "too many" in F.last_error() and F.launch_count() == before


def test_owning_lists_that_name_2_31_table_entries(F):
    """The entries of all listed ranges are counted in 32 bits, a sequence that is listed again anew."""
    pages = ctypes.byref(F._PagesStruct(4096, 4096, 4096, 1 << 20, 2, 1 << 22))
    before = F.launch_count()
    assert F.lib.focus_pages_own(pages, P, P, P, 1024, P, 16, P, P, None) == UNSUPPORTED
    assert "entries" in F.last_error()
    assert F.lib.focus_pages_own(pages, P, P, P, 512, P, 16, P, P, None) == UNSUPPORTED
    pages = ctypes.byref(F._PagesStruct(4096, 4096, 4096, 1 << 20, 1, 2 ** 31 - 1000))      # (the step behind the last entry)
    assert F.lib.focus_pages_own(pages, P, P, P, 1, P, 16, P, P, None) == UNSUPPORTED
    assert F.launch_count() == before
