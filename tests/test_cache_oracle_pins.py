"""The cache oracle's own pins (CPU): codes against torch's conversions, brute force for pages,
and the refusals of the cache calls, none of which reaches a GPU."""
import ctypes
import random

import numpy as np
import pytest
import torch

from diffusion_long_context_b200 import build as focus_build
from oracle import cache_oracle as orc


@pytest.fixture(scope="module")
def F():
    focus_build.build()
    from diffusion_long_context_b200 import focus
    return focus


def test_e4m3_values_match_torch():
    t = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(t, orc.E4M3_VALUES)


def test_nearest_e4m3_matches_torch_with_ties():
    g = orc.E4M3_VALUES[:127]
    mid = ((g[1:] + g[:-1]) / 2).astype(np.float32)          # exact: five significant bits
    y = np.concatenate([mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(1e9)), g.astype(np.float32)])
    rng = np.random.default_rng(1)
    y = np.concatenate([y, -y, rng.uniform(-448, 448, 20000).astype(np.float32),
                        np.exp2(rng.uniform(-12, 8, 20000)).astype(np.float32)])
    exp = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(orc.nearest_codes(y, orc.E4M3), exp)


def test_nearest_int8_matches_torch():
    y = np.concatenate([np.arange(-127.5, 128, 0.5), np.random.default_rng(2).uniform(-127, 127, 5000)]).astype(np.float32)
    exp = torch.from_numpy(y).round().clamp(-127, 127).to(torch.int8).numpy().view(np.uint8)
    np.testing.assert_array_equal(orc.nearest_codes(y, orc.INT8), exp)


@pytest.mark.parametrize("fmt", [orc.E4M3, orc.INT8])
def test_encode_is_within_half_a_step(fmt):
    x = np.random.default_rng(3).standard_normal((3, 64, 128)).astype(np.float32)
    s = orc.page_scale(x, fmt)[..., None, None]
    back = orc.code_values(orc.encode(x, s, fmt), fmt) * s
    step = s if fmt == orc.INT8 else np.maximum(np.abs(x) / 8, s * 2.0 ** -9)
    assert np.all(np.abs(back - x) <= step / 2 * (1 + 1e-6))
    assert np.all(orc.encode(np.zeros((2, 4, 8)), np.zeros((2, 1, 1)), fmt) == 0)


def test_attention_rows_matches_torch():
    rng = np.random.default_rng(4)
    q, K, V = rng.standard_normal((5, 64)), rng.standard_normal((33, 64)), rng.standard_normal((33, 64))
    o = orc.attention_rows(q, K, V, 0.125)[0]
    ref = torch.nn.functional.scaled_dot_product_attention(*(torch.from_numpy(x)[None] for x in (q, K, V)), scale=0.125)
    np.testing.assert_allclose(o, ref[0].numpy(), rtol=1e-12, atol=1e-13)


def test_page_oracle_counts_match_its_tables():
    rng = random.Random(5)
    for _ in range(40):
        o = orc.PageOracle(30, 6, 9)
        for _ in range(25):
            s = [rng.randrange(6) for _ in range(2)]
            op = rng.randrange(5)
            if op == 0:
                o.reserve(s, [rng.randrange(10) for _ in s])
            elif op == 1:
                o.fork(s[:1], s[1:], [rng.randrange(10)])
            elif op == 2:
                o.own(s, [rng.randrange(5) for _ in s], [rng.randrange(10) for _ in s], 30)
            elif op == 3:
                o.release(s, [rng.randrange(6) for _ in s])
            else:
                o.compact()
                n = sum(r > 0 for r in o.refs)
                assert all(r > 0 for r in o.refs[:n]) and not any(o.refs[n:])
            count = [0] * 30
            for row, h in zip(o.table, o.held):
                assert all(p == -1 for p in row[h:])
                for p in row[:h]:
                    count[p] += 1
            assert count == o.refs


# ------------------------------------------------------------------ refusals (no GPU is reached)
FAKE = ctypes.c_void_p(4096)                # never dereferenced: validation fails first


def _cache(F, **kw):
    c = dict(k=4096, v=4096, k_scale=4096, v_scale=4096, n_mat=1, n_pages=8, Hkv=4, page=64, d=128, format=0)
    c.update(kw)
    return F._CacheStruct(*(c[n] for n in ("k", "v", "k_scale", "v_scale", "n_mat", "n_pages", "Hkv", "page", "d",
                                           "format")))


@pytest.mark.parametrize("bad,status", [
    (dict(k=None), -1), (dict(v_scale=None), -1), (dict(format=2), -1), (dict(n_pages=0), -1), (dict(Hkv=0), -1),
    (dict(n_mat=-1), -1), (dict(k=4104), -1), (dict(k_scale=4098), -1), (dict(n_pages=1 << 30, Hkv=4), -1),
    (dict(d=96), -2), (dict(d=256), -2), (dict(page=48), -2), (dict(page=256), -2)])
def test_bad_caches_are_refused(F, bad, status):
    lib, ref = F.lib, ctypes.byref(_cache(F, **bad))
    before = lib.focus_launch_count()
    assert lib.focus_cache_store(FAKE, FAKE, 1, 64, None, FAKE, 1, ref, None) == status
    assert lib.focus_cache_load(ref, FAKE, 1, FAKE, 1, 0, 64, FAKE, FAKE, None) == status
    assert lib.focus_cache_scatter_rows(FAKE, FAKE, FAKE, FAKE, 1, 8, FAKE, FAKE, 1, ref, None) == status
    assert lib.focus_cache_attention(FAKE, None, ref, FAKE, 1, FAKE, 1, 8, 1, 0.1, FAKE, FAKE, 1 << 30, None) == status
    assert lib.focus_cache_sparse_attention(FAKE, FAKE, ref, FAKE, 1, FAKE, FAKE, 32, FAKE, 4, FAKE, 4, 1, 8, 1, 0.1,
                                            FAKE, FAKE, 1 << 30, None) == status
    assert lib.focus_pages_copy(ref, FAKE, FAKE, 4, None) == status
    assert lib.focus_last_error() and lib.focus_launch_count() == before


def test_bad_arguments_are_refused(F):
    lib, ref = F.lib, ctypes.byref(_cache(F))
    before = lib.focus_launch_count()
    odd = ctypes.c_void_p(4104)
    assert lib.focus_cache_store(None, FAKE, 1, 64, None, FAKE, 1, ref, None) == -1
    assert lib.focus_cache_store(odd, FAKE, 1, 64, None, FAKE, 1, ref, None) == -1
    assert lib.focus_cache_store(FAKE, FAKE, 1, 0, None, FAKE, 1, ref, None) == -1
    assert lib.focus_cache_store(FAKE, FAKE, 1, 64, None, None, 1, ref, None) == -1
    assert lib.focus_cache_store(FAKE, FAKE, 1, 64, None, FAKE, 0, ref, None) == -1
    assert lib.focus_cache_scatter_rows(FAKE, FAKE, FAKE, FAKE, 1, 4097, FAKE, FAKE, 1, ref, None) == -2
    assert lib.focus_cache_scatter_rows(FAKE, FAKE, FAKE, FAKE, 1, 0, FAKE, FAKE, 1, ref, None) == -1
    assert lib.focus_cache_scatter_rows(FAKE, FAKE, FAKE, FAKE, 1, 8, None, FAKE, 1, ref, None) == -1
    assert lib.focus_cache_load(ref, FAKE, 1, FAKE, 1, -1, 64, FAKE, FAKE, None) == -1
    assert lib.focus_cache_load(ref, FAKE, 1, FAKE, 1, 1 << 30, (1 << 30) + 5, FAKE, FAKE, None) == -1

    def dense(Hq=8, qcap=1, cols=1, lens=FAKE, O=FAKE, c=ref):
        return lib.focus_cache_attention(FAKE, None, c, FAKE, cols, lens, 1, Hq, qcap, 0.1, O, FAKE, 1 << 30, None)

    assert dense(Hq=6) == -1 and dense(Hq=0) == -1 and dense(qcap=0) == -1 and dense(lens=None) == -1
    assert dense(O=odd) == -1 and dense(cols=1 << 26) == -1
    assert dense(c=ctypes.byref(_cache(F, n_mat=2))) == -1

    def sparse(G=32, S=4, C=4, sinks=FAKE, P=FAKE):
        return lib.focus_cache_sparse_attention(FAKE, FAKE, ref, FAKE, 1, P, FAKE, G, sinks, S, FAKE, C, 1, 8, 1, 0.1,
                                                FAKE, FAKE, 1 << 30, None)

    assert sparse(G=0) == -1 and sparse(C=0) == -1 and sparse(S=-1) == -1 and sparse(sinks=None) == -1
    assert sparse(P=None) == -1 and sparse(S=1025) == -2 and sparse(C=1025) == -2
    pages = F._PagesStruct(4096, 4096, 4096, 8, 2, 4)
    pref = ctypes.byref(pages)
    assert lib.focus_pages_reserve(pref, FAKE, FAKE, 1025, FAKE, None) == -2
    assert lib.focus_pages_reserve(pref, FAKE, FAKE, -1, FAKE, None) == -1
    assert lib.focus_pages_reserve(pref, FAKE, None, 1, FAKE, None) == -1
    assert lib.focus_pages_reserve(pref, FAKE, FAKE, 1, None, None) == -1
    assert lib.focus_pages_fork(ctypes.byref(F._PagesStruct(4096, None, 4096, 8, 2, 4)), FAKE, FAKE, FAKE, 1, None) == -1
    assert lib.focus_pages_fork(ctypes.byref(F._PagesStruct(4096, 4096, 4096, 8, 1 << 20, 1 << 12)), FAKE, FAKE, FAKE, 1,
                                None) == -1
    assert lib.focus_pages_own(pref, FAKE, FAKE, FAKE, 1, None, 4, FAKE, FAKE, None) == -1
    assert lib.focus_pages_compact(pref, FAKE, 3, FAKE, FAKE, None) == -4
    assert lib.focus_pages_fork(pref, None, None, None, 0, None) == 0      # an empty list does nothing
    assert lib.focus_launch_count() == before


def test_the_binding_refuses_what_does_not_fit(F):
    k = torch.zeros((1, 4, 2, 16, 64), dtype=torch.int8)
    s = torch.zeros((1, 4, 2))
    with pytest.raises(TypeError):
        F.Cache(k.float(), k.float(), s, s)
    with pytest.raises(ValueError):
        F.Cache(k, k, s, s)                        # not on the GPU
    with pytest.raises(ValueError):
        F.Pages(torch.zeros(4, dtype=torch.int32), torch.zeros((2, 2), dtype=torch.int32),
                torch.zeros(2, dtype=torch.int32))


def test_more_heads_than_a_grid_holds_are_refused(F):
    lib, before = F.lib, F.lib.focus_launch_count()
    many = ctypes.byref(_cache(F, n_mat=300))
    assert lib.focus_cache_store(FAKE, FAKE, 219, 64, None, FAKE, 1, many, None) == -2
    assert lib.focus_cache_load(many, FAKE, 1, FAKE, 219, 0, 64, FAKE, FAKE, None) == -2
    assert lib.focus_cache_scatter_rows(FAKE, FAKE, FAKE, FAKE, 55, 8, FAKE, FAKE, 1, many, None) == -2
    wide = ctypes.byref(_cache(F, Hkv=32768))
    assert lib.focus_cache_store(FAKE, FAKE, 1, 64, None, FAKE, 1, wide, None) == -2
    assert lib.focus_cache_load(wide, FAKE, 1, FAKE, 1, 0, 64, FAKE, FAKE, None) == -2
    assert lib.focus_launch_count() == before
