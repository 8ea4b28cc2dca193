"""The 8-bit paged cache on the GPU against the float64 oracle: rows, attention, pages, and a
run of them together.

Codes, scales and page accounting must match exactly: both sides follow the same float32
definition. Attention is held to a bound made of its own roundings (see attention_bound).
"""
import random

import numpy as np
import pytest
import torch

from oracle import cache_oracle as orc

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPE = {orc.E4M3: torch.float8_e4m3fn, orc.INT8: torch.int8}
FMTS = [orc.E4M3, orc.INT8]


@pytest.fixture(scope="module")
def F():
    from diffusion_long_context_b200 import build
    build.build()
    from diffusion_long_context_b200 import focus
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    return focus


@pytest.fixture(autouse=True)
def no_device_error(request, F):
    """Every test but those that plant bad pages leaves the device error word clear."""
    F.device_error()
    yield
    err = F.device_error()
    assert (err == 5) if "flagged" in request.node.name else (err == 0)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def rand_bf16(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16).to(DEV)


class World:
    """A cache with random codes everywhere and B sequences on scattered pages, on both sides."""

    def __init__(self, F, fmt, n_mat, B, H, page, d, cols, seed, spare=3, junk=False):
        rng = np.random.default_rng(seed)
        n_pages = B * cols + spare
        self.fmt, self.page, self.d, self.H, self.B = fmt, page, d, H, B
        shape = (n_mat, n_pages, H, page, d)
        x = rng.standard_normal(shape).astype(np.float32)
        unit = np.float32(35 if fmt == orc.INT8 else 120)
        self.codes = [orc.nearest_codes(x * unit, fmt), orc.nearest_codes(rng.permuted(x, axis=-1) * unit, fmt)]
        self.scales = [(np.exp(0.4 * rng.standard_normal(shape[:3])) / unit).astype(np.float32) for _ in range(2)]
        self.table = rng.permutation(n_pages)[:B * cols].reshape(B, cols).astype(np.int32)
        if junk:        # pages that no sequence names, and all codes that no position names, are NaN
            free = sorted(set(range(n_pages)) - set(self.table.ravel().tolist()))
            for c, s in zip(self.codes, self.scales):
                c[:, free], s[:, free] = 0xFF, np.nan
        self.upload(F)

    def upload(self, F):
        self.t_codes = [torch.from_numpy(c).to(DEV).view(DTYPE[self.fmt]) for c in self.codes]
        self.t_scales = [torch.from_numpy(s).to(DEV) for s in self.scales]
        self.t_table = torch.from_numpy(self.table).to(DEV)
        self.cache = F.Cache(*self.t_codes, *self.t_scales)

    def assert_same(self):
        for kv in range(2):
            np.testing.assert_array_equal(self.t_codes[kv].view(torch.uint8).cpu().numpy(), self.codes[kv])
            np.testing.assert_array_equal(self.t_scales[kv].cpu().numpy(), self.scales[kv])


# ------------------------------------------------------------------ store and load
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n_mat,B,H,L,page,d", [(1, 1, 1, 1, 16, 64), (2, 3, 4, 130, 64, 128), (1, 4, 2, 257, 16, 128),
                                                (3, 2, 3, 95, 32, 64), (1, 2, 2, 300, 128, 128),
                                                (1, 5, 2, 128, 128, 64)])
def test_store_then_load(F, fmt, n_mat, B, H, L, page, d):
    cols = -(-L // page)
    w = World(F, fmt, n_mat, B, H, page, d, cols, seed=L + d)
    K, V = rand_bf16((n_mat, B, H, L, d), 1), rand_bf16((n_mat, B, H, L, d), 2, 30.0)
    K[..., L // 2, :] = 0
    K[0, 0, 0] = 0                                          # a head of zeros: scale 0
    V[0, 0, 0, :, 0] = 1e-38                                # quotients far below one step, scales of subnormals
    lens = [L, 0, 1, L - 1, -3][:B]
    F.focus_cache_store(K, V, w.cache, w.t_table, i32(lens))
    for kv, X in enumerate((K, V)):
        orc.store(X.float().cpu().numpy(), w.codes[kv], w.scales[kv], w.table, lens, fmt)
    w.assert_same()
    # back again, from an offset, with rows behind the sequence left as they were
    for start, n in ((0, L), (min(5, L - 1), L + 7)):
        outs = [torch.full((n_mat, B, H, n, d), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        F.focus_cache_load(w.cache, w.t_table, i32(lens), start, *outs)
        for kv in range(2):
            exp = np.full((n_mat, B, H, n, d), 7.0)
            for b in range(B):
                pos = np.arange(start, min(start + n, lens[b]))
                for m in range(n_mat):
                    for h in range(H):
                        if pos.size:
                            exp[m, b, h, :pos.size] = orc.values(w.codes[kv], w.scales[kv], w.table[b], pos, h, fmt, m)
            ref = torch.from_numpy(exp).float().to(torch.bfloat16)
            assert torch.equal(outs[kv].cpu(), ref)


@pytest.mark.parametrize("fmt", FMTS)
def test_store_all_bf16_ratios(F, fmt):
    """Every pair of bf16 mantissas as (element, largest of its page): exact ties between codes included."""
    d, page = 128, 16
    m = (128 + torch.arange(128)).float() / 128               # the 128 mantissas, [1, 2)
    X = torch.zeros((1, 1, 1, 128 * page, d))
    for j in range(128):                                      # page j: largest element m[j], all x m 2^-k
        rows = torch.stack([m * 2.0 ** -(k + 1) for k in range(page)])
        rows[0, 0] = m[j]
        X[0, 0, 0, j * page:(j + 1) * page] = rows
    K = X.to(torch.bfloat16).to(DEV)
    V = (-X).to(torch.bfloat16).to(DEV)
    w = World(F, fmt, 1, 1, 1, page, d, 128, seed=3)
    F.focus_cache_store(K, V, w.cache, w.t_table)
    for kv, Y in enumerate((K, V)):
        orc.store(Y.float().cpu().numpy(), w.codes[kv], w.scales[kv], w.table, [128 * page], fmt)
    w.assert_same()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_page_that_is_not_finite_reads_as_nan(F, fmt, bad):
    w = World(F, fmt, 1, 1, 2, 32, 64, 2, seed=4)
    K, V = rand_bf16((1, 1, 2, 64, 64), 1), rand_bf16((1, 1, 2, 64, 64), 2)
    K[0, 0, 1, 3, 5] = bad
    F.focus_cache_store(K, V, w.cache, w.t_table)
    out = [torch.zeros_like(K) for _ in range(2)]
    F.focus_cache_load(w.cache, w.t_table, i32([64]), 0, *out)
    assert out[0][0, 0, 1, :32].isnan().any() and not out[0][0, 0, 1, :32].isinf().any()
    assert out[0][0, 0, 0].isfinite().all() and out[0][0, 0, 1, 32:].isfinite().all() and out[1].isfinite().all()
    Q, O = rand_bf16((1, 2, 1, 64), 3), torch.zeros((1, 2, 1, 64), dtype=torch.bfloat16, device=DEV)
    F.focus_cache_attention(Q, None, w.cache, w.t_table, i32([64]), O)
    assert O[0, 1].isnan().all() and O[0, 0].isfinite().all()


def test_bad_pages_are_flagged_and_skipped(F):
    w = World(F, orc.E4M3, 1, 2, 1, 16, 64, 2, seed=5)
    before = [c.copy() for c in w.codes]
    w.table[0] = [-1, 10 ** 6]
    w.upload(F)
    K = rand_bf16((1, 2, 1, 40, 64), 1)                       # 40 positions, 32 in the table
    F.focus_cache_store(K, K, w.cache, w.t_table, i32([32, 40]))
    w.codes = before
    for kv in range(2):
        orc.store(K[:, 1:].float().cpu().numpy()[..., :32, :], w.codes[kv], w.scales[kv], w.table[1:], [32], w.fmt)
    w.assert_same()
    out = torch.full((1, 2, 1, 40, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    F.focus_cache_load(w.cache, w.t_table, i32([32, 40]), 0, out, torch.empty_like(out))
    assert (out[0, 0, 0, :32] == 0).all() and (out[0, 0, 0, 32:] == 7).all()
    assert (out[0, 1, 0, 32:] == 0).all() and (out[0, 1, 0, :32] != 0).any()
    # attention leaves those positions out
    Q = rand_bf16((2, 1, 3, 64), 2)
    O, O2 = torch.full_like(Q, 9.0), torch.full_like(Q, 9.0)
    F.focus_cache_attention(Q, None, w.cache, w.t_table, i32([32, 40]), O)
    F.focus_cache_attention(Q, None, w.cache, w.t_table, i32([0, 32]), O2)
    assert (O[0] == 0).all() and torch.equal(O[1], O2[1])
    rows = i32([[3, -1, 900], [31, 32, 5]])
    F.focus_cache_scatter_rows(K[..., :3, :].contiguous(), K[..., :3, :].contiguous(), rows, i32([3, 3]), w.cache,
                               w.t_table, i32([32, 32]))
    for kv in range(2):
        orc.scatter_rows(K[:, 1:, :, :3].float().cpu().numpy(), np.array([[31, 32, 5]]), [3], w.codes[kv], w.scales[kv],
                         w.table[1:], [32], w.fmt)
    w.assert_same()


# ------------------------------------------------------------------ scatter_rows
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n_mat,B,H,page,d,cols,cap,kind", [
    (1, 1, 1, 16, 64, 1, 1, "sorted"), (2, 3, 2, 64, 128, 5, 32, "sorted"), (1, 2, 2, 16, 128, 40, 300, "sorted"),
    (1, 3, 2, 32, 64, 6, 50, "any"), (1, 2, 1, 128, 128, 3, 40, "any"), (1, 2, 1, 16, 64, 30, 600, "repeat")])
def test_scatter_rows(F, fmt, n_mat, B, H, page, d, cols, cap, kind):
    rng = np.random.default_rng(cap + d)
    w = World(F, fmt, n_mat, B, H, page, d, cols, seed=cap)
    top = cols * page
    rows = np.full((B, cap), -9, dtype=np.int32)
    n_rows, lens = [], []
    for b in range(B):
        n = int(rng.integers(max(1, min(cap, top) // 2), min(cap, top) + 1)) if b != 1 else min(cap, top)
        r = rng.choice(top, n, replace=kind == "repeat")
        rows[b, :n] = np.sort(r) if kind == "sorted" else r
        n_rows.append(n)
        lens.append([top, top // 2 + 3, 0][b % 3])
    n_rows[-1] = 0 if B > 2 else n_rows[-1]
    K = rand_bf16((n_mat, B, H, cap, d), 1) * torch.logspace(-2, 1, cap).to(DEV).to(torch.bfloat16)[:, None]
    V = rand_bf16((n_mat, B, H, cap, d), 2, 0.3)
    F.focus_cache_scatter_rows(K, V, torch.from_numpy(rows).to(DEV), i32(n_rows), w.cache, w.t_table, i32(lens))
    for kv, X in enumerate((K, V)):
        orc.scatter_rows(X.float().cpu().numpy(), rows, n_rows, w.codes[kv], w.scales[kv], w.table, lens, fmt)
    w.assert_same()


# ------------------------------------------------------------------ attention
def attention_bound(o, mean_abs_v, floor_v, spread):
    """How far a correct kernel may be from the float64 result o of a row.

    Output in bf16: half a step, 2^-8 |o|. Probabilities enter the product in 8 + 8 bits: an
    e4m3 pair keeps 2^-8 of its value, an int8 pair 2^-15 of the largest in its tile, so
    2^-8 of the mean |v| under p and 2^-15 of sum |v| relative to the largest p. Queries enter
    in 8 + 8 bits too, within 2^-14 of the row's largest: a score is off by
    2^-14 scale max|q| sum|k| = 2^-14 spread, and by as much again at most for 128 products
    summed in fp32 (128 * 2^-24 < 2^-14) and for its scaling; an error e in all scores moves
    the output by at most 2 e of the mean |v|.
    """
    return 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2 * 2 * 2.0 ** -14 * spread) * mean_abs_v + 2.0 ** -15 * floor_v + 1e-30


def check_attention(w, Q, O, n_q, keys_of, scale):
    g = Q.shape[1] // w.H
    q, got = Q.double().cpu().numpy(), O.double().cpu().numpy()
    worst = 0.0
    for b in range(Q.shape[0]):
        n = Q.shape[2] if n_q is None else max(0, min(n_q[b], Q.shape[2]))
        assert np.all(got[b, :, n:] == 0), "rows behind n_q must be zero"
        for h in range(w.H):
            keys = np.asarray(keys_of(b, h), dtype=np.int64)
            K, V = (orc.values(w.codes[kv], w.scales[kv], w.table[b], keys, h, w.fmt) for kv in range(2))
            for x in range(g):
                o, *parts = orc.attention_rows(q[b, h * g + x, :n], K, V, scale)
                err, lim = np.abs(got[b, h * g + x, :n] - o), attention_bound(o, *parts)
                assert np.all(err <= lim), (b, h, x, float((err / lim).max()))
                worst = max(worst, float((err / lim).max(initial=0)))
    return worst


LENS = [1, 15, 16, 17, 127, 128, 129, 255, 300, 700, 0, 513]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("Hq,H,page,d,qcap", [(2, 2, 64, 128, 32), (7, 1, 64, 128, 1), (14, 2, 32, 128, 32),
                                              (2, 1, 16, 128, 5), (4, 4, 128, 128, 16), (2, 2, 64, 64, 32),
                                              (8, 1, 16, 64, 1), (6, 2, 128, 64, 33), (3, 3, 32, 64, 17)])
def test_dense_attention(F, fmt, Hq, H, page, d, qcap):
    B = len(LENS)
    w = World(F, fmt, 1, B, H, page, d, -(-max(LENS) // page), seed=Hq * page + d, junk=True)
    Q = rand_bf16((B, Hq, qcap, d), 11)
    O = torch.full_like(Q, 5.0)
    n_q = None if qcap == 1 else [qcap, 1, 0, qcap // 2, *[qcap] * (B - 5), qcap + 3]
    F.focus_cache_attention(Q, None if n_q is None else i32(n_q), w.cache, w.t_table, i32(LENS), O)
    check_attention(w, Q, O, n_q, lambda b, h: np.arange(LENS[b]), 1 / np.sqrt(d))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("scale", [0.0, 0.3, -0.1, 3.0])
def test_dense_attention_scales_and_peaks(F, fmt, scale):
    """Sharp and flat rows, a few keys of great norm, rows of unlike norm in one tile."""
    w = World(F, fmt, 1, 1, 2, 64, 128, 12, seed=21)
    w.scales[0][0, w.table[0, 3]] *= 6
    w.scales[1][0, w.table[0, 5]] *= 1e4                     # values of unlike size
    w.scales[1][0, w.table[0, 6]] *= 1e-6
    w.scales[0][0, w.table[0, 7]] = 0                        # a page of zero keys, one of zero values
    w.scales[1][0, w.table[0, 8]] = 0
    w.upload(F)
    Q = rand_bf16((1, 4, 9, 128), 3) * torch.logspace(-3, 0.5, 9).to(DEV).to(torch.bfloat16)[:, None]
    Q[0, 0, 2] = 0
    O = torch.zeros_like(Q)
    F.focus_cache_attention(Q, None, w.cache, w.t_table, i32([701]), O, scale=scale)
    check_attention(w, Q, O, None, lambda b, h: np.arange(701), float(np.float32(scale)))


@pytest.mark.parametrize("fmt", FMTS)
def test_codes_behind_the_end_are_never_used(F, fmt):
    """The rest of the last page holds NaN codes; its scale is the page's own."""
    w = World(F, fmt, 1, 3, 2, 64, 128, 3, seed=22)
    lens = [70, 1, 129]
    for b, n in enumerate(lens):
        for c in w.codes:
            for pos in range(n, 192):
                c[0, w.table[b, pos // 64], :, pos % 64] = 0xFF
    w.upload(F)
    Q = rand_bf16((3, 2, 4, 128), 3)
    O = torch.zeros_like(Q)
    F.focus_cache_attention(Q, None, w.cache, w.t_table, i32(lens), O)
    check_attention(w, Q, O, None, lambda b, h: np.arange(lens[b]), 1 / np.sqrt(128))


def test_a_query_that_is_not_finite_gives_nan_in_its_row_alone(F):
    for fmt in FMTS:
        w = World(F, fmt, 1, 1, 1, 64, 128, 4, seed=23)
        for bad in (float("nan"), float("inf")):
            Q = rand_bf16((1, 1, 6, 128), 3)
            Q[0, 0, 2, 7] = bad
            O = torch.zeros_like(Q)
            F.focus_cache_attention(Q, None, w.cache, w.t_table, i32([200]), O)
            assert O[0, 0, 2].isnan().all()
            ok = [0, 1, 3, 4, 5]
            Q2, O2 = Q[:, :, ok].contiguous(), torch.zeros((1, 1, 5, 128), dtype=torch.bfloat16, device=DEV)
            F.focus_cache_attention(Q2, None, w.cache, w.t_table, i32([200]), O2)
            assert torch.equal(O[:, :, ok], O2)


@pytest.mark.parametrize("fmt", FMTS)
def test_long_ragged_batch(F, fmt):
    """Split over many CTAs: lengths from nothing to 9001, one token each, grouped heads."""
    lens = [9001, 0, 3, 2500, 128, 4097]
    w = World(F, fmt, 1, len(lens), 2, 32, 128, 282, seed=24, spare=0)
    Q = rand_bf16((len(lens), 8, 1, 128), 4)
    O = torch.full_like(Q, 3.0)
    F.focus_cache_attention(Q, None, w.cache, w.t_table, i32(lens), O)
    check_attention(w, Q, O, None, lambda b, h: np.arange(lens[b]), 1 / np.sqrt(128))


def test_offsets_beyond_32_bits(F):
    """A pool of more than 2^32 bytes of codes: the last pages are stored, attended and loaded."""
    n_pages, H, page, d = 18000, 32, 64, 128
    shape = (1, n_pages, H, page, d)
    k, v = (torch.empty(shape, dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2))
    ks, vs = (torch.empty(shape[:3], device=DEV) for _ in range(2))
    cache = F.Cache(k, v, ks, vs)
    table = i32([[n_pages - 1, 5, n_pages - 3]])
    K, V = rand_bf16((1, 1, H, 150, d), 1), rand_bf16((1, 1, H, 150, d), 2)
    F.focus_cache_store(K, V, cache, table)
    out = [torch.zeros_like(K) for _ in range(2)]
    F.focus_cache_load(cache, table, i32([150]), 0, *out)
    # one code is within 1/16 of its value (or half the smallest step of its page)
    assert ((out[0] - K).abs() <= K.abs() / 16 + 2e-5 * K.abs().max()).all()
    pairs = i32([[n_pages - 1, 7], [5, n_pages - 2]])
    F.focus_pages_copy(cache, pairs, i32([2]))
    assert torch.equal(k[0, 7].view(torch.uint8), k[0, n_pages - 1].view(torch.uint8))
    assert torch.equal(v[0, n_pages - 2].view(torch.uint8), v[0, 5].view(torch.uint8))
    Q = rand_bf16((1, H, 3, d), 3)
    O = torch.zeros_like(Q)
    F.focus_cache_attention(Q, None, cache, table, i32([150]), O)
    ref = torch.nn.functional.scaled_dot_product_attention(Q.float(), out[0][0].float(), out[1][0].float())
    # against the values rounded to bf16 once more (2^-8 of each key and value): a few 2^-8 of O(1) values
    assert (O.float() - ref).abs().max() < 0.1 and (O.float() - ref).norm() / ref.norm() < 2e-2


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("Hq,H,page,d,qcap,G,C,S", [(2, 2, 64, 128, 32, 32, 4, 8), (14, 2, 32, 128, 9, 32, 6, 5),
                                                    (2, 1, 16, 128, 3, 20, 9, 0), (4, 2, 128, 64, 16, 130, 2, 33),
                                                    (2, 2, 64, 64, 1, 1, 1, 1), (3, 1, 16, 64, 40, 100, 40, 140)])
def test_sparse_attention(F, fmt, Hq, H, page, d, qcap, G, C, S):
    rng = np.random.default_rng(G * C + page)
    B, L = 4, 900
    cols = -(-L // page)
    w = World(F, fmt, 1, B, H, page, d, cols, seed=G + C, junk=True)
    P = [700, 641, 0, 333][:B]
    g0 = [700, 650, 17, min(333 + 5, L - G)]
    nb = [-(-p // page) for p in P]
    blocks = np.full((B, H, C), -1, dtype=np.int32)
    sinks = np.full((B, H, max(S, 1)), -1, dtype=np.int32)
    for b in range(B):
        for h in range(H):
            n = min(C, nb[b])
            blocks[b, h, :n] = np.sort(rng.choice(max(nb[b], 1), n, replace=False))
            if n and b == 1:
                blocks[b, h, n - 1] = nb[b] - 1               # the last block, cut at P, reaching into the current one
            n = min(S, L)
            sinks[b, h, :n] = np.sort(rng.choice(L, n, replace=False))
    Q = rand_bf16((B, Hq, qcap, d), 5)
    O = torch.full_like(Q, 5.0)
    n_q = [qcap, max(1, qcap // 2), qcap, 1]
    F.focus_cache_sparse_attention(Q, i32(n_q), w.cache, w.t_table, i32(P), i32(g0), G,
                                   torch.from_numpy(sinks).to(DEV) if S else None, torch.from_numpy(blocks).to(DEV), O)
    check_attention(w, Q, O, n_q, lambda b, h: orc.key_set(P[b], g0[b], G, sinks[b, h] if S else [], blocks[b, h], page),
                    1 / np.sqrt(d))


@pytest.mark.parametrize("fmt", FMTS)
def test_sparse_attention_counts_a_key_once(F, fmt):
    """Unsorted and repeated blocks and sinks, sinks inside kept blocks and the current block, blocks behind P."""
    w = World(F, fmt, 1, 1, 1, 16, 128, 20, seed=31)
    P, g0, G = 150, 152, 20
    blocks = [9, 3, 3, -1, 0, 9, 12, 19]
    sinks = [151, 48, 48, 5, 155, 300, -1, 149, 151, 160, 200]
    Q = rand_bf16((1, 2, 4, 128), 6)
    O = torch.zeros_like(Q)
    F.focus_cache_sparse_attention(Q, i32([4]), w.cache, w.t_table, i32([P]), i32([g0]), G, i32([[sinks]]),
                                   i32([[blocks]]), O)
    check_attention(w, Q, O, [4], lambda b, h: orc.key_set(P, g0, G, sinks, blocks, 16), 1 / np.sqrt(128))


def test_sparse_attention_of_many_sinks_and_blocks(F):
    w = World(F, orc.E4M3, 1, 1, 1, 16, 128, 1100, seed=32, spare=0)
    rng = np.random.default_rng(8)
    P, g0, G = 17000, 17000, 64
    blocks = np.sort(rng.choice(1062, 1024, replace=False)).astype(np.int32)
    sinks = np.sort(rng.choice(17064, 1024, replace=False)).astype(np.int32)
    Q = rand_bf16((1, 1, 2, 128), 6)
    O = torch.zeros_like(Q)
    F.focus_cache_sparse_attention(Q, i32([2]), w.cache, w.t_table, i32([P]), i32([g0]), G, i32([[sinks.tolist()]]),
                                   i32([[blocks.tolist()]]), O)
    check_attention(w, Q, O, [2], lambda b, h: orc.key_set(P, g0, G, sinks, blocks, 16), 1 / np.sqrt(128))


def test_sparse_attention_of_bad_positions_is_flagged(F):
    """A current block that reaches behind the table, or starts before 0: those positions are left out."""
    w = World(F, orc.INT8, 1, 2, 1, 16, 64, 4, seed=33)
    Q = rand_bf16((2, 1, 3, 64), 6)
    O = torch.zeros_like(Q)
    F.focus_cache_sparse_attention(Q, None, w.cache, w.t_table, i32([30, 0]), i32([50, -5]), 20,
                                   i32([[[900]], [[2 ** 31 - 1]]]), i32([[[1]], [[2 ** 31 - 1]]]), O)
    keys = [list(range(16, 30)) + list(range(50, 64)), list(range(0, 15))]
    check_attention(w, Q, O, None, lambda b, h: keys[b], 1 / np.sqrt(64))


def test_queries_of_no_sequence(F):
    w = World(F, orc.E4M3, 1, 1, 1, 16, 64, 2, seed=34)
    none = torch.empty((0, 1, 3, 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises((F.FocusError, ValueError)):
        F.focus_cache_attention(none, None, w.cache, w.t_table, i32([5]), none.clone())


def test_refused_on_another_shape_or_workspace(F):
    w = World(F, orc.E4M3, 1, 2, 2, 16, 64, 2, seed=35)
    Q = rand_bf16((2, 4, 3, 64), 6)
    with pytest.raises(ValueError):
        F.focus_cache_attention(Q, None, w.cache, w.t_table, i32([5]), torch.empty_like(Q))
    with pytest.raises(ValueError):
        F.focus_cache_attention(Q, i32([1]), w.cache, w.t_table, i32([5, 5]), torch.empty_like(Q))
    with pytest.raises(ValueError):
        F.focus_cache_attention(rand_bf16((2, 4, 3, 128), 6), None, w.cache, w.t_table, i32([5, 5]), torch.empty_like(Q))
    with pytest.raises(F.FocusError):
        F.focus_cache_attention(rand_bf16((2, 3, 3, 64), 6), None, w.cache, w.t_table, i32([5, 5]), rand_bf16((2, 3, 3, 64), 6))
    with pytest.raises(ValueError):
        F.focus_cache_attention(Q.transpose(1, 2), None, w.cache, w.t_table, i32([5, 5]), torch.empty_like(Q))
    with pytest.raises(ValueError):
        F.focus_cache_attention(Q, None, w.cache, w.t_table[:1], i32([5, 5]), torch.empty_like(Q))
    need = F.cache_workspace_bytes(2, 4, 2, 64, 3)
    if need:
        with pytest.raises(ValueError):
            F.focus_cache_attention(Q, None, w.cache, w.t_table, i32([5, 5]), torch.empty_like(Q),
                                    ws=torch.empty(need - 1, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        F.focus_cache_store(rand_bf16((1, 2, 3, 5, 64), 1), rand_bf16((1, 2, 3, 5, 64), 1), w.cache, w.t_table)


# ------------------------------------------------------------------ pages
class PageWorld:
    def __init__(self, F, n_pages, n_seq, cols):
        self.F, self.o, self.n_pages = F, orc.PageOracle(n_pages, n_seq, cols), n_pages
        self.refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
        self.table = torch.full((n_seq, cols), -1, dtype=torch.int32, device=DEV)
        self.held = torch.zeros(n_seq, dtype=torch.int32, device=DEV)
        self.p = F.Pages(self.refs, self.table, self.held)
        self.status, self.n_pairs = i32([-7]), i32([-7])
        self.pairs = torch.zeros((n_pages, 2), dtype=torch.int32, device=DEV)
        self.remap = torch.zeros(n_pages, dtype=torch.int32, device=DEV)

    def same(self):
        assert self.refs.tolist() == self.o.refs
        assert self.held.tolist() == self.o.held
        assert self.table.tolist() == self.o.table

    def got_pairs(self):
        return [tuple(p) for p in self.pairs[:int(self.n_pairs)].tolist()]

    def reserve(self, seqs, want):
        self.F.focus_pages_reserve(self.p, i32(seqs), i32(want), self.status)
        assert int(self.status) == self.o.reserve(seqs, want)
        self.same()

    def fork(self, src, dst, keep):
        self.F.focus_pages_fork(self.p, i32(src), i32(dst), i32(keep))
        self.o.fork(src, dst, keep)
        self.same()

    def own(self, seqs, first, last, cap=None):
        pairs = self.pairs if cap is None else self.pairs[:cap]
        self.F.focus_pages_own(self.p, i32(seqs), i32(first), i32(last), pairs, self.n_pairs, self.status)
        st, exp = self.o.own(seqs, first, last, pairs.shape[0])
        if cap is None:
            assert int(self.status) == st
        else:
            assert (int(self.status) > 0) == (st > 0)
        assert self.got_pairs() == exp
        self.same()

    def release(self, seqs, keep):
        self.F.focus_pages_release(self.p, i32(seqs), i32(keep))
        self.o.release(seqs, keep)
        self.same()

    def compact(self):
        self.F.focus_pages_compact(self.p, self.pairs, self.n_pairs, self.remap)
        exp, remap = self.o.compact()
        assert self.got_pairs() == exp and self.remap.tolist() == remap
        self.same()


@pytest.mark.parametrize("n_pages,n_seq,cols,seed", [(1, 1, 1, 0), (40, 6, 9, 1), (200, 12, 40, 2), (5000, 20, 600, 3),
                                                     (9000, 40, 300, 4)])
def test_random_page_operations(F, n_pages, n_seq, cols, seed):
    rng = random.Random(seed)
    w = PageWorld(F, n_pages, n_seq, cols)
    for _ in range(60):
        n = rng.randint(1, min(n_seq, 6))
        s = [rng.randrange(n_seq) for _ in range(n)]           # the same sequence twice included
        op = rng.randrange(6)
        if op <= 1:
            w.reserve(s, [rng.randint(0, cols) for _ in s])
        elif op == 2:
            # targets that hold nothing, chains included
            empty = [x for x in range(n_seq) if w.o.held[x] == 0]
            rng.shuffle(empty)
            dst = empty[:n]
            src = [rng.choice([x for x in range(n_seq) if x != t and (w.o.held[x] or x in dst[:i])] or [t])
                   for i, t in enumerate(dst)]
            use = [(a, b) for a, b in zip(src, dst) if a != b]
            if use:
                w.fork([a for a, _ in use], [b for _, b in use], [rng.randint(0, cols) for _ in use])
        elif op == 3:
            w.own(s, [rng.randint(0, cols) for _ in s], [rng.randint(0, cols + 2) for _ in s])
        elif op == 4:
            w.release(s, [rng.choice([0, rng.randint(0, cols)]) for _ in s])
        else:
            w.compact()


def test_short_of_pages_changes_nothing(F):
    w = PageWorld(F, 10, 4, 10)
    w.reserve([0, 1], [4, 3])
    w.reserve([2, 3], [2, 2])                                  # 3 free, 4 wanted
    assert int(w.status) == 1
    w.fork([0, 0], [2, 3], [4, 4])
    w.own([2, 3], [0, 0], [4, 4])                              # 8 copies, 3 free
    assert int(w.status) == 5 and int(w.n_pairs) == 0
    w.own([2, 3], [1, 2], [3, 3], cap=2)                       # 3 copies, room for 2 pairs
    w.own([2, 3, 2], [1, 2, 0], [3, 3, 2])                     # 4 copies, 3 free
    w.own([2, 3, 2], [1, 2, 1], [3, 3, 2])                     # 3: the repeated entry counts once
    w.reserve([1], [3])
    assert int(w.status) == 0


def test_many_shared_entries(F):
    """More entries than one pass over them takes, every page shared by all of its sequences."""
    w = PageWorld(F, 4000, 9, 400)
    w.reserve([0], [400])
    w.fork([0] * 7, list(range(1, 8)), [400, 399, 400, 1, 0, 400, 400])
    w.own(list(range(8)), [0] * 8, [400] * 8)
    w.release([3, 0], [0, 2])
    w.compact()


def test_bad_lists_are_flagged(F):
    w = PageWorld(F, 20, 4, 5)
    w.reserve([0, 9, -1, 1, 2], [2, 3, 3, 6, 1])               # no sequence 9 or -1, want 6 above 5 columns
    w.fork([0, 0, 7, 0], [3, 2, 1, 0], [2, 2, 2, 2])           # 2 holds a page, 7 is no sequence, 0 into itself
    w.own([5, 3], [0, 0], [9, 9])
    w.release([-4, 3, 44], [0, 0, 0])


def test_copy_of_pages(F):
    for fmt, page, d, H, n_mat in ((orc.E4M3, 64, 128, 3, 2), (orc.INT8, 16, 64, 1, 3), (orc.INT8, 128, 128, 2, 1)):
        w = World(F, fmt, n_mat, 1, H, page, d, 6, seed=41)
        w.F = F
        n = w.codes[0].shape[1]
        src, dst = [0, 2, 2, 5], [1, 3, 4, 6]
        pairs = i32(list(map(list, zip(src, dst))) + [[0, 7], [0, 8]])
        for count, use in ((4, 4), (0, 0), (-1, 0)):
            F.focus_pages_copy(w.cache, pairs, i32([count]))
            for arr in (*w.codes, *w.scales):
                arr[:, dst[:use]] = arr[:, src[:use]]
            w.assert_same()
        F.focus_pages_copy(w.cache, pairs[:3].contiguous(), i32([50]))       # no more than there are
        w.assert_same()
        assert n == 9


def test_copy_of_bad_pairs_is_flagged(F):
    w = World(F, orc.INT8, 2, 1, 2, 16, 64, 4, seed=42)
    F.focus_pages_copy(w.cache, i32([[0, 99], [-1, 2], [7, 1], [3, 2]]), i32([4]))
    for arr in (*w.codes, *w.scales):
        arr[:, 2] = arr[:, 3]
    w.assert_same()


# ------------------------------------------------------------------ streams, graphs, all together
@pytest.mark.parametrize("fmt", FMTS)
def test_on_another_stream_and_in_a_graph(F, fmt):
    w = World(F, fmt, 1, 2, 2, 32, 128, 8, seed=51)
    Q, lens = rand_bf16((2, 4, 5, 128), 1), i32([250, 100])
    blocks, sinks = i32([[[0, 3], [1, -1]]] * 2), i32([[[5, 70], [90, 99]]] * 2)
    P, g0 = i32([200, 60]), i32([200, 64])
    ws = torch.empty(max(256, F.cache_workspace_bytes(2, 4, 2, 128, 5)), dtype=torch.uint8, device=DEV)
    out = [torch.zeros_like(Q) for _ in range(2)]

    def both(o):
        F.focus_cache_attention(Q, None, w.cache, w.t_table, lens, o[0], ws=ws)
        F.focus_cache_sparse_attention(Q, None, w.cache, w.t_table, P, g0, 30, sinks, blocks, o[1], ws=ws)

    both(out)
    side, o2 = torch.cuda.Stream(), [torch.zeros_like(Q) for _ in range(2)]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(o2)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, o2))
    graphs, outs = [], []
    for _ in range(2):                                           # two graphs that share the workspace
        o, g = [torch.zeros_like(Q) for _ in range(2)], torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            both(o)
        graphs.append(g)
        outs.append(o)
    lens.copy_(i32([33, 256]))                                   # read when the graph runs, not when it is made
    for g in graphs + graphs[::-1]:
        g.replay()
    both(out)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for a, b in zip(out, o))


def test_two_calls_at_once_with_a_workspace_each(F):
    w = World(F, orc.E4M3, 1, 3, 4, 64, 128, 40, seed=52)
    Q, lens = rand_bf16((3, 8, 32, 128), 1), i32([2500, 1300, 2000])
    n = max(256, F.cache_workspace_bytes(3, 8, 4, 128, 32))
    ref = torch.zeros_like(Q)
    F.focus_cache_attention(Q, None, w.cache, w.t_table, lens, ref)
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs, wss = [torch.zeros_like(Q) for _ in streams], [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, o, ws in zip(streams, outs, wss):
            with torch.cuda.stream(s):
                F.focus_cache_attention(Q, None, w.cache, w.t_table, lens, o, ws=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(ref, o) for o in outs)


@pytest.mark.parametrize("fmt", FMTS)
def test_a_served_sequence_and_its_branches(F, fmt):
    """Reserve, store, attend, fork, own, copy, write the branch, attend both, compact, attend again, release."""
    n_mat, H, page, d, n_pages, cols, L = 2, 2, 32, 128, 64, 12, 301
    w = World(F, fmt, n_mat, 1, H, page, d, n_pages, seed=61, spare=0)
    pw = PageWorld(F, n_pages, 5, cols)
    K, V = rand_bf16((n_mat, 1, H, L, d), 1), rand_bf16((n_mat, 1, H, L, d), 2)
    need = -(-L // page)
    pw.reserve([4, 0], [7, need])                              # sequence 4 takes the front of the pool
    F.focus_cache_store(K, V, w.cache, pw.table[:1], i32([L]))
    for kv, X in enumerate((K, V)):
        orc.store(X.float().cpu().numpy(), w.codes[kv], w.scales[kv], pw.table[:1].cpu().numpy(), [L], fmt)
    w.assert_same()
    Q = rand_bf16((1, 4, 3, d), 3)

    def attend(seq, layer):
        O = torch.zeros_like(Q)
        F.focus_cache_attention(Q, None, w.cache.layer(layer), pw.table[seq:seq + 1], i32([L]), O)
        view = World.__new__(World)
        view.codes, view.scales = [c[layer:layer + 1] for c in w.codes], [s[layer:layer + 1] for s in w.scales]
        view.table, view.fmt, view.H = pw.table[seq:seq + 1].cpu().numpy(), fmt, H
        check_attention(view, Q, O, None, lambda b, h: np.arange(L), 1 / np.sqrt(d))
        return O

    base = [attend(0, m) for m in range(n_mat)]
    pw.fork([0, 0], [1, 2], [need, need])
    assert all(torch.equal(attend(2, m), base[m]) for m in range(n_mat))
    pw.own([1], [(L - 20) // page], [need])                    # the pages that the branch will write
    F.focus_pages_copy(w.cache, pw.pairs, pw.n_pairs)
    for a, b in pw.got_pairs():
        for arr in (*w.codes, *w.scales):
            arr[:, b] = arr[:, a]
    w.assert_same()
    assert all(torch.equal(attend(1, m), base[m]) for m in range(n_mat))
    rows = np.arange(L - 20, L - 2, dtype=np.int32)[None]
    X = rand_bf16((n_mat, 1, H, rows.shape[1], d), 5, 2.0)
    F.focus_cache_scatter_rows(X, X, torch.from_numpy(rows).to(DEV), i32([rows.shape[1]]), w.cache, pw.table[1:2], i32([L]))
    for kv in range(2):
        orc.scatter_rows(X.float().cpu().numpy(), rows, [rows.shape[1]], w.codes[kv], w.scales[kv],
                         pw.table[1:2].cpu().numpy(), [L], fmt)
    w.assert_same()
    branch = [attend(1, m) for m in range(n_mat)]
    assert all(torch.equal(attend(0, m), base[m]) and not torch.equal(branch[m], base[m]) for m in range(n_mat))
    pw.release([4, 2], [0, 0])
    pw.compact()
    F.focus_pages_copy(w.cache, pw.pairs, pw.n_pairs)
    for a, b in pw.got_pairs():
        for arr in (*w.codes, *w.scales):
            arr[:, b] = arr[:, a]
    w.assert_same()
    assert pw.got_pairs()
    assert all(torch.equal(attend(0, m), base[m]) and torch.equal(attend(1, m), branch[m]) for m in range(n_mat))
    pw.release([0, 1], [0, 0])
    assert not pw.refs.any()
