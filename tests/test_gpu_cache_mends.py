"""Calls of the 8-bit cache at the ends of their ranges: scores of any size, keys that each show in
the output, workspaces of other streams, pages that run short over several passes."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as orc
from test_gpu_cache import DEV, F, FMTS, PageWorld, World, check_attention, i32, no_device_error, rand_bf16  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ scores
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("score", [1e3, 1e5, -1e5, 1e6, 1e7, -1e7, 3e8, 1e12, 1e30])
def test_keys_that_take_all_the_weight(F, fmt, score):
    """Three keys of 300, two of them in one tile, share the largest score, and every other lies far
    below: the output is the mean of their values, however large the scores.

    256 heads of 6 rows, each with a size of its own between one and four times `score`. A row's
    elements are alike and the codes powers of two, so both enter in 8 + 8 bits without a rounding and
    the three scores are equal in fp32 as well. Each of their probabilities may be off by 2^-8 of
    itself (2^-14 in int8), the output by half a step, 2^-8."""
    H, page, d, L = 256, 16, 64, 300
    rng = np.random.default_rng(7)
    w = World(F, fmt, 1, 1, H, page, d, -(-L // page), seed=5)
    code = lambda x: orc.nearest_codes(np.float32([x]), fmt)[0]
    best = [17, 100, 290]
    w.codes[0][:] = code(32.0 if score > 0 else 127.0)       # (below, or with a negative sign far above)
    for pos in best:
        w.codes[0][0, w.table[0, pos // page], :, pos % page] = code(64.0)
    w.scales[0][:] = ((1 + rng.random(H)) / 64).astype(np.float32)
    w.scales[1][:] = np.float32(1 / orc.TOP[fmt])
    w.upload(F)
    q = torch.from_numpy((1 + rng.random((1, 2 * H, 3, 1))).astype(np.float32)).to(torch.bfloat16).to(DEV)
    Q = q.expand(-1, -1, -1, d).contiguous()
    O = torch.zeros_like(Q)
    F.focus_cache_attention(Q, None, w.cache, w.t_table, i32([L]), O, scale=score / d)
    for h in range(H):
        V = orc.values(w.codes[1], w.scales[1], w.table[0], best, h, fmt)
        err = np.abs(O[0, 2 * h:2 * h + 2].double().cpu().numpy() - V.mean(axis=0))
        lim = 2.0 ** -8 * (np.abs(V.mean(axis=0)) + np.abs(V).mean(axis=0))
        assert np.all(err <= lim), (h, float((err / lim).max()))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("k,q,v", [(101, -98, 58), (101, -97, -60), (-100, 98, 0), (0, 0, -80)])
def test_keys_queries_and_values_of_extreme_size(F, fmt, k, q, v):
    """Keys about 2^k, queries about 2^q, values about 2^v, of either format, within the header's ranges:
    scores of a few units all the same."""
    w = World(F, fmt, 1, 1, 2, 32, 64, 20, seed=k + 200)
    w.scales[0] = w.scales[0] * np.float32(2.0 ** k)
    w.scales[1] = w.scales[1] * np.float32(2.0 ** v)
    w.upload(F)
    Q = (rand_bf16((1, 4, 5, 64), 3).float() * 2.0 ** q).to(torch.bfloat16)
    O = torch.zeros_like(Q)
    F.focus_cache_attention(Q, None, w.cache, w.t_table, i32([600]), O)
    assert bool(O.any())
    check_attention(w, Q, O, None, lambda b, h: np.arange(600), 1 / 8)


@pytest.mark.parametrize("G", [2 ** 31 - 1, 2 ** 31 - 100, 10 ** 6])
def test_a_current_block_far_behind_the_table_is_flagged(F, G):
    """What lies in the table is attended, however many positions behind it the block names."""
    w = World(F, orc.E4M3, 1, 2, 2, 16, 64, 20, seed=6)
    Q = rand_bf16((2, 4, 3, 64), 6)
    O = torch.zeros_like(Q)
    P, g0 = [100, 0], [130, 0]
    F.focus_cache_sparse_attention(Q, None, w.cache, w.t_table, i32(P), i32(g0), G, None, i32([[[1], [2]]] * 2), O)
    check_attention(w, Q, O, None, lambda b, h: sorted({*(range(16 * (h + 1), 16 * (h + 2)) if P[b] else ()), *range(g0[b], 320)}),
                    1 / np.sqrt(64))


# ------------------------------------------------------------------ streams
@pytest.mark.parametrize("sparse", [False, True])
def test_a_call_on_a_given_stream_takes_its_workspace_there(F, sparse):
    """The side stream is behind, so its call has not started when the current stream fills memory of
    the workspace's size: neither may write into the other's."""
    w = World(F, orc.E4M3, 1, 1, 2, 64, 128, 40, seed=3)
    Q = rand_bf16((1, 4, 16, 128), 4)
    lens, P, blocks = i32([2500]), i32([2400]), i32([[list(range(30)), list(range(5, 35))]])
    side = torch.cuda.Stream()

    def call(O, **kw):
        if sparse:
            F.focus_cache_sparse_attention(Q, None, w.cache, w.t_table, P, P, 64, None, blocks, O, **kw)
        else:
            F.focus_cache_attention(Q, None, w.cache, w.t_table, lens, O, **kw)

    want, O = torch.zeros_like(Q), torch.zeros_like(Q)
    call(want)
    n = F.cache_workspace_bytes(1, 4, 2, 128, 16)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    call(O, stream=side)
    taken = [torch.full((n,), 7, dtype=torch.uint8, device=DEV) for _ in range(8)]
    torch.cuda.synchronize()
    assert all(bool((t == 7).all()) for t in taken) and torch.equal(O, want)


# ------------------------------------------------------------------ rows
def test_store_of_a_short_sequence_in_a_very_long_input(F):
    """Pages that start 2^27 positions and more behind the sequence: none of their rows is read or
    written (rows of 34 GB of memory that nothing has touched)."""
    page, d, L = 64, 128, 2 ** 27 + 69
    w = World(F, orc.INT8, 1, 1, 1, page, d, 2, seed=9)
    X = torch.empty((1, 1, 1, L, d), dtype=torch.bfloat16, device=DEV)
    X[..., :100, :] = rand_bf16((100, d), 3)
    for n in (0, 5, 70):
        F.focus_cache_store(X, X, w.cache, w.t_table, i32([n]))
        for kv in range(2):
            orc.store(X[..., :100, :].float().cpu().numpy(), w.codes[kv], w.scales[kv], w.table, [n], w.fmt)
        w.assert_same()


# ------------------------------------------------------------------ pages
@pytest.mark.parametrize("cap", [0, 1, 100, 1500, 2500, 2799, 2800])
@pytest.mark.parametrize("keeps", [[400] * 7, [400, 399, 7, 1, 0, 400, 350]])
def test_own_says_how_many_are_missing(F, cap, keeps):
    """Eight sequences with up to 400 shared pages, more entries than one pass takes, and room for `cap`
    pairs: the number that is missing, and nothing changed; then, with room, what has to be copied."""
    w = PageWorld(F, 4000, 9, 400)
    w.reserve([0], [400])
    w.fork([0] * 7, list(range(1, 8)), keeps)
    order = [3, 0, 5, 1, 7, 2, 6, 4]
    for seqs, first, last in ((order, [0] * 8, [400] * 8), (order + [0, 7], [3] * 8 + [0, 0], [390] * 8 + [400, 400])):
        short = w.o.own(seqs, first, last, 0)[0]              # (copies that are needed; changes nothing)
        F.focus_pages_own(w.p, i32(seqs), i32(first), i32(last), w.pairs[:cap], w.n_pairs, w.status)
        want, pairs = w.o.own(seqs, first, last, cap)
        assert want == max(0, short - cap)
        assert int(w.status) == want and w.got_pairs() == pairs
        w.same()


def test_own_is_short_of_pages_and_of_pairs(F):
    """Fewer free pages than pairs, and the other way: the smaller room counts."""
    w = PageWorld(F, 700, 5, 300)
    w.reserve([0], [300])
    w.fork([0] * 4, [1, 2, 3, 4], [300] * 4)                  # 1200 copies for 400 free pages
    for cap in (700, 400, 399, 20):
        F.focus_pages_own(w.p, i32([0, 1, 2, 3, 4]), i32([0] * 5), i32([300] * 5), w.pairs[:cap], w.n_pairs, w.status)
        assert int(w.status) == 1200 - min(cap, 400) and int(w.n_pairs) == 0
        w.same()
