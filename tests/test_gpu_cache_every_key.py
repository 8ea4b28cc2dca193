"""Attention from the 8-bit cache where every key shows in the output: none is lost, none counts twice.

All scores are 0, so each of n keys has the weight 1 / n. Value rows are one-hot: in head h the key at
place 128 h + i of the sequence has its largest code in dim i and zeros elsewhere, and enough heads
give every key of the sequence an element of the output of its own. That is 1 / n if the key belongs
to the set, and 0 if not. The probabilities are powers of two and exact, sums of ones too; 1 / n and
the quotient are fp32, the output is rounded by half a step: an error of 2^-8 (1 / n) and a little,
where a lost or repeated key would be off by all of it."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as orc
from test_gpu_cache import DEV, DTYPE, F, FMTS, check_attention, i32, no_device_error, rand_bf16, World  # noqa: F401

pytestmark = pytest.mark.gpu


class OneHot:
    """H heads of cols pages, physical pages in reverse; masked rows, too, have their element."""

    def __init__(self, F, fmt, page, d, cols, B=1):
        L = cols * page
        self.H, self.d, self.L, self.B = -(-L // d), d, L, B
        k = torch.zeros((1, cols, self.H, page, d), dtype=torch.uint8, device=DEV)
        v = torch.zeros_like(k)
        pos = torch.arange(L, device=DEV)
        top = int(orc.nearest_codes(np.float32([orc.TOP[fmt]]), fmt)[0])
        v[0, cols - 1 - pos // page, pos // d, pos % page, pos % d] = top
        ks = torch.ones((1, cols, self.H), device=DEV)
        self.cache = F.Cache(k.view(DTYPE[fmt]), v.view(DTYPE[fmt]), ks, ks / float(orc.TOP[fmt]))
        self.table = torch.arange(cols - 1, -1, -1, dtype=torch.int32, device=DEV).repeat(B, 1)

    def check(self, O, keys_of, n_q=None):
        """O [B, g H, qcap, d] against the key sets (in every head the same)."""
        B, Hq, qcap, d = O.shape
        got = O.double().reshape(B, self.H, Hq // self.H, qcap, d)
        for b in range(B):
            keys = torch.as_tensor(sorted(keys_of(b)), dtype=torch.long, device=DEV)
            want = torch.zeros(self.H * d, dtype=torch.float64, device=DEV)
            if keys.numel():
                want[keys] = 1.0 / keys.numel()
            nq = qcap if n_q is None else n_q[b]
            want = want.view(self.H, 1, 1, d).expand(-1, Hq // self.H, nq, -1)
            err = (got[b, :, :, :nq] - want).abs()
            assert bool((err <= 1.01 * 2.0 ** -8 * want).all()), [int(x) for x in (err > 1.01 * 2.0 ** -8 * want).nonzero()[0]]
            assert not got[b, :, :, nq:].any()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("page,d,g,qcap,lens", [
    (64, 128, 1, 32, [4097, 1, 4096, 127, 0, 129, 2500]), (16, 128, 7, 1, [9001, 16, 128, 8999]),
    (32, 64, 2, 5, [700, 513, 3]), (128, 64, 1, 16, [5000, 4992]), (16, 128, 4, 150, [1025, 300]),
    (64, 64, 3, 41, [640, 1, 639]), (128, 128, 1, 300, [1300])])
def test_dense(F, fmt, page, d, g, qcap, lens):
    B = len(lens)
    w = OneHot(F, fmt, page, d, -(-max(lens) // page), B)
    Q = rand_bf16((B, g * w.H, qcap, d), 3)
    O = torch.full_like(Q, 5.0)
    n_q = [max(0, qcap - 3 * b) for b in range(B)]
    F.focus_cache_attention(Q, i32(n_q), w.cache, w.table, i32(lens), O)
    w.check(O, lambda b: range(lens[b]), n_q)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("order", ["ascending", "any", "repeated"])
@pytest.mark.parametrize("page,d,L,P,g0,G,C,S", [
    (16, 128, 17600, 17000, 17000, 64, 1024, 1024),      # the longest lists
    (16, 128, 17600, 17000, 17005, 129, 1000, 0),
    (64, 128, 8192, 8000, 8000, 32, 64, 33), (128, 64, 2048, 1900, 1900, 100, 9, 1000),
    (32, 64, 1000, 641, 700, 250, 7, 140), (16, 64, 400, 399, 399, 1, 1, 1)])
def test_sparse(F, fmt, order, page, d, L, P, g0, G, C, S):
    rng = np.random.default_rng(C + S)
    w = OneHot(F, fmt, page, d, -(-L // page))
    nb = -(-P // page)
    blocks = rng.choice(nb, min(C, nb), replace=False)
    blocks[0] = nb - 1                                        # the block that P cuts
    sinks = rng.choice(L, min(S, L), replace=False)
    if S >= 8:                                                # sinks at the edges, and inside kept blocks
        sinks[:8] = [0, P - 1, g0 - 1, g0, g0 + G - 1, min(L - 1, g0 + G), L - 1, int(blocks[-1]) * page]
    if order == "repeated":
        blocks, sinks = rng.choice(blocks, C), rng.choice(sinks, S) if S else sinks
    elif order == "ascending":
        blocks, sinks = np.sort(blocks), np.unique(sinks)
    lists = []
    for x, n in ((blocks, C), (sinks, S)):
        row = np.full(n, -1, dtype=np.int32)
        row[:min(n, x.size)] = x[:n]
        lists.append(row)
    blocks, sinks = lists
    Q = rand_bf16((1, 2 * w.H, 3, d), 4)
    O = torch.full_like(Q, 5.0)
    every = lambda x: torch.from_numpy(np.tile(x, (1, w.H, 1))).to(DEV)
    F.focus_cache_sparse_attention(Q, None, w.cache, w.table, i32([P]), i32([g0]), G, every(sinks) if S else None,
                                   every(blocks), O)
    w.check(O, lambda b: orc.key_set(P, g0, G, sinks, blocks, page))


@pytest.mark.parametrize("fmt", FMTS)
def test_sparse_in_batches_with_lists_of_their_own(F, fmt):
    """Every (sequence, head) its own lists; shares that end inside units of several heads."""
    page, d, L, B = 64, 128, 4096, 5
    rng = np.random.default_rng(2)
    w = OneHot(F, fmt, page, d, L // page, B)
    P, g0, G, C, S = [4000, 3999, 100, 0, 2048], [4000, 4000, 101, 7, 2050], 46, 20, 12
    blocks = np.stack([np.stack([np.sort(rng.choice(64, C, replace=False)) for _ in range(w.H)]) for _ in range(B)]).astype(np.int32)
    sinks = np.stack([np.stack([rng.choice(L, S, replace=False) for _ in range(w.H)]) for _ in range(B)]).astype(np.int32)
    Q = rand_bf16((B, w.H, 24, d), 4)
    O = torch.full_like(Q, 5.0)
    F.focus_cache_sparse_attention(Q, None, w.cache, w.table, i32(P), i32(g0), G, torch.from_numpy(sinks).to(DEV),
                                   torch.from_numpy(blocks).to(DEV), O)
    for b in range(B):
        for h in range(w.H):
            keys = orc.key_set(P[b], g0[b], G, sinks[b, h], blocks[b, h], page)
            want = np.zeros(d)
            mine = [k for k in keys if k // d == h]
            want[[k % d for k in mine]] = 1.0 / len(keys)
            err = np.abs(O[b, h].double().cpu().numpy() - want)
            assert np.all(err <= 1.01 * 2.0 ** -8 * want), (b, h)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("g,qcap", [(2, 41), (1, 129), (7, 64), (3, 200)])
def test_many_query_rows(F, fmt, g, qcap):
    """More than 64 rows a KV head, in slices of 32 and fewer, against float64."""
    B, H, page, d, L = 2, 2, 32, 128, 700
    w = World(F, fmt, 1, B, H, page, d, -(-L // page), seed=qcap, junk=True)
    Q = rand_bf16((B, g * H, qcap, d), 11)
    O = torch.full_like(Q, 5.0)
    n_q, lens = [qcap, qcap // 2], [L, 133]
    F.focus_cache_attention(Q, i32(n_q), w.cache, w.t_table, i32(lens), O)
    check_attention(w, Q, O, n_q, lambda b, h: np.arange(lens[b]), 1 / np.sqrt(d))
