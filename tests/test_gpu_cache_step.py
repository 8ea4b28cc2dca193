"""The denoising step from the 8-bit cache, and cases of its attention and rows that ordinary
batches do not reach: an attention sink above thousands of small probabilities, more short
sequences than CTAs, lengths outside the table, scales at the ends of fp32."""
import numpy as np
import pytest
import torch

from diffusion_long_context_b200 import inputs
from oracle import cache_oracle as orc
from test_gpu_cache import DEV, DTYPE, F, FMTS, World, check_attention, i32, no_device_error, rand_bf16  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ the step
def view_of(step, l, fmt):
    """Layer l of a step's cache as the oracle sees it."""
    w = World.__new__(World)
    c = step.cache
    w.codes = [t[l:l + 1].view(torch.uint8).cpu().numpy() for t in (c.k, c.v)]
    w.scales = [t[l:l + 1].cpu().numpy() for t in (c.k_scale, c.v_scale)]
    w.table, w.fmt, w.H = step.table.cpu().numpy(), fmt, c.Hkv
    return w


def make_steps(cfg, fmt):
    from diffusion_long_context_b200.step import SparseStep
    st = inputs.step_state(cfg)
    layers = [inputs.make_layer(cfg, l, DEV, st.sink_pos) for l in range(cfg.n_layers)]
    Q = torch.stack([lay[0] for lay in layers])
    K, V = [lay[1] for lay in layers], [lay[2] for lay in layers]
    steps = [SparseStep(cfg, Q, K, V, device=DEV, cache=DTYPE[fmt]), SparseStep(cfg, Q, K, V, device=DEV, fused=False)]
    for s in steps:
        s.set_state(torch.from_numpy(st.conf_prev), torch.from_numpy(st.mask), non_blocking=False)
        s.block_entry()
    return steps


def check_step(step, cfg, fmt):
    nA = step.n_active.cpu().tolist()
    scale = 1 / np.sqrt(cfg.d)
    sinks = step.sinks.cpu().numpy()
    for l in range(cfg.n_layers):
        w = view_of(step, l, fmt)
        if l in step.sparse_layers:
            blocks = step.blocks[l].cpu().numpy()
            keys = lambda b, h: orc.key_set(cfg.P, cfg.g0, cfg.G, sinks[b, h], blocks[b, h], cfg.bs)
        elif l == cfg.l_dense:
            continue                                    # read as bf16 rows, by the kernels of the uncached step
        else:
            keys = lambda b, h: np.arange(cfg.L)
        check_attention(w, step.Q_active[l], step.O_active[l], nA, keys, scale)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("variant", ["plain", "focus_mean_query_tail"])
def test_step_from_the_cache(F, fmt, variant):
    """All layers of a step against float64 over what the cache holds; the selection, which does
    not read the cache, as in the uncached step; then rows refreshed, and the step as a graph."""
    from diffusion_long_context_b200 import configs as cf
    cfg = cf.scaled(cf.LLADA_8K, 1024, n_layers=4, Hq=4, Hkv=2, l_dense=1, C=4, S=8)
    if variant != "plain":
        cfg = cfg.replace(dense_tail=1, relevance="focus", sink_agg="mean_query")
    step, plain = make_steps(cfg, fmt)
    for l in range(cfg.n_layers):                        # block entry stored every layer
        for kv, X in enumerate((step.K[l], step.V[l])):
            got = (step.cache.k, step.cache.v)[kv][l:l + 1].view(torch.uint8).cpu().numpy()
            s = (step.cache.k_scale, step.cache.v_scale)[kv][l:l + 1].cpu().numpy()
            want, ws = np.zeros_like(got), np.zeros_like(s)
            orc.store(X[None].float().cpu().numpy(), want, ws, step.table.cpu().numpy(), [cfg.L] * cfg.B, fmt)
            np.testing.assert_array_equal(got, want)
            np.testing.assert_array_equal(s, ws)
    step.run()
    plain.run()
    torch.cuda.synchronize()
    assert torch.equal(step.i_active, plain.i_active) and torch.equal(step.n_active, plain.n_active)
    assert all(torch.equal(step.blocks[l], plain.blocks[l]) for l in step.sparse_layers)
    check_step(step, cfg, fmt)
    # the sinks, and the sink layer, are those of the uncached call on the cached rows
    l = cfg.l_dense
    K, V = torch.empty_like(step.K[l]), torch.empty_like(step.V[l])
    F.focus_cache_load(step.cache_layers[l], step.table, step.lens, 0, K, V)
    plain.K[l], plain.V[l] = K, V
    plain.run()
    torch.cuda.synchronize()
    assert torch.equal(step.sinks, plain.sinks)
    # (the sink layer's tiles are claimed dynamically, so the last bits may differ)
    torch.testing.assert_close(step.O_active[l].float(), plain.O_active[l].float(), rtol=0, atol=1e-2)

    rows = (cfg.n_layers, cfg.B, cfg.Hkv, cfg.acap, cfg.d)
    new = rand_bf16(rows, 1), rand_bf16(rows, 2)
    act, nA = step.i_active.cpu().numpy(), step.n_active.cpu().tolist()
    want = [(t.view(torch.uint8).cpu().numpy().copy(), s.cpu().numpy().copy())
            for t, s in ((step.cache.k, step.cache.k_scale), (step.cache.v, step.cache.v_scale))]
    step.refresh_rows(*new)
    for (codes, scales), X, t, s in zip(want, new, (step.cache.k, step.cache.v), (step.cache.k_scale, step.cache.v_scale)):
        orc.scatter_rows(X.float().cpu().numpy(), act, nA, codes, scales, step.table.cpu().numpy(), [cfg.L] * cfg.B, fmt)
        np.testing.assert_array_equal(t.view(torch.uint8).cpu().numpy(), codes)
        np.testing.assert_array_equal(s.cpu().numpy(), scales)
    before = [o.clone() for o in step.O_active]
    step.run()
    torch.cuda.synchronize()
    check_step(step, cfg, fmt)
    eager = [o.clone() for o in step.O_active]
    assert all(not torch.equal(a, b) for l, (a, b) in enumerate(zip(before, eager)) if l != cfg.l_dense)
    step.capture()
    step.O_active.fill_(3.0)
    step.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for l, (a, b) in enumerate(zip(eager, step.O_active)) if l != cfg.l_dense)
    step.release()


def test_step_without_a_cache_refuses_its_calls(F):
    from diffusion_long_context_b200 import configs as cf
    from diffusion_long_context_b200.step import SparseStep
    cfg = cf.scaled(cf.LLADA_8K, 1024, n_layers=2, Hq=4, Hkv=2, l_dense=0, C=4, S=8)
    K = [torch.zeros(cfg.B, cfg.Hkv, cfg.L, cfg.d, dtype=torch.bfloat16, device=DEV)] * 2
    Q = torch.zeros(2, cfg.B, cfg.Hq, cfg.L, cfg.d, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="cache"):
        SparseStep(cfg, Q, K, K, device=DEV).refresh_rows(K[0], K[0])
    with pytest.raises(TypeError, match="int8"):
        SparseStep(cfg, Q, K, K, device=DEV, cache=torch.uint8)


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("below", [9.0, 10.6, 11.7, 13.0])
def test_small_probabilities_behind_a_sink(F, fmt, below):
    """One key with almost all the weight and no value, 6000 whose equal probabilities lie
    e^-below under it and make the output. attention_bound allows 2^-15 of the largest
    probability of all for each key; a tile's probabilities are relative to its own largest, so
    here each key's error is 2^-15 of its tile's, which matters outside the sink's tile only."""
    H, page, d, L = 1, 64, 128, 6080
    w = World(F, fmt, 1, 1, H, page, d, -(-L // page), seed=5)
    top = 96.0 if fmt == orc.E4M3 else 120.0
    codes, scales = w.codes, w.scales
    code = lambda x: orc.nearest_codes(np.float32([x]), fmt)[0]
    codes[0][:] = code(0.0)
    scales[0][:], scales[1][:] = 1 / top, 1 / top
    first = w.table[0, 0]
    codes[0][0, first, 0, 0, :] = code(top)                     # the sink: every dim 1
    codes[1][0, first, 0, 0, :] = code(0.0)
    w.upload(F)
    scale = below / d                                           # q = 1 everywhere: the sink scores `below`, all others 0
    Q = torch.ones((1, 4, 3, d), dtype=torch.bfloat16, device=DEV)
    O = torch.zeros_like(Q)
    F.focus_cache_attention(Q, None, w.cache, w.t_table, i32([L]), O, scale=scale)
    K, V = (orc.values(codes[kv], scales[kv], w.table[0], np.arange(L), 0, fmt) for kv in range(2))
    t = scale * K.sum(axis=1)
    p = np.exp(t - t.max())
    l = p.sum()
    o = (p[:, None] * V).sum(axis=0) / l
    # output 2^-8 |o|; each probability 2^-8 of itself (a bias, if all are equal) and 2^-15 of its
    # tile's largest; scores as in attention_bound with spread = scale sum|k| max|q| <= below
    tiles = np.arange(L) // 128
    largest = np.array([p[tiles == i].max() for i in range(tiles.max() + 1)])[tiles]
    mean_abs = (p[:, None] * np.abs(V)).sum(axis=0) / l
    floor = (largest[:, None] * np.abs(V)).sum(axis=0) / l
    lim = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2 * 2 * 2.0 ** -14 * below) * mean_abs + 2.0 ** -15 * floor
    err = np.abs(O.double().cpu().numpy() - o)
    assert np.all(err <= lim), float((err / lim).max())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("score", [-5000.0, 300.0, 1500.0, 7000.0, 60000.0])
def test_scores_far_from_zero(F, fmt, score):
    """All keys score the same, far from zero: the output is the mean value. The query is exact in
    8 bits (2^n, or the row's largest) and the keys' codes alike, so the scores are the same in
    fp32 too; each probability, equal for all, may be off by 2^-8, and the output by half a step."""
    H, page, d, L = 2, 32, 64, 700
    w = World(F, fmt, 1, 1, H, page, d, -(-L // page), seed=5)
    w.codes[0][:] = orc.nearest_codes(np.float32([64.0]), fmt)[0]
    w.scales[0][:] = 1 / 64
    w.upload(F)
    Q = torch.ones((1, 4, 3, d), dtype=torch.bfloat16, device=DEV)
    O = torch.zeros_like(Q)
    F.focus_cache_attention(Q, None, w.cache, w.t_table, i32([L]), O, scale=score / d)
    for h in range(H):
        V = orc.values(w.codes[1], w.scales[1], w.table[0], np.arange(L), h, fmt)
        err = np.abs(O[0, 2 * h:2 * h + 2].double().cpu().numpy() - V.mean(axis=0))
        assert np.all(err <= 2.0 ** -8 * np.abs(V.mean(axis=0)) + 2.0 ** -8 * np.abs(V).mean(axis=0))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("kv", [0, 1])
@pytest.mark.parametrize("sparse", [False, True])
def test_a_page_that_is_not_finite_makes_its_readers_nan(F, fmt, bad, kv, sparse):
    """One element of one head's keys or values is not finite: all rows of that head that read its
    page are NaN, in every dim; the other head and a sequence that does not read the page are not."""
    B, H, page, d, L = 2, 2, 32, 64, 300
    w = World(F, fmt, 1, B, H, page, d, -(-L // page), seed=4)
    K, V = rand_bf16((B, H, L, d), 1), rand_bf16((B, H, L, d), 2)
    (K, V)[kv][0, 1, 70, 5] = bad
    F.focus_cache_store(K, V, w.cache, w.t_table)
    Q = rand_bf16((B, 4, 5, d), 6)
    O = torch.full_like(Q, 5.0)
    n_q = i32([5, 4])
    if sparse:                                                  # the page through a sink and through a block
        blocks = torch.tensor([[[0, -1], [2, 5]], [[2, -1], [2, 3]]], dtype=torch.int32, device=DEV)
        sinks = torch.tensor([[[4], [10]], [[4], [70]]], dtype=torch.int32, device=DEV)
        F.focus_cache_sparse_attention(Q, n_q, w.cache, w.t_table, i32([256, 256]), i32([256, 256]), 32, sinks, blocks, O)
    else:
        F.focus_cache_attention(Q, n_q, w.cache, w.t_table, i32([L, L]), O)
    assert torch.all(torch.isnan(O[0, 2:]))
    assert torch.all(torch.isfinite(O[0, :2])) and torch.all(torch.isfinite(O[1])) and not O[1, :, 4].any()
    if sparse:
        sinks[0, 1, 0], blocks[0, 1, 0] = 70, 7                 # by the sink alone
        F.focus_cache_sparse_attention(Q, n_q, w.cache, w.t_table, i32([256, 256]), i32([256, 256]), 32, sinks, blocks, O)
        assert torch.all(torch.isnan(O[0, 2:])) and torch.all(torch.isfinite(O[0, :2])) and torch.all(torch.isfinite(O[1]))


@pytest.mark.parametrize("fmt", FMTS)
def test_more_short_sequences_than_ctas(F, fmt):
    """Several runs to a CTA: 200 sequences, 2 KV heads, lengths about one tile, some empty."""
    B, H, page, d, qcap = 200, 2, 16, 64, 2
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 140, B)
    lens[rng.integers(0, B, 30)] = 0
    lens[[0, B - 1]] = 0, 129
    w = World(F, fmt, 1, B, H, page, d, 9, seed=8, junk=True)
    Q = rand_bf16((B, 6, qcap, d), 6)
    O = torch.full_like(Q, 5.0)
    n_q = rng.integers(0, qcap + 1, B)
    F.focus_cache_attention(Q, i32(n_q), w.cache, w.t_table, i32(lens), O)
    check_attention(w, Q, O, n_q, lambda b, h: np.arange(lens[b]), 1 / np.sqrt(d))


@pytest.mark.parametrize("graph", [False, True])
def test_inputs_that_change_from_call_to_call(F, graph):
    """Lengths, row counts, prompt ends and table are written right before each call, without a wait
    in between (the joining kernel reads some of them while the attention still runs)."""
    B, H, page, d, qcap, n = 5, 2, 32, 128, 3, 24
    rng = np.random.default_rng(9)
    w = World(F, orc.E4M3, 1, B, H, page, d, 40, seed=3)
    Q = rand_bf16((B, 4, qcap, d), 6)
    lens, n_q = (i32(rng.integers(0, top, (n, B))) for top in (1281, qcap + 1))
    P = i32(rng.integers(0, 1200, (n, B)))
    tables = torch.stack([w.t_table[i32(rng.permutation(B)).long()] for _ in range(n)])
    blocks = i32(rng.integers(-1, 38, (B, H, 6)))
    ws = torch.empty(F.cache_workspace_bytes(B, 4, H, d, qcap), dtype=torch.uint8, device=DEV)
    cur = [torch.zeros_like(x[0]) for x in (lens, n_q, P, tables)]
    O = torch.zeros((n, 2, *Q.shape), dtype=torch.bfloat16, device=DEV)

    def call(i, out, copy=True):
        args = [x[i] for x in (lens, n_q, P, tables)]
        if copy:
            for c, x in zip(cur, args):
                c.copy_(x)
            args = cur
        F.focus_cache_attention(Q, args[1], w.cache, args[3], args[0], out[0], ws=ws)
        F.focus_cache_sparse_attention(Q, args[1], w.cache, args[3], args[2], args[2], 32, None, blocks, out[1], ws=ws)

    if graph:
        side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side), torch.cuda.graph(g, stream=side):
            for i in range(n):
                call(i, O[i])
        torch.cuda.current_stream().wait_stream(side)
        g.replay()
        g.replay()
    else:
        for i in range(n):
            call(i, O[i])
    torch.cuda.synchronize()
    want = torch.zeros_like(O[0])
    for i in range(n):
        call(i, want, copy=False)
        torch.cuda.synchronize()
        assert torch.equal(O[i], want), i


def test_lengths_below_zero_have_no_keys(F):
    w = World(F, orc.INT8, 1, 3, 2, 32, 128, 4, seed=2)
    Q = rand_bf16((3, 4, 5, 128), 6)
    O = torch.full_like(Q, 5.0)
    F.focus_cache_attention(Q, None, w.cache, w.t_table, i32([-1, 100, -2 ** 31]), O)
    assert not O[0].any() and not O[2].any()
    check_attention(w, Q, O, None, lambda b, h: np.arange([0, 100, 0][b]), 1 / np.sqrt(128))
    X = torch.full((1, 3, 2, 8, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    Y = X.clone()
    F.focus_cache_load(w.cache, w.t_table, i32([-1, 0, -2 ** 31]), 0, X, Y)
    assert torch.all(X == 7) and torch.all(Y == 7)
    F.focus_cache_store(X, Y, w.cache, w.t_table, i32([-1, 0, -2 ** 31]))
    w.assert_same()


def test_lengths_beyond_the_table_are_cut_and_flagged(F):
    w = World(F, orc.E4M3, 1, 2, 2, 32, 128, 4, seed=2)
    Q = rand_bf16((2, 4, 5, 128), 6)
    O = torch.full_like(Q, 5.0)
    F.focus_cache_attention(Q, None, w.cache, w.t_table, i32([129, 2 ** 31 - 1]), O)
    check_attention(w, Q, O, None, lambda b, h: np.arange(128), 1 / np.sqrt(128))


# ------------------------------------------------------------------ rows
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("power", [-133, -126, -95, -80, -62, -1, 60, 95, 118, 127])
def test_codes_at_every_scale(F, fmt, power):
    """Rows whose largest is about 2^power, beside elements down to 2^-40 of it and both zeros:
    stored, then refreshed with larger rows, so that the held codes are made anew."""
    page, d, H = 32, 64, 3
    w = World(F, fmt, 1, 1, H, page, d, 2, seed=1)
    rng = np.random.default_rng(abs(power))
    shape = (1, 1, H, 2 * page, d)
    with np.errstate(under="ignore", over="ignore"):
        x = (1 + rng.random(shape)) * rng.choice([-1.0, 1.0], shape) * 2.0 ** (power - rng.integers(0, 41, shape) * (rng.random(shape) < 0.5))
    x[..., 0], x[..., 1] = 0.0, -0.0
    X = torch.from_numpy(x.clip(-3e38, 3e38).astype(np.float32)).to(torch.bfloat16).to(DEV)
    F.focus_cache_store(X, -X, w.cache, w.t_table)
    for kv, Y in enumerate((X, -X)):
        orc.store(Y.float().cpu().numpy(), w.codes[kv], w.scales[kv], w.table, [2 * page], fmt)
    w.assert_same()
    rows = np.array([[3, 40, 41]], dtype=np.int32)
    R = (X[:, :, :, 5:8].float() * 1.7).clamp(-3e38, 3e38).to(torch.bfloat16).contiguous()
    F.focus_cache_scatter_rows(R, -R, torch.from_numpy(rows).to(DEV), i32([3]), w.cache, w.t_table, i32([2 * page]))
    for kv, Y in enumerate((R, -R)):
        orc.scatter_rows(Y.float().cpu().numpy(), rows, [3], w.codes[kv], w.scales[kv], w.table, [2 * page], fmt)
    w.assert_same()


@pytest.mark.parametrize("fmt", FMTS)
def test_recoding_under_many_scales(F, fmt):
    """Every code under 2048 pairs of scales: the held codes of 2048 heads grow by a ratio each."""
    page, d, H = 16, 64, 2048
    w = World(F, fmt, 1, 1, H, page, d, 1, seed=1)
    rng = np.random.default_rng(4)
    p = w.table[0, 0]
    every = np.arange(256, dtype=np.uint8)
    every = every[(every & 0x7F) != 0x7F] if fmt == orc.E4M3 else every[every != 0x80]
    held = np.resize(every, (15, d))
    for kv in range(2):
        w.codes[kv][0, p, :, :15] = held
        w.scales[kv][0, p] = (0.5 + rng.random(H)).astype(np.float32) * np.float32(2.0) ** rng.integers(-20, 20, H)
    w.upload(F)
    top = orc.TOP[fmt]
    R = [torch.from_numpy((w.scales[kv][0, p] * top * (1 + 3 * rng.random(H)))[None, None, :, None, None] *
                          np.ones((1, 1, H, 1, d))).to(torch.bfloat16).to(DEV) for kv in range(2)]
    rows = np.array([[15]], dtype=np.int32)
    F.focus_cache_scatter_rows(*R, torch.from_numpy(rows).to(DEV), i32([1]), w.cache, w.t_table, i32([16]))
    for kv in range(2):
        orc.scatter_rows(R[kv].float().cpu().numpy(), rows, [1], w.codes[kv], w.scales[kv], w.table, [16], fmt)
    w.assert_same()
