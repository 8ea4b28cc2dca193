"""Cases for the 8-bit paged key/value cache: what goes into it, the attention that reads it, and the care of its pages.

The cache holds the keys and values of n_mat layers as codes [n_mat, n_pages, Hkv, page, d]
(e4m3 or 8-bit integers) with one fp32 scale for each page and head, [n_mat, n_pages, Hkv];
table [B, cols] names the page that holds positions [j * page, (j + 1) * page) of a sequence.

A page's scale is s = (largest |x| of its rows) / top, top = 448 (e4m3) or 127 (int8), and a
code is x / s rounded to the nearest (ties to even); both are formed in fp32, which is part of
the definition, and a page of zeros has s = 0 and zero codes.

Kinds of case, and the calls that each stands for:
  store   a prompt's bf16 keys and values go into the cache, and the layer that needs them in
          bf16 (the sink layer) reads them back
  update  the active rows of a denoising step replace their cached rows, and are read back
  attend  attention of few queries over all cached positions (dense layers; single tokens)
  sparse  attention over sinks, kept pages of the prompt and the current block
  fork    branches of a sequence: drop the old ones, share the pages, copy those to be written
  compact the live pages of a fragmented pool move to its front
"""
import math

import torch

own = False

DEV = "cuda"
FORMATS = {"e4m3": (torch.float8_e4m3fn, 448.0), "int8": (torch.int8, 127.0)}


def listed():
    return [
        # block entry at 32K: one layer's keys and values of the whole context
        dict(name="store_32k_mha_e4m3", kind="store", fmt="e4m3", n_mat=1, B=1, Hkv=32, L=32768, d=128, page=64),
        # three prompts of unlike, odd lengths, two layers at a time, grouped heads
        dict(name="store_ragged_gqa_int8", kind="store", fmt="int8", n_mat=2, B=3, Hkv=4, L=5003, d=128, page=32),
        # the rows of one denoising step, all 32 layers, a block of 32 behind an 8K context
        dict(name="update_32_layers_e4m3", kind="update", fmt="e4m3", n_mat=32, B=1, Hkv=32, L=8192, d=128, page=64,
             cap=32),
        # the same for four sequences of grouped heads, one layer, 23 rows of room
        dict(name="update_1_layer_int8", kind="update", fmt="int8", n_mat=1, B=4, Hkv=4, L=2100, d=128, page=16,
             cap=23),
        # one token of one sequence, grouped heads, 8K: latency counts
        dict(name="attend_1_token_8k_gqa", kind="attend", fmt="e4m3", B=1, Hq=28, Hkv=4, L=8192, d=128, page=64,
             qcap=1),
        # a dense layer of the 32K denoising step: 32 active queries over the whole context
        dict(name="attend_32_rows_32k_mha", kind="attend", fmt="e4m3", B=1, Hq=32, Hkv=32, L=32768, d=128, page=64,
             qcap=32),
        # the 16K grouped-head model's dense layer, 8-bit integers
        dict(name="attend_32_rows_16k_gqa_int8", kind="attend", fmt="int8", B=1, Hq=28, Hkv=4, L=16384, d=128,
             page=64, qcap=32),
        # sixteen sequences of very unlike lengths, one token each, small pages
        dict(name="attend_ragged_16_seqs", kind="attend", fmt="int8", B=16, Hq=32, Hkv=8, L=12289, d=128, page=32,
             qcap=1),
        # a sparse layer of the 32K step: 64 kept blocks, 32 sinks, the current block
        dict(name="sparse_32k_mha", kind="sparse", fmt="e4m3", B=1, Hq=32, Hkv=32, L=32768, d=128, page=64, qcap=32,
             G=32, C=64, S=32),
        # four sequences with prompts of their own, 16 kept blocks, 8K, 8-bit integers
        dict(name="sparse_8k_batch_int8", kind="sparse", fmt="int8", B=4, Hq=32, Hkv=32, L=8192, d=128, page=64,
             qcap=24, G=32, C=16, S=16),
        # eight branches of one 4K sequence, each about to write its last block
        dict(name="fork_8_branches", kind="fork", fmt="e4m3", n_mat=8, Hkv=32, d=128, page=64, n_pages=256, held=64,
             n=8, own=2),
        # a pool of 512 pages, two fifths of it in use all over
        dict(name="compact_512_pages", kind="compact", fmt="int8", n_mat=4, Hkv=32, d=128, page=64, n_pages=512,
             n=12),
    ]


def draw(rng):
    def log(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    kind = rng.choice(["store", "update", "attend", "attend", "sparse", "sparse", "fork", "compact"])
    fmt = rng.choice(["e4m3", "int8"])
    page = rng.choice([16, 32, 64, 128])
    d = rng.choice([64, 128, 128])
    Hq, Hkv = rng.choice([(32, 32), (28, 4), (4, 4), (32, 8)])
    if kind in ("store", "update"):
        n_mat, B, L = rng.choice([1, 2, 5]), rng.randint(1, 4), log(1, 20000)
        while n_mat * B * Hkv * L > 32 * 32768:
            L = max(1, L // 2)
        c = dict(kind=kind, fmt=fmt, n_mat=n_mat, B=B, Hkv=Hkv, L=L, d=d, page=page)
        return c if kind == "store" else dict(c, cap=rng.randint(1, 40))
    if kind == "attend":
        B, qcap, L = log(1, 24), rng.choice([1, 1, rng.randint(2, 40)]), log(1, 32768)
        while B * Hkv * L > 32 * 32768 or B * Hq * L * qcap > 32 * 32 * 32768:
            B, L = max(1, B // 2), max(1, L - L // 3)
        return dict(kind=kind, fmt=fmt, B=B, Hq=Hq, Hkv=Hkv, L=L, d=d, page=page, qcap=qcap)
    if kind == "sparse":
        B, L, C = rng.randint(1, 4), log(600, 32768), log(1, 64)
        while B * L > 65536 or B * Hq * C * page > 32 * 64 * 64:
            B, C = max(1, B - 1), max(1, C // 2)
            if B * L > 65536:
                L //= 2
        return dict(kind=kind, fmt=fmt, B=B, Hq=Hq, Hkv=Hkv, L=L, d=d, page=page, qcap=rng.randint(1, 40),
                    G=rng.choice([16, 32, 48]), C=C, S=rng.randint(0, 48))
    n_mat, n_pages = rng.randint(1, 4), rng.randint(60, 400)
    c = dict(kind=kind, fmt=fmt, n_mat=n_mat, Hkv=Hkv, d=d, page=page, n_pages=n_pages)
    if kind == "fork":
        held = rng.randint(2, n_pages // 3)
        n = rng.randint(1, 6)
        return dict(c, held=held, n=n, own=rng.randint(1, max(1, min(held, (n_pages - held) // n))))
    return dict(c, n=rng.randint(1, 12))


# --------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1_000_003 + 17)
    return g


def _lens(B, L, g):
    """Unlike lengths up to L, the first of them L itself; of more than two sequences one is empty."""
    lens = torch.randint(1, L + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    lens[0] = L
    if B > 2:
        lens[B // 2] = 0
    return lens


def _table(B, cols, spare, g):
    """Pages of B sequences in random order, out of B * cols + spare."""
    n_pages = B * cols + spare
    return torch.randperm(n_pages, generator=g, device=DEV)[: B * cols].to(torch.int32).view(B, cols), n_pages


def _codes(shape, fmt, g):
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    if fmt == "int8":
        return (x * 35).clamp_(-127, 127).round_().to(torch.int8)
    return (x * 120).clamp_(-448, 448).to(torch.float8_e4m3fn)


def _scales(shape, fmt, g):
    """Scales of keys and values of about unit size, unlike from page to page."""
    unit = 1.0 / (35 if fmt == "int8" else 120)
    return torch.exp(0.4 * torch.randn(shape, generator=g, device=DEV)) * unit


def _pool(n_mat, n_pages, c, g):
    shape = (n_mat, n_pages, c["Hkv"], c["page"], c["d"])
    return dict(k=_codes(shape, c["fmt"], g), v=_codes(shape, c["fmt"], g), ks=_scales(shape[:3], c["fmt"], g),
                vs=_scales(shape[:3], c["fmt"], g))


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(case)
    kind = c["kind"]
    if kind in ("store", "update", "attend", "sparse"):
        B, cols = c["B"], -(-c["L"] // c["page"])
        s["table"], n_pages = _table(B, cols, 3, g)
        s["lens"] = _lens(B, c["L"], g)
    i32 = dict(device=DEV, dtype=torch.int32)
    if kind == "store":
        shape = (c["n_mat"], B, c["Hkv"], c["L"], c["d"])
        s["K"] = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
        s["V"] = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
        s["K"][..., :: max(1, c["L"] // 5), :] *= 3          # a few large keys, as attention sinks have
        s.update(_pool(c["n_mat"], n_pages, c, g))
        for k in ("ks", "vs"):
            s[k].zero_()
        s["outK"], s["outV"] = torch.zeros_like(s["K"]), torch.zeros_like(s["V"])
    elif kind == "update":
        cap, L = c["cap"], c["L"]
        s.update(_pool(c["n_mat"], n_pages, c, g))
        shape = (c["n_mat"], B, c["Hkv"], cap, c["d"])
        s["K_rows"] = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
        s["V_rows"] = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
        # the first sequence holds L positions, and some of its last ones are replaced; the
        # others grow by rows that are new
        wide = min(L, cap + cap // 2)
        lo, n = L - wide, min(cap, wide)
        s["n_rows"] = torch.randint(max(1, n // 2), n + 1, (B,), generator=g, **i32)
        some = torch.rand((wide,), generator=g, device=DEV).argsort()
        some = torch.where(torch.arange(wide, device=DEV) < s["n_rows"][0], some, wide).sort().values[:cap]
        rows = torch.full((B, cap), -1, **i32)
        rows[:, :n] = lo + torch.arange(n, **i32)
        rows[0, : some.numel()] = torch.where(some < wide, lo + some, -1).to(torch.int32)
        s["rows"] = rows
        s["lens"] = torch.full((B,), lo, **i32)
        s["after"] = lo + s["n_rows"]
        s["lens"][0] = s["after"][0] = L
        s["start"] = lo // c["page"] * c["page"]
        s["W"] = L - s["start"]
        oshape = (c["n_mat"], B, c["Hkv"], s["W"], c["d"])
        s["outK"] = torch.zeros(oshape, device=DEV, dtype=torch.bfloat16)
        s["outV"] = torch.zeros(oshape, device=DEV, dtype=torch.bfloat16)
    elif kind in ("attend", "sparse"):
        s.update(_pool(1, n_pages, c, g))
        qshape = (B, c["Hq"], c["qcap"], c["d"])
        s["Q"] = torch.randn(qshape, generator=g, device=DEV, dtype=torch.bfloat16)
        s["n_q"] = torch.randint(1, c["qcap"] + 1, (B,), generator=g, **i32)
        s["n_q"][0] = c["qcap"]
        s["O"] = torch.zeros(qshape, device=DEV, dtype=torch.bfloat16)
    if kind == "sparse":
        G, C, S, page = c["G"], c["C"], c["S"], c["page"]
        top = c["L"] - G
        P = torch.randint(max(1, top // 2), top + 1, (B,), generator=g, **i32)
        P[0] = top
        s["P"], s["g0"], s["Gn"] = P, P.clone(), G
        nb = -(-top // page)
        score = torch.rand((B, c["Hkv"], nb), generator=g, device=DEV)
        have = -(-P.long() // page)                          # blocks of each prompt
        score = torch.where(torch.arange(nb, device=DEV) < have[:, None, None], score, -1.0)
        k = min(C, nb)
        best = score.topk(k, dim=-1)
        idx = torch.where(best.values >= 0, best.indices, 1 << 30).sort(-1).values
        blocks = torch.full((B, c["Hkv"], C), -1, **i32)
        blocks[..., :k] = torch.where(idx < (1 << 30), idx, -1).to(torch.int32)
        s["blocks"] = blocks
        pos = torch.rand((B, c["Hkv"], c["L"]), generator=g, device=DEV)
        pos = torch.where(torch.arange(c["L"], device=DEV) < (P.long() + G)[:, None, None], pos, -1.0)
        s["sinks"] = pos.topk(S, dim=-1).indices.sort(-1).values.to(torch.int32).contiguous() if S else None
    elif kind == "fork":
        s.update(_pool(c["n_mat"], c["n_pages"], c, g))
        n, held, cols = c["n"], c["held"], c["held"] + 2
        table = torch.full((n + 1, cols), -1, **i32)
        pages = torch.randperm(c["n_pages"], generator=g, device=DEV).to(torch.int32)
        table[0, :held] = pages[:held]
        refs = torch.zeros(c["n_pages"], **i32)
        refs[pages[:held].long()] = 1
        heldv = torch.zeros(n + 1, **i32)
        heldv[0] = held
        s.update(table=table, refs=refs, held_v=heldv)
        s["dst"] = torch.arange(1, n + 1, **i32)
        s["src"] = torch.zeros(n, **i32)
        s["keep"] = torch.full((n,), held, **i32)
        s["none"] = torch.zeros(n, **i32)
        s["first"] = torch.full((n,), held - c["own"], **i32)
    elif kind == "compact":
        s.update(_pool(c["n_mat"], c["n_pages"], c, g))
        n, cols = c["n"], max(1, int(0.4 * c["n_pages"]) // c["n"])
        pages = torch.randperm(c["n_pages"], generator=g, device=DEV).to(torch.int32)
        table = pages[: n * cols].view(n, cols).clone()
        refs = torch.zeros(c["n_pages"], **i32)
        refs[table.long().view(-1)] = 1
        table[n - 1, : cols // 2] = table[0, : cols // 2]    # a branch: its own first pages are free, it shares
        refs.zero_()
        refs.index_add_(0, table.long().view(-1), torch.ones(n * cols, **i32))
        s.update(table0=table, refs0=refs, table=table.clone(), refs=refs.clone(),
                 held_v=torch.full((n,), cols, **i32))
    if kind in ("fork", "compact"):
        s["pairs"] = torch.zeros((c["n_pages"], 2), **i32)
        s["n_pairs"] = torch.zeros(1, **i32)
        s["remap"] = torch.zeros(c["n_pages"], **i32)
        s["status"] = torch.zeros(1, **i32)
    return s


# --------------------------------------------------------------------------- the framework's calls
def _handles(s):
    """The handles that a program makes once, when it lays out its cache."""
    if "cache" not in s:
        from diffusion_long_context_b200 import focus as F
        s["F"] = F
        s["cache"] = F.Cache(s["k"], s["v"], s["ks"], s["vs"])
        if s["kind"] in ("fork", "compact"):
            s["pages"] = F.Pages(s["refs"], s["table"], s["held_v"])
        if s["kind"] in ("attend", "sparse"):
            n = F.cache_workspace_bytes(s["B"], s["Hq"], s["Hkv"], s["d"], s["qcap"])
            s["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)
    return s["F"], s["cache"]


def _run_own(s):
    F, cache = _handles(s)
    kind = s["kind"]
    if kind == "store":
        F.focus_cache_store(s["K"], s["V"], cache, s["table"], s["lens"])
        F.focus_cache_load(cache, s["table"], s["lens"], 0, s["outK"], s["outV"])
    elif kind == "update":
        F.focus_cache_scatter_rows(s["K_rows"], s["V_rows"], s["rows"], s["n_rows"], cache, s["table"], s["lens"])
        F.focus_cache_load(cache, s["table"], s["after"], s["start"], s["outK"], s["outV"])
    elif kind == "attend":
        F.focus_cache_attention(s["Q"], s["n_q"], cache, s["table"], s["lens"], s["O"], ws=s["ws"])
    elif kind == "sparse":
        F.focus_cache_sparse_attention(s["Q"], s["n_q"], cache, s["table"], s["P"], s["g0"], s["Gn"], s["sinks"],
                                       s["blocks"], s["O"], ws=s["ws"])
    elif kind == "fork":
        F.focus_pages_release(s["pages"], s["dst"], s["none"])
        F.focus_pages_fork(s["pages"], s["src"], s["dst"], s["keep"])
        F.focus_pages_own(s["pages"], s["dst"], s["first"], s["keep"], s["pairs"], s["n_pairs"], s["status"])
        F.focus_pages_copy(cache, s["pairs"], s["n_pairs"])
    else:
        s["table"].copy_(s["table0"])
        s["refs"].copy_(s["refs0"])
        F.focus_pages_compact(s["pages"], s["pairs"], s["n_pairs"], s["remap"])
        F.focus_pages_copy(cache, s["pairs"], s["n_pairs"])


# --------------------------------------------------------------------------- plain forms
def _encode(x, scale, fmt):
    """Codes of x (fp32) under a scale that broadcasts against it."""
    dt, top = FORMATS[fmt]
    y = torch.where(scale > 0, x / torch.where(scale > 0, scale, 1.0), 0.0).clamp(-top, top)
    return y.round().to(dt) if fmt == "int8" else y.to(dt)


def _paged(x, cols, page):
    """[n, B, H, L, d] -> [n, B, H, cols, page, d] with zeros behind L."""
    pad = cols * page - x.shape[3]
    return torch.nn.functional.pad(x, (0, 0, 0, pad)).unflatten(3, (cols, page))


def _plain_store(s):
    page, fmt = s["page"], s["fmt"]
    table, lens = s["table"].long(), s["lens"].long()
    cols = table.shape[1]
    top = torch.full((), FORMATS[fmt][1], device=DEV)
    pos = torch.arange(cols * page, device=DEV).view(cols, page)
    live = pos < lens[:, None, None]                                   # [B, cols, page]
    bi, ci = live.any(-1).nonzero(as_tuple=True)
    phys = table[bi, ci]
    for x, code, scale in ((s["K"], s["k"], s["ks"]), (s["V"], s["v"], s["vs"])):
        xp = _paged(x, cols, page)[:, bi, :, ci].float()               # [pages, n, H, page, d]
        m = live[bi, ci][:, None, None, :, None]
        sc = torch.where(m, xp, 0.0).abs().amax((-1, -2)) / top
        new = _encode(xp, sc[..., None, None], fmt)
        old = code[:, phys].transpose(0, 1)
        code.view(torch.uint8)[:, phys] = torch.where(m, new.view(torch.uint8), old.view(torch.uint8)).transpose(0, 1)
        scale[:, phys] = sc.transpose(0, 1)
    _plain_load(s, s["lens"], 0)


def _plain_load(s, lens, start):
    page, table = s["page"], s["table"].long()
    W = s["outK"].shape[3]
    pos = start + torch.arange(W, device=DEV)
    phys = table[:, pos // page]                                       # [B, W]
    row = (pos % page).expand_as(phys)
    live = (pos < lens.long()[:, None])[None, :, None, :, None]
    for code, scale, out in ((s["k"], s["ks"], s["outK"]), (s["v"], s["vs"], s["outV"])):
        # [B, W, n, H, d]: the layers and heads of each position's row
        x = code.view(torch.uint8).permute(1, 3, 0, 2, 4)[phys, row].view(code.dtype).float()
        x = x * scale.permute(1, 0, 2)[phys][..., None]
        out.copy_(torch.where(live, x.permute(2, 0, 3, 1, 4), out.float()))


def _plain_update(s):
    page, fmt, start = s["page"], s["fmt"], s["start"]
    table, lens, rows = s["table"].long(), s["lens"].long(), s["rows"].long()
    B, cap = rows.shape
    W = -(-s["W"] // page) * page
    top = torch.full((), FORMATS[fmt][1], device=DEV)
    real = torch.arange(cap, device=DEV) < s["n_rows"].long()[:, None]
    at = torch.where(real, rows - start, W)                            # place in the window, W = nowhere
    src = torch.full((B, W + 1), -1, device=DEV).scatter_(1, at, torch.arange(cap, device=DEV).expand(B, cap))
    src = src[:, :W].view(B, W // page, page)                          # the row that each position takes
    fresh = src >= 0
    pos = start + torch.arange(W, device=DEV).view(W // page, page)
    had = (pos < lens[:, None, None]) & ~fresh
    bi, ci = fresh.any(-1).nonzero(as_tuple=True)                      # the pages that rows fall in
    phys = table[bi, ci + start // page]
    new_m, had_m = (t[bi, ci][:, None, None, :, None] for t in (fresh, had))
    used = (pos[ci, 0] < lens[bi])[:, None, None]
    for x, code, scale in ((s["K_rows"], s["k"], s["ks"]), (s["V_rows"], s["v"], s["vs"])):
        xr = x.permute(1, 3, 0, 2, 4)[bi[:, None], src[bi, ci].clamp(min=0)].permute(0, 2, 3, 1, 4).float()
        m = torch.where(new_m, xr, 0.0).abs().amax((-1, -2)) / top
        old_s = torch.where(used, scale[:, phys].transpose(0, 1), 0.0)
        sc = torch.maximum(old_s, m)
        old = code.view(torch.uint8)[:, phys].transpose(0, 1)
        again = _encode(old.view(code.dtype).float() * old_s[..., None, None], sc[..., None, None], fmt)
        out = torch.where(new_m, _encode(xr, sc[..., None, None], fmt).view(torch.uint8),
                          torch.where(had_m & (sc > old_s)[..., None, None], again.view(torch.uint8), old))
        code.view(torch.uint8)[:, phys] = out.transpose(0, 1)
        scale[:, phys] = sc.transpose(0, 1)
    _plain_load(s, s["after"], start)


def _attend(s, K, V, live):
    """softmax(Q K^T / sqrt(d)) V of grouped heads over keys [B, H, n, d] where live [B, H, n]."""
    B, Hq, A, d = s["Q"].shape
    H = s["Hkv"]
    q = s["Q"].float().view(B, H, Hq // H * A, d)
    t = (q @ K.transpose(-1, -2)) / math.sqrt(d)
    t = t.masked_fill(~live[:, :, None], -torch.inf)
    top = t.amax(-1, keepdim=True)
    p = torch.exp(t - torch.where(top == -torch.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = (p @ V) / torch.where(total > 0, total, 1.0)
    o = o.view(B, Hq, A, d)
    rows = torch.arange(A, device=DEV) < s["n_q"].long()[:, None]
    s["O"].copy_(torch.where(rows[:, None, :, None], o, 0.0))


def _plain_attention(s):
    B, H, page = s["B"], s["Hkv"], s["page"]
    phys = s["table"].long()
    L = phys.shape[1] * page
    live = torch.arange(L, device=DEV) < s["lens"].long()[:, None]

    def take(code, scale):
        x = code[0].view(torch.uint8)[phys].view(code.dtype).float() * scale[0][phys][..., None, None]
        x = x.permute(0, 2, 1, 3, 4).reshape(B, H, L, -1)
        return torch.where(live[:, None, :, None], x, 0.0)

    _attend(s, take(s["k"], s["ks"]), take(s["v"], s["vs"]), live[:, None].expand(B, H, L))


def _plain_sparse(s):
    B, H, page, G = s["B"], s["Hkv"], s["page"], s["Gn"]
    blocks = s["blocks"].long()
    P, g0 = (s[k].long()[:, None, None] for k in ("P", "g0"))
    gen = (g0 + torch.arange(G, device=DEV)).expand(B, H, G)
    blk = blocks[..., None] * page + torch.arange(page, device=DEV)
    blk_live = ((blocks >= 0)[..., None] & (blk < P[..., None])).flatten(2)
    blk = blk.flatten(2)
    parts, live = [gen, blk], [torch.ones_like(gen, dtype=torch.bool), blk_live & ((blk < g0) | (blk >= g0 + G))]
    if s["sinks"] is not None:
        snk = s["sinks"].long()
        kept = ((snk // page)[..., None] == blocks[..., None, :]).any(-1) & (snk < P)
        parts.append(snk)
        live.append((snk >= 0) & ~kept & ((snk < g0) | (snk >= g0 + G)))
    pos, live = torch.cat(parts, -1), torch.cat(live, -1)
    pos = torch.where(live, pos, 0)
    phys = s["table"].long()[torch.arange(B, device=DEV)[:, None, None], pos // page]
    heads = torch.arange(H, device=DEV)[None, :, None]

    def take(code, scale):
        x = code[0].view(torch.uint8)[phys, heads, pos % page].view(code.dtype).float() * scale[0][phys, heads][..., None]
        return torch.where(live[..., None], x, 0.0)

    _attend(s, take(s["k"], s["ks"]), take(s["v"], s["vs"]), live)


def _plain_copy(s, src, dst):
    for t in (s["k"].view(torch.uint8), s["v"].view(torch.uint8), s["ks"], s["vs"]):
        t[:, dst] = t[:, src]


def _plain_fork(s):
    table, refs, held = s["table"], s["refs"], s["held_v"]
    dst, one = s["dst"].long(), torch.ones((), device=DEV, dtype=torch.int32)
    col = torch.arange(table.shape[1], device=DEV)
    # the old branches go
    old = table[dst]
    has = col < held[dst][:, None]
    refs.index_add_(0, old[has].long(), -one.expand(int(has.sum())))
    table[dst] = -1
    # the new ones share the source's pages
    keep = torch.minimum(s["keep"], held[s["src"].long()])
    rows = torch.where(col < keep[:, None], table[s["src"].long()], -1)
    table[dst] = rows
    held[dst] = keep
    has = rows >= 0
    refs.index_add_(0, rows[has].long(), one.expand(int(has.sum())))
    # and get their own copies of those that they will write
    mine = (col >= s["first"][:, None]) & (col < keep[:, None])
    bi, ci = mine.nonzero(as_tuple=True)
    src = table[dst[bi], ci].long()
    rank = ((src[:, None] == src) & (torch.arange(src.numel(), device=DEV) < torch.arange(src.numel(), device=DEV)[:, None])).sum(1)
    move = rank < refs[src] - 1
    src, bi, ci = src[move], bi[move], ci[move]
    new = (refs == 0).nonzero()[: src.numel(), 0]
    refs.index_add_(0, src, -one.expand(src.numel()))
    refs[new] = 1
    table[dst[bi], ci] = new.to(torch.int32)
    s["pairs"][: src.numel()] = torch.stack([src, new], 1).to(torch.int32)
    s["n_pairs"].fill_(src.numel())
    s["status"].zero_()
    _plain_copy(s, src, new)


def _plain_compact(s):
    s["table"].copy_(s["table0"])
    s["refs"].copy_(s["refs0"])
    table, refs = s["table"], s["refs"]
    used = refs > 0
    n_live = int(used.sum())
    idx = torch.arange(refs.numel(), device=DEV)
    src = (used & (idx >= n_live)).nonzero()[:, 0]
    dst = (~used & (idx < n_live)).nonzero()[:, 0]
    remap = torch.where(used, idx, -1).to(torch.int32)
    remap[src] = dst.to(torch.int32)
    s["remap"].copy_(remap)
    refs[dst] = refs[src]
    refs[src] = 0
    table.copy_(torch.where(table >= 0, remap[table.clamp(min=0).long()], -1))
    s["pairs"][: src.numel()] = torch.stack([src, dst], 1).to(torch.int32)
    s["n_pairs"].fill_(src.numel())
    _plain_copy(s, src, dst)


_PLAIN = dict(store=_plain_store, update=_plain_update, attend=_plain_attention, sparse=_plain_sparse,
              fork=_plain_fork, compact=_plain_compact)


def run(state):
    s = state
    if own:
        _run_own(s)
    else:
        _PLAIN[s["kind"]](s)
    kind = s["kind"]
    if kind in ("attend", "sparse"):
        return {"O": s["O"]}
    if kind in ("store", "update"):
        return {"K": s["outK"], "V": s["outV"], "k_scale": s["ks"], "v_scale": s["vs"]}
    out = {"k": s["k"], "v": s["v"], "k_scale": s["ks"], "v_scale": s["vs"], "table": s["table"], "refs": s["refs"],
           "n_pairs": s["n_pairs"]}
    return dict(out, held=s["held_v"], status=s["status"]) if kind == "fork" else dict(out, remap=s["remap"])


# --------------------------------------------------------------------------- work
def work(case):
    c = case
    d, page = c["d"], c["page"]
    if c["kind"] == "store":
        # bf16 in, codes out; codes in, bf16 out; for an average sequence of half of L (the first has all of it)
        n = c["n_mat"] * c["Hkv"] * d * _positions(c)
        return {"bytes": 2.0 * n * (2 + 1 + 1 + 2), "flops": 0}
    if c["kind"] == "update":
        # the rows in, the pages that they fall in out and in again, the window's bf16 rows out
        n = c["n_mat"] * c["B"] * c["Hkv"] * d
        rows = n * min(c["cap"], c["L"]) * 0.75
        window = n * min(c["L"], c["cap"] + c["cap"] // 2)
        return {"bytes": 2.0 * (2 * rows + window + window + 2 * window), "flops": 0}
    if c["kind"] == "attend":
        n = c["Hkv"] * _positions(c)
        q = c["B"] * c["Hq"] * c["qcap"] * d
        rows = c["Hq"] // c["Hkv"] * c["qcap"]
        return {"bytes": 2.0 * n * (d + 4.0 / page) + 4.0 * q, "flops": 4.0 * n * rows * d}
    if c["kind"] == "sparse":
        nb = max(1, (c["L"] - c["G"]) // page)
        n = c["B"] * c["Hkv"] * (min(c["C"], nb) * page + c["G"] + c["S"])
        q = c["B"] * c["Hq"] * c["qcap"] * d
        rows = c["Hq"] // c["Hkv"] * c["qcap"]
        return {"bytes": 2.0 * n * (d + 4.0 / page) + 4.0 * q, "flops": 4.0 * n * rows * d}
    one = 2.0 * c["n_mat"] * c["Hkv"] * (page * d + 4)                 # a page's codes and scales
    if c["kind"] == "fork":
        return {"bytes": 2 * one * c["n"] * c["own"] + 8.0 * c["n_pages"], "flops": 0}
    live = max(1, int(0.4 * c["n_pages"]))
    return {"bytes": 2 * one * live * 0.6 + 16.0 * c["n_pages"], "flops": 0}


def _positions(c):
    """Cached positions of all sequences: the first holds L, the others half of it on average, one of three or more none."""
    return c["L"] * (1 + 0.5 * (c["B"] - (2 if c["B"] > 2 else 1)))


# --------------------------------------------------------------------------- from the definition, in 64 bits
def _top_of(fmt):
    return 448.0 if fmt == "e4m3" else 127.0


def _nearest(x, scale, fmt):
    """The values that codes of x stand for: x / scale (rounded to fp32, as the definition has it) to the nearest
    code, ties to even, times the scale; float64 in and out."""
    safe = torch.where(scale == 0, torch.ones_like(scale), scale)
    y = (x / safe).float().double()
    if fmt == "int8":
        y = torch.round(y)
    else:
        # e4m3: 3 bits behind the leading one, exponents down to -6, steps of 2^-9 below
        e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -9))).clamp_min(-6.0)
        e = torch.where(y.abs() >= torch.exp2(e + 1), e + 1, e)
        step = torch.exp2(e - 3)
        y = torch.round(y / step) * step
    return torch.where(scale == 0, torch.zeros_like(y), y) * scale


def _exact_store(s):
    out = []
    for x, ks in ((s["K"], s["ks"]), (s["V"], s["vs"])):
        vals, scales = torch.zeros(x.shape, device=DEV, dtype=torch.float64), ks.double()
        for b, n in enumerate(s["lens"].tolist()):
            for j in range(-(-n // s["page"])):
                lo, hi = j * s["page"], min(n, (j + 1) * s["page"])
                rows = x[:, b, :, lo:hi].double()
                sc = (rows.abs().amax((-1, -2)) / _top_of(s["fmt"])).float().double()
                vals[:, b, :, lo:hi] = _nearest(rows, sc[..., None, None], s["fmt"])
                scales[:, int(s["table"][b, j])] = sc
        out.append((vals, scales))
    return {"K": out[0][0], "V": out[1][0], "k_scale": out[0][1], "v_scale": out[1][1]}


def _exact_update(s):
    page, fmt, start = s["page"], s["fmt"], s["start"]
    out = []
    for x, code, ks in ((s["K_rows"], s["k"], s["ks"]), (s["V_rows"], s["v"], s["vs"])):
        scales = ks.double()
        vals = torch.zeros(s["outK"].shape, device=DEV, dtype=torch.float64)
        for b, had in enumerate(s["lens"].tolist()):
            rows = s["rows"][b, : int(s["n_rows"][b])].tolist()
            after = int(s["after"][b])
            for j in range(start // page, s["table"].shape[1]):
                p = int(s["table"][b, j])
                mine = [(i, r) for i, r in enumerate(rows) if r // page == j]
                old_s = scales[:, p].clone()
                now = code[:, p].double() * old_s[..., None, None]      # [n, H, page, d]
                if mine:
                    new = x[:, b, :, [i for i, _ in mine]].double()
                    sc = (new.abs().amax((-1, -2)) / _top_of(fmt)).float().double()
                    if j * page < had:
                        sc = torch.maximum(sc, old_s)
                        grown = (sc > old_s)[..., None, None]
                        now = torch.where(grown, _nearest(now.float().double(), sc[..., None, None], fmt), now)
                    scales[:, p] = sc
                    now[:, :, [r % page for _, r in mine]] = _nearest(new, sc[..., None, None], fmt)
                for r in range(page):
                    t = j * page + r
                    if t < after and 0 <= t - start < vals.shape[3]:
                        vals[:, b, :, t - start] = now[:, :, r]
        out.append((vals, scales))
    return {"K": out[0][0], "V": out[1][0], "k_scale": out[0][1], "v_scale": out[1][1]}


def _exact_attention(s):
    page, g = s["page"], s["Hq"] // s["Hkv"]
    O = torch.zeros(s["O"].shape, device=DEV, dtype=torch.float64)
    for b in range(s["B"]):
        n = int(s["n_q"][b])
        for h in range(s["Hkv"]):
            if s["kind"] == "attend":
                keys = torch.arange(int(s["lens"][b]), device=DEV)
            else:
                P, g0 = int(s["P"][b]), int(s["g0"][b])
                want = set(range(g0, g0 + s["Gn"]))
                for j in s["blocks"][b, h].tolist():
                    if j >= 0:
                        want |= set(range(j * page, min(P, (j + 1) * page)))
                if s["sinks"] is not None:
                    want |= set(s["sinks"][b, h].tolist())
                keys = torch.tensor(sorted(want), device=DEV)
            if not keys.numel():
                continue
            phys, row = s["table"][b].long()[keys // page], keys % page
            K = s["k"][0].view(torch.uint8)[phys, h, row].view(s["k"].dtype).double() * s["ks"][0][phys, h].double()[:, None]
            V = s["v"][0].view(torch.uint8)[phys, h, row].view(s["v"].dtype).double() * s["vs"][0][phys, h].double()[:, None]
            q = s["Q"][b, h * g:(h + 1) * g, :n].double()
            w = torch.softmax(torch.einsum("had,kd->hak", q, K) * (s["d"] ** -0.5), -1)
            O[b, h * g:(h + 1) * g, :n] = torch.einsum("hak,kd->had", w, V)
    return {"O": O}


def exact(case, seed):
    s = prepare(case, seed)
    if s["kind"] == "store":
        return _exact_store(s)
    if s["kind"] == "update":
        return _exact_update(s)
    if s["kind"] in ("attend", "sparse"):
        return _exact_attention(s)
    return None
