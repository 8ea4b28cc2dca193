"""Plain numpy oracle of the 8-bit paged cache: its codes, its attention in float64, its pages.

Written from the definitions in include/focus.h; shares no code with the CUDA path. Codes are
uint8 arrays (the raw bytes of an e4m3 or int8 code), scales float32, as they lie in memory.
"""
import numpy as np

E4M3, INT8 = "e4m3", "int8"
TOP = {E4M3: np.float32(448.0), INT8: np.float32(127.0)}


def _e4m3_table():
    """Value of every e4m3 byte: 1 sign, 4 exponent (bias 7), 3 mantissa bits; 0x7f / 0xff are NaN."""
    v = np.zeros(256, dtype=np.float64)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m / 8.0 * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
        v[c] = np.nan if (c & 0x7F) == 0x7F else (-x if c & 0x80 else x)
    return v


E4M3_VALUES = _e4m3_table()


def code_values(codes, fmt):
    """Float64 values of raw code bytes (without the scale)."""
    codes = np.asarray(codes, dtype=np.uint8)
    return codes.view(np.int8).astype(np.float64) if fmt == INT8 else E4M3_VALUES[codes]


def nearest_codes(y, fmt):
    """Bytes of the codes nearest to y (float32), ties to the even code, out of range to the largest."""
    y = np.asarray(y, dtype=np.float32).astype(np.float64)
    if fmt == INT8:
        return np.clip(np.rint(y), -127, 127).astype(np.int8).view(np.uint8)
    grid = E4M3_VALUES[:127]                       # 0 .. 448 in steps, ascending; index = code
    a = np.minimum(np.abs(y), 448.0)
    hi = np.clip(np.searchsorted(grid, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - a, a - grid[lo]
    pick = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (pick | np.where(np.signbit(y), 0x80, 0)).astype(np.uint8)


def encode(x, scale, fmt):
    """Codes of float32 x under float32 scale (broadcast): nearest to the float32 quotient."""
    x, scale = np.broadcast_arrays(np.asarray(x, np.float32), np.asarray(scale, np.float32))
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(scale == 0, np.float32(0), x / scale)
    return np.where(scale == 0, np.uint8(0), nearest_codes(y, fmt)).astype(np.uint8)


def page_scale(rows, fmt):
    """s = max|x| / top over the last two axes, in float32."""
    return (np.abs(np.asarray(rows, np.float32)).max(axis=(-1, -2)) / TOP[fmt]).astype(np.float32)


def store(X, codes, scales, table, lens, fmt):
    """X [n_mat, B, H, L, d] float32 into codes [n_mat, n_pages, H, page, d], scales (in place)."""
    page = codes.shape[3]
    for b in range(X.shape[1]):
        n = min(int(lens[b]), X.shape[3])
        for j in range(-(-max(n, 0) // page)):
            rows = X[:, b, :, j * page:min(n, (j + 1) * page)]
            s = page_scale(rows, fmt)
            codes[:, table[b, j], :, :rows.shape[2]] = encode(rows, s[..., None, None], fmt)
            scales[:, table[b, j]] = s


def scatter_rows(X_rows, rows, n_rows, codes, scales, table, lens, fmt):
    """Replaces single rows (in place); see focus_cache_scatter_rows."""
    page = codes.shape[3]
    for b in range(X_rows.shape[1]):
        last = {}                                   # position -> listed row, the last one listed
        for i in range(int(n_rows[b])):
            r = int(rows[b, i])
            if 0 <= r < table.shape[1] * page:
                last[r] = i
        for j in sorted({r // page for r in last}):
            p, mine = table[b, j], {r % page: i for r, i in last.items() if r // page == j}
            at, idx = list(mine), list(mine.values())
            new = X_rows[:, b, :, idx].transpose(1, 2, 0, 3)
            s = page_scale(new, fmt)
            if j * page < lens[b]:
                old = scales[:, p].copy()
                s = np.maximum(s, old)
                held = [r for r in range(page) if j * page + r < lens[b] and r not in mine]
                if held:
                    was = codes[:, p][:, :, held]
                    x = (code_values(was, fmt).astype(np.float32) * old[..., None, None]).astype(np.float32)
                    again = encode(x, s[..., None, None], fmt)
                    tmp = codes[:, p]
                    tmp[:, :, held] = np.where((s > old)[..., None, None], again, was)
                    codes[:, p] = tmp
            tmp = codes[:, p]
            tmp[:, :, at] = encode(new, s[..., None, None], fmt)
            codes[:, p] = tmp
            scales[:, p] = s


def values(codes, scales, table_row, positions, h, fmt, m=0):
    """Float64 rows of the given positions of one sequence and head."""
    positions = np.asarray(positions, dtype=np.int64)
    page = codes.shape[3]
    p = np.asarray(table_row)[positions // page]
    return code_values(codes[m, p, h, positions % page], fmt) * scales[m, p, h].astype(np.float64)[:, None]


def key_set(P, g0, G, sinks, blocks, page):
    """Sorted positions of sinks U kept blocks (cut at P) U [g0, g0 + G)."""
    want = set(range(g0, g0 + G))
    for j in blocks:
        if j >= 0:
            want |= set(range(int(j) * page, min(P, (int(j) + 1) * page)))
    want |= {int(s) for s in sinks if s >= 0}
    return sorted(want)


def attention_rows(q, K, V, scale):
    """softmax(scale q K^T) V in float64 and what an error bound needs: (o, |v| mean under p,
    sum |v| over sum of p relative to its largest, largest |score| error per unit of q and k)."""
    if K.shape[0] == 0:
        z = np.zeros((q.shape[0], V.shape[1]))
        return z, z, z, np.zeros((q.shape[0], 1))
    t = scale * (q @ K.T)
    p = np.exp(t - t.max(axis=1, keepdims=True))
    l = p.sum(axis=1, keepdims=True)
    spread = abs(scale) * np.abs(q).max(axis=1, keepdims=True) * np.abs(K).sum(axis=1).max()
    return p @ V / l, p @ np.abs(V) / l, np.abs(V).sum(axis=0)[None] / l, spread


# ----------------------------------------------------------------------------- pages
class PageOracle:
    """refs, table, held as python lists; the same operations, one entry after another."""

    def __init__(self, n_pages, n_seq, cols):
        self.refs = [0] * n_pages
        self.table = [[-1] * cols for _ in range(n_seq)]
        self.held = [0] * n_seq
        self.cols = cols

    def _free(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def reserve(self, seqs, want):
        need, held = [], list(self.held)
        for s, w in zip(seqs, want):
            if 0 <= s < len(held) and w <= self.cols and w > held[s]:
                need += [(s, j) for j in range(held[s], w)]
                held[s] = w
        free = self._free()
        if len(need) > len(free):
            return len(need) - len(free)
        for (s, j), p in zip(need, free):
            self.table[s][j] = p
            self.refs[p] = 1
        self.held = held
        return 0

    def fork(self, src, dst, keep):
        for s, t, k in zip(src, dst, keep):
            if not (0 <= s < len(self.held) and 0 <= t < len(self.held)) or s == t or self.held[t]:
                continue
            k = max(0, min(k, self.held[s]))
            self.table[t][:k] = self.table[s][:k]
            for p in self.table[s][:k]:
                self.refs[p] += 1
            self.held[t] = k

    def own(self, seqs, first, last, pair_cap):
        refs, todo, seen = list(self.refs), [], set()
        for s, a, b in zip(seqs, first, last):
            if not 0 <= s < len(self.held):
                continue
            for j in range(max(0, a), min(b, self.held[s])):
                p = self.table[s][j]
                if (s, j) not in seen and refs[p] > 1:
                    refs[p] -= 1
                    todo.append((s, j, p))
                seen.add((s, j))
        free = self._free()
        room = min(len(free), pair_cap)
        if len(todo) > room:
            return len(todo) - room, []
        self.refs, pairs = refs, []
        for (s, j, p), f in zip(todo, free):
            self.table[s][j] = f
            self.refs[f] = 1
            pairs.append((p, f))
        return 0, pairs

    def release(self, seqs, keep):
        for s, k in zip(seqs, keep):
            if not 0 <= s < len(self.held):
                continue
            for j in range(max(0, k), self.held[s]):
                self.refs[self.table[s][j]] -= 1
                self.table[s][j] = -1
            self.held[s] = min(self.held[s], max(0, k))

    def compact(self):
        live = [p for p, r in enumerate(self.refs) if r > 0]
        n = len(live)
        pairs = list(zip([p for p in live if p >= n], [p for p in range(n) if self.refs[p] == 0]))
        remap = [p if r > 0 else -1 for p, r in enumerate(self.refs)]
        for a, b in pairs:
            remap[a] = b
            self.refs[b], self.refs[a] = self.refs[a], 0
        for s, h in enumerate(self.held):
            self.table[s][:h] = [remap[p] for p in self.table[s][:h]]
        return pairs, remap
