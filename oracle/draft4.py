"""Float64 CPU oracle of a draft held in 4 bits: the cache's rows, the attention over
them with a sliding window and sinks, products with 4-bit weights, and the moves of
cache pages.

TEST INFRASTRUCTURE, NOT PRODUCT CODE (see ``oracle/__init__.py``).  Arrays are float64
(already widened from their storage type); it shares no code with the CUDA path.

Readings:
  R34 a row of D values is stored as s = bf16((max - min) / 15), m = min (a bf16 value
      already) and codes c = min(round((x - m) / s), 15), ties to even; s = 0 has codes 0.
      A row with a value that is not finite has s = m = NaN.  Its values are m + s c.
  R35 the query at position i has the own index p = L + i - 1 (the convention of R32); with
      a window w > 0 it sees the tokens j <= p with j > p - w or j < sinks.
  R36 shares[p] counts a page's block-table entries beyond the first.  A fork shares the
      full pages of L = seq_lens[src] tokens and copies the one that is partly full; the
      pages it needs come from the top of the free stack in the order of the forks.  Released
      pages go on the stack in descending order of their ids.
  R37 compaction with n pages in use moves the k-th lowest used id >= n to the k-th lowest
      unused id < n; the free stack is then num_pages - 1 .. n.
"""

from __future__ import annotations

import numpy as np

FLAG_CAPACITY = 64
FLAG_BAD_N = 256
FLAG_BAD_PAGE = 512


def bf16(v):
    """The nearest bf16 values (ties to even), subnormal ones too."""
    v = np.asarray(v, np.float64)
    step = np.ldexp(1.0, np.maximum(np.frexp(v)[1], -125) - 8)
    return np.rint(v / step) * step


def quantise(x):
    """(codes, s, m) of rows (the last axis)."""
    x = np.asarray(x, np.float64)
    fine = np.isfinite(x).all(-1)
    y = np.where(fine[..., None], x, 0.0)
    m = y.min(-1)
    s = bf16((y.max(-1) - m) / 15)
    q = np.rint((y - m[..., None]) / np.where(s > 0, s, 1.0)[..., None])
    codes = np.where(s[..., None] > 0, np.minimum(q, 15), 0).astype(np.uint8)
    return codes, np.where(fine, s, np.nan), np.where(fine, m, np.nan)


def head_bytes(D: int, page_size: int) -> int:
    return -(-page_size * (D + 8) // 16) * 16


def bf16_bits(v):
    return (np.asarray(v, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def write_token(pool, page: int, slot: int, page_size: int, k, v):
    """Store one token's keys and values [Hkv, D] into pool [pages, page_bytes] (uint8)."""
    H, D = k.shape
    hb = head_bytes(D, page_size)
    for h in range(H):
        for part, row in enumerate((k[h], v[h])):
            codes, s, m = quantise(row)
            at = h * hb + part * page_size * D // 2 + slot * D // 2
            pool[page, at:at + D // 2] = codes[0::2] | codes[1::2] << 4
            at = h * hb + page_size * D + part * page_size * 4 + slot * 4
            word = np.array([0x7fc0, 0x7fc0], np.uint16) if np.isnan(s) else bf16_bits([s, m])
            pool[page, at:at + 4] = word.view(np.uint8)


def read_tokens(pool, pages, page_size: int, n: int, Hkv: int, D: int):
    """(codes, s, m) of a sequence's first n tokens: [2, n, Hkv, D], [2, n, Hkv] twice."""
    hb = head_bytes(D, page_size)
    codes, s, m = np.zeros((2, n, Hkv, D)), np.zeros((2, n, Hkv)), np.zeros((2, n, Hkv))
    for t in range(n):
        page, slot = pool[int(pages[t // page_size])], t % page_size
        for h in range(Hkv):
            for part in range(2):
                at = h * hb + part * page_size * D // 2 + slot * D // 2
                raw = page[at:at + D // 2]
                codes[part, t, h, 0::2], codes[part, t, h, 1::2] = raw & 15, raw >> 4
                at = h * hb + page_size * D + part * page_size * 4 + slot * 4
                word = page[at:at + 4].copy().view(np.uint16).astype(np.uint32) << 16
                s[part, t, h], m[part, t, h] = word.view(np.float32)
    return codes, s, m


def visible(p: int, window: int, sinks: int):
    """The tokens that the query of own index p sees."""
    return [j for j in range(p + 1) if window <= 0 or j > p - window or j < sinks]


def attention(q, codes, s, m, length: int, scale: float, window: int = 0, sinks: int = 0):
    """One sequence: q [Q, Hq, D], its tokens as read_tokens gives them.  Returns out, lse and
    what bounds their rounding: coded [Q, Hq, D] = sum p s c, weight = sum p (|m| + s c), and
    spread [Q, Hq] = max_j |scale| sum |q| (s c + |m|)."""
    Q, Hq, D = q.shape
    Hkv = codes.shape[2]
    G = Hq // Hkv
    values = m[..., None] + s[..., None] * codes
    out, lse = np.zeros((Q, Hq, D)), np.full((Q, Hq), -np.inf)
    coded, weight, spread = np.zeros((Q, Hq, D)), np.zeros((Q, Hq, D)), np.zeros((Q, Hq))
    for i in range(Q):
        see = visible(length + i - 1, window, sinks)
        if not see:
            continue
        for hq in range(Hq):
            h = hq // G
            z = scale * (values[0, see, h] @ q[i, hq])
            top = z.max()
            if np.isneginf(top):
                continue
            p = np.exp(z - top)
            p /= (total := p.sum())
            out[i, hq] = p @ values[1, see, h]
            lse[i, hq] = top + np.log(total)
            sc = s[1, see, h][:, None] * codes[1, see, h]
            coded[i, hq] = p @ sc
            weight[i, hq] = p @ (sc + np.abs(m[1, see, h])[:, None])
            sk = s[0, see, h][:, None] * codes[0, see, h] + np.abs(m[0, see, h])[:, None]
            spread[i, hq] = abs(scale) * (sk @ np.abs(q[i, hq])).max()
    return out, lse, coded, weight, spread


def weights(W, scales, zeros, group: int):
    """[N, K] from bytes [N, K / 2], scales [N, K / group], zeros or None."""
    codes = np.zeros((W.shape[0], W.shape[1] * 2))
    codes[:, 0::2], codes[:, 1::2] = W & 15, W >> 4
    z = 8.0 if zeros is None else np.repeat(np.asarray(zeros, np.float64), group, 1)
    return (codes - z) * np.repeat(np.asarray(scales, np.float64), group, 1)


class Pages:
    """A pool's books as plain lists; ``data`` maps a page id to whatever it holds."""

    def __init__(self, table, lens, shares, stack, page_size: int, num_pages: int, data):
        self.table = [list(map(int, r)) for r in table]
        self.lens, self.shares, self.stack = list(map(int, lens)), list(map(int, shares)), list(map(int, stack))
        self.P, self.num_pages, self.data, self.flags = page_size, num_pages, list(data), 0

    def fork(self, src, dst):
        good = []
        for f, (s, d) in enumerate(zip(src, dst)):
            others = [x for g, x in enumerate(dst) if g != f]
            sources = [x for g, x in enumerate(src) if g != f]
            B = len(self.lens)
            if not (0 <= s < B and 0 <= d < B) or s == d or s in others or d in others or d in sources:
                self.flags |= FLAG_BAD_N
                continue
            L = self.lens[s]
            if not 0 <= L <= len(self.table[s]) * self.P or self.lens[d] != 0 or any(p >= 0 for p in self.table[d]):
                self.flags |= FLAG_BAD_N
                continue
            if any(not 0 <= p < self.num_pages for p in self.table[s][:-(-L // self.P)]):
                self.flags |= FLAG_BAD_PAGE
                continue
            good.append((s, d, L))
        need = sum(L % self.P > 0 for _, _, L in good)
        if need > len(self.stack):
            self.flags |= FLAG_CAPACITY
            return
        for s, d, L in good:
            full = L // self.P
            for j in range(full):
                self.table[d][j] = self.table[s][j]
                self.shares[self.table[s][j]] += 1
            if L % self.P:
                page = self.stack.pop()
                self.data[page] = self.data[self.table[s][full]]
                self.table[d][full] = page
            self.lens[d] = L

    def free(self, seqs):
        gone, done = [], set()
        for s in seqs:
            if not 0 <= s < len(self.lens) or s in done:
                self.flags |= FLAG_BAD_N
                continue
            done.add(s)
            for j, p in enumerate(self.table[s]):
                if p < 0:
                    continue
                self.table[s][j] = -1
                if p >= self.num_pages:
                    self.flags |= FLAG_BAD_PAGE
                elif p in gone:
                    self.flags |= FLAG_BAD_PAGE
                elif self.shares[p] == 0:
                    gone.append(p)
                else:
                    self.shares[p] -= 1
            self.lens[s] = 0
        self.stack += sorted(gone, reverse=True)

    def compact(self, prefix):
        used = sorted({p for r in self.table for p in r if 0 <= p < self.num_pages} | set(prefix))
        n = len(used)
        holes = [p for p in range(n) if p not in used]
        to = dict(zip([p for p in used if p >= n], holes))
        for p, q in to.items():
            self.data[q], self.shares[q], self.shares[p] = self.data[p], self.shares[p], 0
        self.table = [[to.get(p, p) for p in r] for r in self.table]
        self.stack = list(range(self.num_pages - 1, n - 1, -1))
        return [to.get(p, p) for p in prefix]
