"""Paged key-value cache, by definition: plain loops over NumPy arrays, attention in fp64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

A `Cache` holds, for every layer, page and KV head, the codes and scales (kind "q8", the codec of
oracle/kvcache.py) or the fp16 values ("f16") of T tokens, as separate arrays indexed [layer][page]
[head][token]; `pack` and `unpack` convert to and from the page records of include/qgemv.h:
  q8   K codes int8 [T][D], V codes int8 [T][D], K scales fp16 [T][D/32], V scales fp16 [D/32][T]
  f16  K fp16 [T][D], V fp16 [T][D]
for each head in turn. Table entries outside [0, pages) name no page.

Parity status: the codec is pinned by tests/test_oracle_kvcache.py; the attention formula and the
page operations are definitions of this repository (parity unpinned), checked by hand-worked cases
in tests/test_oracle_paged.py.
"""
from __future__ import annotations

import numpy as np

from . import kvcache

GROUP = kvcache.GROUP


class Cache:
    def __init__(self, kind: str, layers: int, pages: int, heads: int, dim: int, tokens: int):
        self.kind, self.layers, self.pages, self.heads, self.dim, self.tokens = kind, layers, pages, heads, dim, tokens
        shape = (layers, pages, heads, tokens)
        if kind == "q8":
            self.codes = [np.zeros(shape + (dim,), np.int8) for _ in range(2)]
            self.scales = [np.zeros(shape + (dim // GROUP,), np.float16) for _ in range(2)]
        else:
            self.values = [np.zeros(shape + (dim,), np.float16) for _ in range(2)]

    @property
    def _arrays(self):
        return self.codes + self.scales if self.kind == "q8" else self.values

    def pack(self) -> np.ndarray:
        """uint8 [layers, pages, page bytes]."""
        flat = lambda a: a.reshape(self.layers, self.pages, self.heads, -1).view(np.uint8)
        if self.kind == "q8":
            vs = np.ascontiguousarray(np.swapaxes(self.scales[1], -1, -2))
            parts = [flat(self.codes[0]), flat(self.codes[1]), flat(self.scales[0]), flat(vs)]
        else:
            parts = [flat(v) for v in self.values]
        return np.concatenate(parts, axis=-1).reshape(self.layers, self.pages, -1)

    def unpack(self, pool: np.ndarray) -> "Cache":
        """Take the contents of a packed pool."""
        t, d, g = self.tokens, self.dim, self.dim // GROUP
        p = pool.reshape(self.layers, self.pages, self.heads, -1)
        take = lambda a, b, dt, shape: np.ascontiguousarray(p[..., a:b]).view(dt).reshape(p.shape[:3] + shape).copy()
        if self.kind == "q8":
            self.codes = [take(0, t * d, np.int8, (t, d)), take(t * d, 2 * t * d, np.int8, (t, d))]
            at = 2 * t * d
            self.scales = [take(at, at + 2 * t * g, np.float16, (t, g)),
                           np.swapaxes(take(at + 2 * t * g, at + 4 * t * g, np.float16, (g, t)), -1, -2).copy()]
        else:
            self.values = [take(0, 2 * t * d, np.float16, (t, d)), take(2 * t * d, 4 * t * d, np.float16, (t, d))]
        return self

    def place(self, table, seq, pos):
        """(page, offset) of a token, or None."""
        if not (0 <= seq < table.shape[0]) or pos < 0 or pos // self.tokens >= table.shape[1]:
            return None
        page = int(table[seq, pos // self.tokens])
        return (page, pos % self.tokens) if 0 <= page < self.pages else None

    def append(self, layer, table, k, v, positions, seqs=None):
        for i, pos in enumerate(positions):
            at = self.place(table, i if seqs is None else int(seqs[i]), int(pos))
            if at is None:
                continue
            for which, x in ((0, k), (1, v)):
                x = np.asarray(x[i], np.float16).reshape(self.heads, self.dim)
                if self.kind == "q8":
                    q, d = kvcache.quantize(x)
                    self.codes[which][layer, at[0], :, at[1]] = q
                    self.scales[which][layer, at[0], :, at[1]] = d
                else:
                    self.values[which][layer, at[0], :, at[1]] = x

    def token(self, layer, which, page, off):
        """fp16 [heads, dim]: a cached token's values."""
        if self.kind == "q8":
            return kvcache.dequantize_fp16(self.codes[which][layer, page, :, off], self.scales[which][layer, page, :, off])
        return self.values[which][layer, page, :, off]

    def gather(self, layer, table, positions, seqs=None):
        out = np.zeros((2, len(positions), self.heads, self.dim), np.float16)
        for i, pos in enumerate(positions):
            at = self.place(table, i if seqs is None else int(seqs[i]), int(pos))
            if at is not None:
                for which in (0, 1):
                    out[which, i] = self.token(layer, which, *at)
        return out.reshape(2, len(positions), -1)

    def copy_page(self, src, dst):
        for a in self._arrays:
            a[:, dst] = a[:, src]


def attention(cache: Cache, layer, q, table, lens, max_len, scale, window=0):
    """(out, lse, bound, reach), all fp64 [batch, heads(, dim)]: bound = sum_j w_j |v_j| for each output, reach =
    the largest scale * sum |q k| of a head's tokens (the size of its scores' terms)."""
    batch, heads, dim = q.shape
    group = heads // cache.heads
    out, bound = np.zeros((2, batch, heads, dim))
    lse, reach = np.full((batch, heads), -np.inf), np.zeros((batch, heads))
    for b in range(batch):
        n = min(max(int(lens[b]), 0), max_len)
        toks = [cache.place(table, b, j) for j in range(max(0, n - window) if window else 0, n)]
        toks = [t for t in toks if t is not None]
        if not toks:
            continue
        k, v = (np.stack([cache.token(layer, which, *t) for t in toks]).astype(np.float64) for which in (0, 1))
        for h in range(heads):
            kh, vh, x = k[:, h // group], v[:, h // group], q[b, h].astype(np.float64)
            s = scale * (kh @ x)
            m = s.max()
            w = np.exp(s - m)
            out[b, h] = (w @ vh) / w.sum()
            bound[b, h] = (w @ np.abs(vh)) / w.sum()
            lse[b, h] = m + np.log(w.sum())
            reach[b, h] = (abs(scale) * (np.abs(kh) @ np.abs(x))).max()
    return out, lse, bound, reach


def fork(cache, table, lens, refs, src_rows, dst_rows, new_pages):
    """In place. Forks are decided on the rows as they are before the call."""
    sources = set(int(s) for s in src_rows)
    for i, (s, d, fresh) in enumerate(zip(src_rows, dst_rows, new_pages)):
        if not (0 <= s < len(lens) and 0 <= d < len(lens)) or int(d) in sources or d in dst_rows[:i]:
            continue
        n = min(max(int(lens[s]), 0), table.shape[1] * cache.tokens)
        whole, rest = divmod(n, cache.tokens)
        tail = int(table[s, whole]) if rest else -1
        copied = 0 <= tail < cache.pages                  # a last page that is partly filled, and is a page
        if copied and (not 0 <= fresh < cache.pages or fresh in new_pages[:i]):
            continue
        row = np.full(table.shape[1], -1, table.dtype)
        row[:whole] = table[s, :whole]
        for e in row[:whole]:
            if 0 <= e < cache.pages:
                refs[e] += 1
        if copied:
            cache.copy_page(tail, fresh)
            row[whole] = fresh
            refs[fresh] = 1
        elif rest:
            row[whole] = tail                             # no page there, as in the source
        table[d] = row
        lens[d] = n


def free(cache, table, lens, refs, rows):
    for r in rows:
        if not 0 <= r < len(lens) or lens[r] <= 0:
            continue
        for e in table[r, :-(-int(lens[r]) // cache.tokens)]:
            if 0 <= e < cache.pages:
                refs[e] -= 1
        table[r] = -1
        lens[r] = 0


def compact(cache, table, refs):
    """(table_out, refs_out, remap, live); pages move in place."""
    held = [p for p in range(cache.pages) if refs[p] > 0]
    live = len(held)
    remap = np.full(cache.pages, -1, np.int32)
    remap[held] = held
    hollow = [p for p in range(live) if refs[p] <= 0]
    for dst, src in zip(hollow, [p for p in held if p >= live]):
        cache.copy_page(src, dst)
        remap[src] = dst
    refs_out = np.zeros_like(refs)
    for p in held:
        refs_out[remap[p]] = refs[p]
    table_out = np.full_like(table, -1)
    ok = (table >= 0) & (table < cache.pages)
    table_out[ok] = remap[table[ok]]
    return table_out, refs_out, remap, live
