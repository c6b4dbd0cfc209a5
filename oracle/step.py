"""What a decode step does round the paged cache, by definition: places for its tokens (extend, trim), the
norm and rotation of queries and keys, and their frequencies. Plain loops over NumPy arrays, fp64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

The attention over shared prefixes is `paged.attention`: sharing changes how it is computed, not what.

Parity status: definitions of this repository (parity unpinned), checked by hand-worked cases and
invariants in tests/test_oracle_step.py.
"""
from __future__ import annotations

import math

import numpy as np


def trim(table, lens, refs, to, tokens):
    """In place."""
    for r in range(len(lens)):
        n = min(int(lens[r]), table.shape[1] * tokens)
        if not 0 <= to[r] < n:
            continue
        for j in range(-(-int(to[r]) // tokens), -(-n // tokens)):
            if 0 <= table[r, j] < len(refs):
                refs[table[r, j]] -= 1
            table[r, j] = -1
        lens[r] = to[r]


def extend(table, lens, refs, add, slots, tokens):
    """In place; (granted, starts, seqs, positions). Rows are served one after the other."""
    rows, width = table.shape
    granted, starts = np.zeros(rows, np.int32), np.zeros(rows + 1, np.int32)
    seqs, positions = np.full((2, slots), -1, np.int32)
    free = [p for p in range(len(refs)) if refs[p] <= 0]
    given = taken = asked = 0                          # pages asked for (whether given or not), given, and tokens asked for
    before = refs.copy()
    for r in range(rows):
        n, at = max(int(add[r]), 0), asked
        starts[r] = min(at, slots)
        asked += n
        starts[r + 1] = min(asked, slots)
        length = min(max(int(lens[r]), 0), width * tokens)
        if n == 0 or asked > slots or length + n > width * tokens:
            continue
        if length % tokens:
            last = table[r, length // tokens]
            if not 0 <= last < len(refs) or before[last] != 1:
                continue
        first, end = -(-length // tokens), -(-(length + n) // tokens)
        given += end - first
        if end > first and given > len(free):
            continue
        for j in range(first, end):
            table[r, j] = free[taken]
            refs[free[taken]] = 1
            taken += 1
        lens[r] = length + n
        granted[r] = n
        seqs[at:at + n] = r
        positions[at:at + n] = range(length, length + n)
    return granted, starts, seqs, positions


def rotate(x, position, freqs, interleaved=False, weight=None, eps=0.0, factor=1.0):
    """A head x [D] in fp64, normed if there is a weight, then its first 2 * len(freqs) elements rotated."""
    y = np.asarray(x, np.float64).copy()
    if weight is not None:
        y = y / math.sqrt(float(np.mean(y * y)) + eps) * np.asarray(weight, np.float64)
    out = y.copy()
    half = len(freqs)
    for j in range(half):
        i, k = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        t = float(position) * float(freqs[j])
        out[i] = factor * (y[i] * math.cos(t) - y[k] * math.sin(t))
        out[k] = factor * (y[k] * math.cos(t) + y[i] * math.sin(t))
    return out


def freqs(kind, dim, base, scale=1.0, context=0.0, low=0.0, high=0.0):
    """Radians a token of pair j < dim / 2."""
    if kind == "base":
        base = base * scale ** (dim / (dim - 2))
    out = []
    for j in range(dim // 2):
        f = base ** (-2 * j / dim)
        slow = {"plain": 0.0, "base": 0.0, "linear": 1.0}.get(kind)
        if kind == "turns":
            turns = context * f / (2 * math.pi)
            slow = 1 - (turns - low) / (high - low)
        if kind == "parts":
            a = max(0, math.floor(dim * math.log(context / (high * 2 * math.pi)) / (2 * math.log(base))))
            b = min(dim - 1, math.ceil(dim * math.log(context / (low * 2 * math.pi)) / (2 * math.log(base))))
            slow = (j - a) / max(b - a, 0.001)
        slow = min(1.0, max(0.0, slow))
        out.append(f * (1 - slow) + f / scale * slow)
    return np.array(out)
