"""Shared helpers of the paged-cache GPU tests: random caches on both sides, and tolerances."""
import numpy as np
import torch

import dequant_gemv_q4g32_amd as qg
from oracle import paged


def random_cache(kind, layers, pages, heads, dim, tokens, seed, poison=False):
    """An oracle cache of plausible entries. poison: every byte random instead (NaN and infinite
    scales and values among them), for places that nothing may read."""
    rng = np.random.default_rng(seed)
    c = paged.Cache(kind, layers, pages, heads, dim, tokens)
    if poison:
        for a in c._arrays:
            a.view(np.uint8)[...] = rng.choice(np.array([0x00, 0x7C, 0x7E, 0xFC, 0xFF, 0x55], np.uint8), a.view(np.uint8).shape)
    elif kind == "q8":
        for a in c.codes:
            a[...] = rng.integers(-127, 128, a.shape)
        for a in c.scales:
            a[...] = np.abs(rng.standard_normal(a.shape)) * 0.02 + 1e-4
    else:
        for a in c.values:
            a[...] = rng.standard_normal(a.shape)
    return c


def random_table(rng, lens, tokens, pages, width):
    """Distinct pages in random order for every sequence, -1 beyond its length."""
    order = rng.permutation(pages)
    table = np.full((len(lens), width), -1, np.int32)
    at = 0
    for i, n in enumerate(lens):
        need = -(-max(0, int(n)) // tokens)
        table[i, :need] = order[at:at + need]
        at += need
    return table


def upload(c, layers_dim=True):
    p = c.pack()
    return qg.KVPool(torch.from_numpy(p if layers_dim else p[0]).cuda(), c.kind, c.heads, c.dim, c.tokens)


def download(c, pool):
    """The pool's contents as an oracle cache of c's shape."""
    return paged.Cache(c.kind, c.layers, c.pages, c.heads, c.dim, c.tokens).unpack(
        pool.pages.cpu().numpy().reshape(c.layers, c.pages, -1))


def assert_same_bytes(a, b, what=""):
    for i, (x, y) in enumerate(zip(a._arrays, b._arrays)):
        same = x.view(np.uint8) == y.view(np.uint8)
        assert same.all(), f"{what}: array {i} differs at {np.argwhere(~same)[:4].tolist()}"


def dev(x, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=dtype)).cuda()


def attention_tolerance(out, lse, bound, reach, tokens, dim, f32):
    """How far (out, lse) may be from the oracle's, from the arithmetic alone.

    Half a step of fp32 is e = 2^-24. A score is a sum of dim products in fp32 (exact fp16
    factors; any order), times the scale, times log2(e) (a constant and a product): off by at most
    (dim + 4) e * reach, reach = scale sum |q k|. An exponential of it carries that as its relative
    error, the reference maximum's subtraction another e of the score's size, and the exponential
    itself 2^-22. Weights as pairs of fp16 numbers: 2^-22 relative, 2^-31 of the largest weight where
    that is more (below fp16's normal range). Sums over the tokens: tokens * e. The numerator and the
    denominator both carry all of it, hence the factor 2; fp16 output adds half a step of its own.
    lse = the denominator's relative error, plus its logarithm and the final sum (4 e of |lse| and
    of reach)."""
    e = 2.0 ** -24
    score = (dim + 8) * e * reach
    rel = 2 * (score + 2.0 ** -21 + tokens * (e + 2.0 ** -30))
    tol = rel[..., None] * bound + 1e-30
    if not f32:
        tol = tol + np.abs(out) * 2.0 ** -11 + 2.0 ** -25
    with np.errstate(invalid="ignore"):
        size = np.where(np.isfinite(lse), np.abs(lse), 0.0)
    return tol, rel + 4 * e * (size + reach) + 4 * e


def check_attention(got, got_lse, ref, tokens, dim):
    out, lse, bound, reach = ref
    f32 = got.dtype == torch.float32
    tol, tol_lse = attention_tolerance(out, lse, bound, reach, tokens, dim, f32)
    g, gl = got.cpu().double().numpy(), got_lse.cpu().double().numpy()
    bad = ~(np.abs(g - out) <= tol)
    assert not bad.any(), (f"out: {int(bad.sum())} of {bad.size}, first {np.argwhere(bad)[0].tolist()}: got {g[bad][0]:.8g} "
                           f"want {out[bad][0]:.8g} tolerance {tol[bad][0]:.3g}")
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(gl), empty)
    bad = ~(np.abs(np.where(empty, 0, gl) - np.where(empty, 0, lse)) <= tol_lse)
    assert not bad.any(), f"lse: {np.argwhere(bad)[0].tolist()}: got {gl[bad][0]:.9g} want {lse[bad][0]:.9g} tolerance {tol_lse[bad][0]:.3g}"
