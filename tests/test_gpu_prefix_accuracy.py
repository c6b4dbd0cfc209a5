"""GPU tests of how exactly attention over shared prefixes adds up: scores of any size, in each of the ways in which
shared tokens are read."""
import numpy as np
import pytest

import dequant_gemv_q4g32_amd as qg
from oracle import paged

from paged_util import attention_tolerance, dev, upload
from test_gpu_prefix_attention import starts_of

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# rows of the groups, heads, kv heads: one group of few workgroups' work, read together; enough groups that their tokens
# are read once for 16 query rows; and the same with 16 heads of a KV head, read for each row apart
WAYS = {"together": ([9, 5], 8, 2), "packs": ([2, 3, 4, 2, 5, 2, 3, 2, 4, 2], 32, 16), "apart": ([2, 3, 2, 2, 3, 2, 2, 2, 3, 2], 256, 16)}


def leveled_cache(kind, sizes, prefix, tails, kv_heads, dim, tokens, level, rng):
    """(oracle cache, table, lens, V of the first row of each group...) of groups whose first `prefix` tokens lie in shared
    pages. Token j of a row has K = (1025 - level(j)) * 8 in 16 of its elements and V of small multiples of 1/4; both exact
    in either kind of page."""
    lens = [prefix + tails[i % len(tails)] for i in range(sum(sizes))]
    width, shared = -(-max(lens) // tokens), prefix // tokens
    table, at, b = np.full((len(lens), width), -1, np.int32), 0, 0
    for size in sizes:
        for i in range(size):
            n = -(-lens[b] // tokens)
            first = shared if i else 0
            table[b, :first] = table[b - i, :first]
            table[b, first:n] = np.arange(at, at + n - first)
            at += n - first
            b += 1
    c = paged.Cache(kind, 1, at, kv_heads, dim, tokens)
    seen = set()
    some = np.arange(dim) % (dim // 16) == 0
    for b, n in enumerate(lens):
        for j in range(n):
            at = (0, table[b, j // tokens], slice(None), j % tokens)
            if at[1] * tokens + at[3] in seen:
                continue
            seen.add(at[1] * tokens + at[3])
            v = rng.integers(-8, 9, (kv_heads, dim))
            if kind == "f16":
                c.values[0][at], c.values[1][at] = some * 8 * (1025 - level[j]), v / 4
            else:
                c.codes[0][at], c.codes[1][at] = some * 64, v
                c.scales[0][at], c.scales[1][at] = (1025 - level[j]) / 8, 0.25
    return c, table, lens


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("kind,dim", [("f16", 64), ("f16", 128), ("f16", 256), ("q8", 64), ("q8", 128), ("q8", 256)])
@pytest.mark.parametrize("order", ["rising", "mixed"])
def test_large_scores(way, kind, dim, order):
    """Scores from 2^19 to 2^31 in units of log2, either sign, with a scale whose product with log2(e) has a full mantissa,
    and heads of ordinary scores between them. <q, k> is exact in fp32 in any order of its sum (35 * 2^a times 8 * 1025 or a bit
    less, 16 times: 21 bits), so tokens of one level have one and the same score; the next level is 2^-10 of it away, which is 2^9
    at least, far past fp32's rounding of the product: its weights are zero. So where scores are large the result is the mean
    of the highest level's V, and nothing but the weights' pairs and the sums may be in its error."""
    sizes, heads, kv_heads = WAYS[way]
    prefix, tails, tokens, scale = 160, [21, 3, 0, 40], 16, 0.3
    rng = np.random.default_rng(dim)
    level = rng.integers(0, 7, prefix + max(tails))
    if order == "rising":
        level = np.sort(level)[::-1]
    c, table, lens = leveled_cache(kind, sizes, prefix, tails, kv_heads, dim, tokens, level, rng)
    powers = np.array([10, 9, 8, 7, 6, 5, 4, 3, 2, 0, -2, -14])   # 35 * 2^10 * 8200 * 16 * 0.3 * log2(e) = 1.89 * 2^30
    which = (np.arange(len(lens))[:, None] * 5 + np.arange(heads)) % len(powers)
    sign = np.where(rng.random(which.shape) < 0.5, 1, -1)
    q = np.zeros((len(lens), heads, dim), np.float16)
    q[:, :, ::dim // 16] = (sign * 35.0 * 2.0 ** powers[which])[:, :, None]
    out, lse, bound, reach = paged.attention(c, 0, q, table, lens, max(lens), scale)
    large = powers[which] > -14
    args = [upload(c), dev(q, np.float16), dev(table), dev(lens), dev(starts_of(sizes)), dev([prefix] * len(sizes))]
    for f32 in (True, False):
        tol, _ = attention_tolerance(out, lse, bound, np.where(large, 0, reach), max(lens), dim, f32)
        tol = tol + max(lens) * 2.0 * 2.0 ** -31 + (0 if f32 else bound * 2.0 ** -11)
        _, tol_lse = attention_tolerance(out, lse, bound, reach, max(lens), dim, f32)
        got, got_lse = qg.prefix_attention(*args, max_tail=40, scale=scale, out_f32=f32, return_lse=True)
        got, got_lse = got.cpu().double().numpy(), got_lse.cpu().double().numpy()
        bad = ~(np.abs(got - out) <= tol).all(-1)
        assert not bad.any(), (f"{int(bad.sum())} heads, of q = 35 * 2^{sorted(set(powers[which][bad].tolist()))}: "
                               f"got {got[bad][0][:4]} want {out[bad][0][:4]}")
        assert (np.abs(got_lse - lse) <= tol_lse).all()


# scale * log2(e) is exactly 1 in fp32 with this scale, so scores in units of log2 are <q, k> itself
LN2 = float(np.float32(np.log(2.0)))


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("kind,dim", [("f16", 64), ("f16", 128), ("f16", 256), ("q8", 64), ("q8", 128), ("q8", 256)])
def test_weights_of_shared_tokens(way, kind, dim):
    """fp16 results whose terms all but cancel: token 2 i + 1 has the V of token 2 i times -2^(y(2 i) - y(2 i + 1)), rounded to
    fp16 (int8 pages: in its scale), with y the scores, which are exact multiples of 1/64. The sum is then some 2^-12 of its
    terms, so that its own rounding to fp16 hides nothing, and the weights have to be good to 22 bits: to 2 (2^-21 + tokens
    (2^-24 + 2^-30)) of the sum of their terms' sizes, as for the one-token attention, and 2^-31 of the sum of |V|."""
    sizes, heads, kv_heads = WAYS[way]
    tokens, prefix, rows = 16, 32, sum(WAYS[way][0])
    rng = np.random.default_rng(dim)
    groups = len(sizes)
    c = paged.Cache(kind, 1, groups * prefix // tokens, kv_heads, dim, tokens)
    table = np.repeat(np.arange(c.pages).reshape(groups, -1), sizes, axis=0).astype(np.int32)
    for g in range(groups):
        for kvh in range(kv_heads):
            y = rng.integers(0, 512, prefix) / 64          # 0 to 8
            v = rng.integers(-100, 101, dim).astype(np.float64)
            for j in range(prefix):
                at = (0, g * prefix // tokens + j // tokens, kvh, j % tokens)
                if j % 2 == 0:
                    v = rng.integers(-100, 101, dim).astype(np.float64)
                    code, step = v, 1 / 64
                else:
                    code, step = -v, np.float16(2.0 ** (y[j - 1] - y[j]) / 64)
                if kind == "f16":
                    c.values[0][at + (0,)], c.values[1][at] = y[j] * 4, (code * np.float64(2.0 ** (y[j - 1] - y[j]) if j % 2 else 1)) / 64
                else:
                    c.codes[0][at + (0,)], c.codes[1][at] = 64, code
                    c.scales[0][at + (0,)], c.scales[1][at] = y[j] * 4 / 64, step
    q = np.zeros((rows, heads, dim), np.float16)
    q[:, :, 0] = 0.25
    lens = [prefix] * rows
    out, lse, bound, reach = paged.attention(c, 0, q, table, lens, prefix, LN2)
    assert (np.abs(out) < 2.0 ** -8 * bound).all()         # they do cancel
    most = float(np.abs(c.values[1]).max() if kind == "f16" else 127 * c.scales[1].max())
    tol, _ = attention_tolerance(out, lse, bound, np.zeros_like(reach), prefix, dim, False)
    tol = tol + prefix * most * 2.0 ** -31
    got = qg.prefix_attention(upload(c), dev(q, np.float16), dev(table), dev(lens), dev(starts_of(sizes)), dev([prefix] * groups),
                              max_tail=0, scale=LN2).cpu().double().numpy()
    off = np.abs(got - out)
    assert (off <= tol).all(), f"{int((off > tol).sum())} of {off.size}, off by up to {(off / tol).max():.3g} of the tolerance"


@pytest.mark.parametrize("kind,heads,kv_heads,dim", [("q8", 16, 4, 128), ("f16", 16, 4, 128), ("f16", 32, 4, 64), ("q8", 16, 1, 256)])
def test_fp16_results_are_off_by_their_own_rounding(kind, heads, kv_heads, dim):
    """Rounding to fp16 is off by a uniform part of half a step either way, the square of a step / 12 on average. Over 16384 results
    and more the mean lies within 2 % of that (the square of a uniform number has a deviation of 0.9 of its mean, and steps span
    some binades: 1.5 % for 16384), and the rest, fp32's 2^-24 of scores of about 100, adds 1 % at most: 10 % are allowed."""
    rows, prefix, tokens = 8, 1008, 16
    rng = np.random.default_rng(heads)
    c = paged.Cache(kind, 1, prefix // tokens, kv_heads, dim, tokens)
    if kind == "q8":
        for a, d in zip(c.codes, c.scales):
            a[...] = rng.integers(-127, 128, a.shape)
            d[...] = rng.random(d.shape) * 0.01 + 0.01
    else:
        for a in c.values:
            a[...] = rng.standard_normal(a.shape)
    table = np.tile(np.arange(c.pages, dtype=np.int32), (rows, 1))
    q = rng.standard_normal((rows, heads, dim)).astype(np.float16)
    lens = [prefix] * rows
    out = paged.attention(c, 0, q, table, lens, prefix, dim ** -0.5)[0]
    got = qg.prefix_attention(upload(c), dev(q, np.float16), dev(table), dev(lens), dev([0, rows]), dev([prefix]), max_tail=0)
    step = np.maximum(2.0 ** (np.floor(np.log2(np.abs(out))) - 10), 2.0 ** -24)
    error = np.square(got.cpu().double().numpy() - out).sum() / (np.square(step).sum() / 12)
    assert error < 1.1, error
