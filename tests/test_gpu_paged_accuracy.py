"""GPU tests of how exactly paged decode attention adds up: scores of any size, every step of a
long cache counted once, long caches to what fp32 sums of the kernel's shape allow, and the smallest
values."""
import numpy as np
import pytest

import dequant_gemv_q4g32_amd as qg
from oracle import paged

from paged_util import attention_tolerance, check_attention, dev, upload
from test_gpu_paged_flow import _filled, _torch_reference

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# scale * log2(e) is exactly 1 in fp32 with this scale, so scores in units of log2 are <q, k> itself
LN2 = float(np.float32(np.log(2.0)))


@pytest.mark.parametrize("kind,dim", [("f16", 64), ("f16", 128), ("f16", 256), ("q8", 64), ("q8", 128), ("q8", 256)])
@pytest.mark.parametrize("exponent", [20, 24, 25, 26, 27, 28, 29])
@pytest.mark.parametrize("sign", [1, -1])
def test_large_scores(kind, dim, exponent, sign):
    """Scores of +-1.5 * 2^exponent that grow by a few of their last places from step to step: the
    weights against a running maximum of that size stay inside fp16's range. All scores are exact in
    fp32 (fp16 factors whose products and sums need no more than 24 bits), so they add nothing to the
    tolerance: weights, sums and the output's rounding only, the same as for small scores. Head h's
    scores grow by (h + 1) last places, every 32 tokens or every 96."""
    heads, tokens, n, seqs = 16, 16, 500, 2000
    ulp = max(1.0, 2.0 ** (exponent - 23))
    c = paged.Cache(kind, 1, -(-n // tokens), 1, dim, tokens)
    rng = np.random.default_rng(exponent)
    half = exponent // 2
    k = np.zeros((n, dim))
    k[:, 0] = sign * 2.0 ** half
    k[:, 33], k[:, 34] = np.arange(n) // 32 % 4, np.arange(n) // 96
    v = rng.integers(-8, 9, (n, dim)) / 4.0
    for j in range(n):
        at = (0, j // tokens, 0, j % tokens)
        if kind == "f16":
            c.values[0][at], c.values[1][at] = k[j], v[j]
        else:                                             # element 0's group has a scale of its own
            c.codes[0][at], c.codes[1][at] = np.where(np.arange(dim) == 0, sign * 64, k[j]), v[j] * 4
            c.scales[0][at], c.scales[1][at] = 1.0, 0.25
            c.scales[0][at + (0,)] = 2.0 ** half / 64
    q = np.zeros((heads, dim))
    q[:, 0] = 1.5 * 2.0 ** (exponent - half)
    q[:, 33], q[:, 34] = ulp * (1 + np.arange(heads)), 2 * ulp
    y = q @ k.T
    assert np.array_equal(q, q.astype(np.float16)) and np.array_equal(y, y.astype(np.float32))
    first = np.array([n, 33, 64, 97])                     # lengths of the first sequences; the others have n tokens
    y = np.where(np.arange(n) < first[:, None, None], y, -np.inf)
    top = y.max(-1, keepdims=True)
    w = np.exp2(y - top)
    total = w.sum(-1)
    out, bound = (w @ v) / total[..., None], (w @ np.abs(v)) / total[..., None]
    lse = (top[..., 0] + np.log2(total)) * np.log(2.0)
    which = np.zeros(seqs, int)
    which[:4] = range(4)
    table = np.tile(np.arange(c.pages, dtype=np.int32), (seqs, 1))
    wide = np.full((seqs, 8192 // tokens), -1, np.int32)
    wide[:, :c.pages] = table
    pool, lens, queries = upload(c), dev(first[which]), dev(np.tile(q, (seqs, 1, 1)), np.float16)
    for f32 in (True, False):
        tol = attention_tolerance(out, lse, bound, np.zeros_like(lse), n, dim, f32)
        ref, ref_lse, tol, tol_lse = (dev(x, np.float64)[which] for x in (out, lse, *tol))
        for t in (table, wide):                           # a workgroup a head tile, and the split
            assert (qg.paged_attention_bytes(pool, seqs, heads, t.shape[1] * tokens) > 0) == (t is wide)
            got, got_lse = qg.paged_attention(pool, queries, dev(t), lens, scale=LN2, out_f32=f32, return_lse=True)
            assert torch.isfinite(got).all() and torch.isfinite(got_lse).all()
            assert ((got.double() - ref).abs() <= tol).all(), f"{(got.double() - ref).abs().max():.3g}"
            assert ((got_lse.double() - ref_lse).abs() <= tol_lse).all()


# ---- each step once ---------------------------------------------------------------------------------

STEPS = [  # kind, heads, kv heads, dim, page tokens, table pages, lens, window
    ("q8", 8, 2, 128, 16, 8192, [131072], 0), ("f16", 4, 1, 64, 256, 157, [40000, 7, 13001], 0),
    ("q8", 16, 1, 256, 64, 313, [9000, 1, 20011], 0), ("f16", 12, 4, 128, 32, 2048, [65536, 0, 65535, 31, 1], 0),
    ("f16", 16, 2, 256, 128, 256, [32768, 20000, 3, 32737], 0), ("q8", 4, 4, 64, 16, 2048, [32768, 32000, 1025], 1025),
    ("f16", 40, 2, 128, 16, 1024, [16384, 9999] * 20, 0), ("q8", 64, 2, 64, 64, 256, [16384, 77, 16000] * 15, 0),
    ("q8", 33, 1, 256, 16, 1250, [20000, 12345] * 8, 0), ("f16", 20, 1, 64, 32, 1000, [32000, 5000] * 20, 4000),
    ("q8", 16, 4, 128, 16, 600, list(range(1, 9601, 31)), 0), ("f16", 8, 8, 64, 16, 300, list(range(0, 4800, 13)), 0),
    ("q8", 8, 8, 128, 32, 64, list(range(2048, 0, -9)), 700)]


@pytest.mark.parametrize("kind,heads,kv_heads,dim,tokens,pages,lens,window", STEPS)
def test_every_step_counts_once(kind, heads, kv_heads, dim, tokens, pages, lens, window):
    """With K = 0 every token has weight 1, so an output is the mean of V and lse is ln of the number of
    tokens. V marks each token's 32-token step in two elements (their pair names the step), with 1 or 2
    by the token's parity; one step left out, or counted twice, shows as 32 in a count.

    All sums are exact: the weights are one power of two, their multiples by 0, 1 and 2 whole numbers
    below 2^24 of it, the factors of the joins 1 (or 0, of parts without a token). What is left is the
    reciprocal's and its product's rounding, 2^-23 of the value and a bit more; for lse a logarithm of
    at most 24 good to 2^-21, and its product with ln 2."""
    n = pages * tokens
    half, step = dim // 2, np.arange(n) // 32
    marks = np.zeros((n, dim))
    value = 1.0 + np.arange(n) % 2
    marks[np.arange(n), step % half] = value
    marks[np.arange(n), half + step // half % half] = value
    c = paged.Cache(kind, 1, pages, kv_heads, dim, tokens)
    v = np.stack([np.roll(marks, g, axis=1).reshape(pages, tokens, dim) for g in range(kv_heads)], axis=1)[None]
    rng = np.random.default_rng(n)
    order = rng.permutation(pages)                        # logical page i lies in page order[i]
    if kind == "q8":
        c.codes[1][:, order], c.scales[1][...], c.scales[0][...] = v, 1.0, 0.5
    else:
        c.values[1][:, order] = v
    sums = np.concatenate([np.zeros((1, dim)), np.cumsum(marks, axis=0)])
    lens = np.array(lens)
    first = np.maximum(0, lens - window) if window else np.zeros_like(lens)
    count = lens - first
    mean = (sums[lens] - sums[first]) / np.maximum(count, 1)[:, None]
    ref = np.stack([np.roll(mean, h // (heads // kv_heads), axis=1) for h in range(heads)], axis=1)
    table = dev(np.tile(order, (len(lens), 1)))
    q = torch.randn((len(lens), heads, dim), generator=torch.Generator("cuda").manual_seed(n), device="cuda").half()
    out, lse = qg.paged_attention(upload(c), q, table, dev(lens), window=window, out_f32=True, return_lse=True)
    want = dev(ref, np.float64)
    off = (out.double() - want).abs() - 1.01 * 2.0 ** -23 * want.abs()
    assert (off <= 0).all(), f"sequence {int(off.flatten(1).amax(1).argmax())}: off by {float((out.double() - want).abs().max()):.3g}"
    with np.errstate(divide="ignore"):
        want = dev(np.log(count), np.float64)[:, None].expand_as(lse)
    some = dev(count)[:, None].expand_as(lse) > 0
    assert torch.all(torch.isneginf(lse[~some]))
    assert ((lse.double() - want).abs()[some] <= 24 * 2.0 ** -21).all(), float((lse.double() - want).abs()[some].max())


# ---- long caches closely ----------------------------------------------------------------------------

def _close_tolerance(out, lse, bound, reach, lens, head_tiles, dim):
    """As paged_util.attention_tolerance, with the roundings of sums counted along the longest chain
    instead of one for each token. Relative to sum w |V| (out) and to sum w (lse), e = 2^-24:
    - a wave runs through `steps` steps of 32 tokens: the share of the 32-token tiles of all head
      tiles (one more for short ones) that falls to each of 1024 waves, which are fewer than the kernel has
      wherever there are tiles enough, and one more;
    - a step adds 32 products twice (the weights are pairs) to a sum of V and 8 weights to the
      denominator, and may scale both: at most 2 * 33 + 1 and 9 roundings;
    - joins: 4 waves, then at most 81 parts one after the other at 3 roundings each, and the quotient:
      fewer than 260;
    - a weight as a pair of fp16 numbers is off by 2^-22 of itself, or 2^-32 of the largest."""
    e = 2.0 ** -24
    total = sum(-(-n // 32) + 1 for n in lens) * head_tiles
    steps = -(-total // 1024) + 1
    score = (dim + 8) * e * reach
    rel = 2 * (score + 2.0 ** -21) + (76 * steps + 520) * e + 2 * max(lens) * 2.0 ** -32
    with np.errstate(invalid="ignore"):
        size = np.where(np.isfinite(lse), np.abs(lse), 0.0)
    return rel[..., None] * bound + 1e-30, rel + 4 * e * (size + reach) + 4 * e


@pytest.mark.parametrize("kind,heads,kv_heads,dim,tokens,lens", [
    ("q8", 8, 2, 128, 16, [20011]), ("f16", 4, 1, 64, 256, [40000, 7, 13001]), ("q8", 16, 1, 256, 64, [9000, 1]),
    ("f16", 8, 8, 128, 32, [5000] * 3), ("q8", 4, 1, 64, 64, [40001, 39999, 20000]), ("f16", 4, 2, 128, 16, [30000, 11])])
def test_long_caches_closely(kind, heads, kv_heads, dim, tokens, lens):
    """fp32 output over long random caches, to a bound that a lost 32-token step of average weight
    passes: lse's is below half of such a step's share (asserted)."""
    pages = sum(-(-n // tokens) for n in lens)
    pool, values, gen = _filled(kind, kv_heads, dim, tokens, pages, dim + len(lens))
    order, table, at = torch.randperm(pages, generator=gen, device="cuda").int(), [], 0
    for n in lens:
        held = -(-n // tokens)
        table.append(torch.nn.functional.pad(order[at:at + held], (0, -(-max(lens) // tokens) - held), value=-1))
        at += held
    table = torch.stack(table)
    q = (torch.randn((len(lens), heads, dim), generator=gen, device="cuda") * 1.5).half()
    out, lse = qg.paged_attention(pool, q, table, dev(lens), out_f32=True, return_lse=True)
    ref = _torch_reference(*values, table, lens, q, dim ** -0.5, 0)
    tol, tol_lse = _close_tolerance(*ref, lens, kv_heads, dim)
    assert max(lens) < 16000 or (tol_lse[int(np.argmax(lens))] < 16 / max(lens)).all()
    got, got_lse = out.cpu().double().numpy(), lse.cpu().double().numpy()
    assert (np.abs(got - ref[0]) <= tol).all(), float((np.abs(got - ref[0]) / tol).max())
    assert (np.abs(got_lse - ref[1]) <= tol_lse).all(), float((np.abs(got_lse - ref[1]) / tol_lse).max())


# ---- small values -----------------------------------------------------------------------------------

@pytest.mark.parametrize("kind,dim", [("f16", 64), ("f16", 128), ("f16", 256), ("q8", 64), ("q8", 128), ("q8", 256)])
@pytest.mark.parametrize("what", ["k", "v", "q", "all"])
def test_subnormal_values(kind, dim, what):
    """K, V or q of fp16 subnormals (int8 pages: with subnormal scales), exact like any others. The scale
    makes up for them, so that the scores differ by far more than the tolerance: taken as zeros they
    would not pass, nor V, whose tolerance is relative."""
    lens, tokens, heads = [300, 33, 1], 16, 8
    rng = np.random.default_rng(dim)
    c = paged.Cache(kind, 1, 25, 2, dim, tokens)
    small = {"k": what in ("k", "all"), "v": what in ("v", "all"), "q": what in ("q", "all")}
    for i, name in enumerate("kv"):
        if kind == "q8":
            c.codes[i][...] = rng.integers(-127, 128, c.codes[i].shape)
            steps = rng.integers(1, 9, c.scales[i].shape)
            c.scales[i][...] = steps * (2.0 ** -24 if small[name] else 2.0 ** -8)
        else:
            c.values[i][...] = rng.integers(-1023, 1024, c.values[i].shape) * (2.0 ** -24 if small[name] else 2.0 ** -9)
    q = (rng.integers(-1023, 1024, (3, heads, dim)) * (2.0 ** -24 if small["q"] else 2.0 ** -9)).astype(np.float16)
    scale = float(np.float32(0.5 * (2.0 ** 15 if small["k"] else 1.0) * (2.0 ** 15 if small["q"] else 1.0) / dim))
    table = rng.integers(0, 25, (3, 19)).astype(np.int32)
    ref = paged.attention(c, 0, q, table, lens, 10 ** 6, scale)
    assert ref[0].any() and (ref[3][0] > 0.25).all()      # the size of the scores' terms
    for f32 in (True, False):
        out, lse = qg.paged_attention(upload(c), dev(q, np.float16), dev(table), dev(lens), scale=scale, out_f32=f32, return_lse=True)
        check_attention(out, lse, ref, max(lens), dim)
