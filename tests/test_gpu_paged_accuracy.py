"""GPU tests of how exactly paged decode attention adds up: scores of any size."""
import numpy as np
import pytest

import dequant_gemv_q4g32_amd as qg
from oracle import paged

from paged_util import attention_tolerance, dev, upload

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
