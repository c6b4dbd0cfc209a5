"""GPU tests of how exactly queries and keys are normed and rotated: heads that hold an infinity, sums whose terms all but
cancel, so that the rounding of the result to fp16 hides nothing of cosine and sine, and the codes of int8 keys."""
import numpy as np
import pytest

import dequant_gemv_q4g32_amd as qg
from oracle import kvcache, paged, step

from paged_util import dev, download, random_table, upload

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,rot,inter", [(64, 32, False), (128, 128, True), (256, 0, False), (256, 192, True)])
def test_norm_of_a_head_with_an_infinity(dim, rot, inter):
    """Its root is infinite: what is finite becomes zero, the infinity itself NaN, and so does its pair's other half."""
    rng = np.random.default_rng(dim)
    w = (rng.random(dim) + 0.5).astype(np.float16)
    freqs = qg.rope_freqs(rot) if rot else None
    rotary = qg.Rotary(dim, freqs, inter, dev(w, np.float16), dev(w, np.float16))
    x = rng.standard_normal((3, 4, dim)).astype(np.float16)
    x[0, 1, 5], x[1, 0, dim - 1], x[2, 3, 0], x[2, 3, 9] = np.inf, -np.inf, np.inf, -np.inf
    pos = np.array([0, 3, 100000], np.int32)
    with np.errstate(invalid="ignore"):
        want = np.stack([[step.rotate(h, p, [] if freqs is None else freqs, inter, w, 1e-6) for h in heads] for heads, p in zip(x, pos)])
    got = qg.qk_rope(rotary, dev(x, np.float16), dev(x, np.float16), dev(pos))
    for out in got:
        out = out.cpu().numpy().astype(np.float64)
        assert np.array_equal(np.isnan(out), np.isnan(want))
        odd = ~np.isfinite(x).all(-1)
        assert (out[odd][~np.isnan(want[odd])] == 0).all() and (want[odd][~np.isnan(want[odd])] == 0).all()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("factor", [1.0, -0.75])
@pytest.mark.parametrize("norm", [False, True])
def test_rotations_that_cancel(inter, factor, norm):
    """(y1, y2) chosen so that y1 cos t - y2 sin t is a 2^-14 and less of its terms. e = 2^-24: cosine and sine, in fp64 with the factor,
    are rounded to fp32 once (e of each term), a product is rounded (e), and the sum (e of the result, which is next to nothing), so
    the result is off by 2 e of its terms, and half a step of fp16. Angles in fp64: 2^-52 of 16000 turns, nothing. Normed
    elements are two products more, each with e of its own; what the root is off by is both terms' and cancels with them."""
    dim, count, e = 128, 64, 2.0 ** -24
    half = dim // 2
    rng = np.random.default_rng(3)
    freqs = qg.rope_freqs(dim)
    pos = rng.integers(0, 100000, count).astype(np.int32)
    t = pos[:, None] * freqs
    cos, sin = np.cos(t), np.sin(t)
    w = (rng.random(dim) + 0.5).astype(np.float16) if norm else np.ones(dim, np.float16)
    first, second = (np.arange(0, dim, 2), np.arange(1, dim, 2)) if inter else (np.arange(half), np.arange(half, dim))
    wide = w.astype(np.float64)
    b = rng.uniform(256, 1024, (2000, count, half)).astype(np.float16)      # candidates of y2, and the y1 next to y2 tan t
    with np.errstate(over="ignore", divide="ignore"):
        a = (b.astype(np.float64) * wide[second] * sin / (wide[first] * cos)).astype(np.float16)
    fits = (np.abs(a) > 2.0 ** -3) & (np.abs(a) < 4096)                     # neither subnormal nor large
    left = np.abs(a.astype(np.float64) * wide[first] * cos - b.astype(np.float64) * wide[second] * sin)
    pick = np.argmin(np.where(fits, left, np.inf), axis=0)[None]
    a, b = (np.take_along_axis(v, pick, 0)[0] for v in (a, b))
    usable = np.take_along_axis(fits, pick, 0)[0]
    x = np.zeros((count, dim), np.float16)
    x[:, first], x[:, second] = np.where(usable, a, 1), b
    rotary = qg.Rotary(dim, freqs, inter, dev(w, np.float16) if norm else None, factor=factor, eps=1e-6)
    got = qg.qk_rope(rotary, dev(x, np.float16), None, dev(pos))[0].cpu().numpy().astype(np.float64)[:, first]
    want = np.stack([step.rotate(h, p, freqs, inter, w if norm else None, 1e-6, factor) for h, p in zip(x, pos)])[:, first]
    y = np.stack([step.rotate(h, p, [], inter, w if norm else None, 1e-6) for h, p in zip(x, pos)])
    size = abs(factor) * (np.abs(y[:, first] * cos) + np.abs(y[:, second] * sin))
    usable &= np.abs(want) < 2.0 ** -14 * size
    assert usable.sum() > count * half * 0.8
    off = np.abs(got - want)
    tol = size * e * (2 + (2 if norm else 0)) + np.abs(want) * (2.0 ** -11 + (16 * e if norm else e)) + 2.0 ** -25
    assert (off <= tol)[usable].all(), (off / tol)[usable].max()


def test_codes_of_int8_keys():
    """Keys are fp64, rounded to fp32 and then to fp16. Against one rounding to fp16 the first of the two puts 2^-13 of the elements
    on a tie, and half of these go the other way: 2^-14 of them, 64 of 2^20, by one step, which is 2^-10 of the element at most. That
    moves its place between two codes by 127 * 2^-10 = 1/8 of their distance at most, and, where it is the largest of its 32, the
    others' places as well: at most 64 * (1 + 32 / 32) / 8 = 16 codes are expected to change, by one. 16 and 4 deviations are 32."""
    count, heads, dim, tokens = 1024, 8, 128, 16
    rng = np.random.default_rng(12)
    k = rng.standard_normal((count, heads, dim)).astype(np.float16)
    w = (rng.random(dim) + 0.5).astype(np.float16)
    freqs = qg.rope_freqs(dim)
    y = k.astype(np.float64)
    y = y / np.sqrt((y * y).mean(-1, keepdims=True) + float(np.float32(1e-6))) * w.astype(np.float64)
    t = np.arange(count)[:, None, None] * freqs
    a, b = y[..., :dim // 2], y[..., dim // 2:]
    exact = np.concatenate([a * np.cos(t) - b * np.sin(t), b * np.cos(t) + a * np.sin(t)], -1)
    once, twice = exact.astype(np.float16), exact.astype(np.float32).astype(np.float16)
    assert 30 < (once != twice).sum() < 110                # 64 and 5 deviations
    c = paged.Cache("q8", 1, count // tokens, heads, dim, tokens)
    pool, table = upload(c), random_table(rng, [count], tokens, count // tokens, count // tokens)
    qg.kv_append_rope(pool, dev(table), qg.Rotary(dim, freqs, k_weight=dev(w, np.float16)), None, dev(k.reshape(count, -1), np.float16),
                      dev(k.reshape(count, -1), np.float16), dev(np.arange(count)), dev(np.zeros(count)))
    torch.cuda.synchronize()
    got = download(c, pool)
    for x, most in ((twice, 0), (once, 32)):
        codes, scales = kvcache.quantize(x.reshape(-1, dim))
        order = lambda v: np.swapaxes(v[0][table[0]], 1, 2).reshape(count, heads, -1)   # [pages, heads, tokens, ..] by token
        off = order(got.codes[0]).astype(int) - codes.reshape(count, heads, -1)
        assert np.abs(off).max() <= 1 and (off != 0).sum() <= most, (off != 0).sum()
        assert most or np.array_equal(order(got.scales[0]), scales.reshape(count, heads, -1))
