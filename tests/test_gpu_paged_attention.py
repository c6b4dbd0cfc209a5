"""GPU tests of paged decode attention against the fp64 oracle (oracle/paged.py), with tolerances
derived from the arithmetic (paged_util.attention_tolerance). Unused places of the pages and
unused pages hold random bytes, NaN and infinities among them: none may reach an output."""
import numpy as np
import pytest

import dequant_gemv_q4g32_amd as qg
from oracle import kvcache, paged

from paged_util import check_attention, dev, random_cache, random_table, upload

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _problem(kind, heads, kv_heads, dim, tokens, lens, seed, layers=1, extra=0):
    """A cache whose tokens up to lens are plausible and whose other bytes are poison."""
    rng = np.random.default_rng(seed)
    width = max(1, -(-max(0, max(lens)) // tokens) + extra)
    pages = sum(-(-max(0, n) // tokens) for n in lens) + 2
    good = random_cache(kind, layers, pages, kv_heads, dim, tokens, seed)
    c = random_cache(kind, layers, pages, kv_heads, dim, tokens, seed + 1, poison=True)
    table = random_table(rng, lens, tokens, pages, width)
    for s, n in enumerate(lens):
        for slot in range(-(-max(0, n) // tokens)):
            page, fill = table[s, slot], min(tokens, n - slot * tokens)
            for a, b in zip(c._arrays, good._arrays):
                a[:, page, :, :fill] = b[:, page, :, :fill]
    q = (rng.standard_normal((len(lens), heads, dim)) * 1.5).astype(np.float16)
    return rng, c, table, q


SHAPES = [  # kind, heads, kv heads, dim, page tokens, lens, window
    ("q8", 1, 1, 64, 16, [1], 0), ("q8", 32, 8, 128, 16, [1, 15, 16, 17, 31, 32, 33, 0, 200], 0),
    ("q8", 8, 8, 128, 32, [63, 64, 65, 127, 128, 129], 0), ("q8", 16, 1, 256, 128, [257, 300, 1], 0),
    ("q8", 40, 2, 64, 64, [100, 0, 511], 0), ("q8", 64, 8, 128, 16, [700], 0), ("q8", 7, 1, 128, 256, [300, 513], 0),
    ("q8", 12, 4, 256, 16, [1000, 3], 0), ("q8", 33, 1, 64, 16, [130, 40], 0),
    ("f16", 1, 1, 64, 16, [1], 0), ("f16", 32, 8, 128, 16, [1, 15, 16, 17, 31, 32, 33, 0, 200], 0),
    ("f16", 12, 12, 64, 32, [63, 64, 65, 127, 128, 129], 0), ("f16", 16, 1, 256, 128, [257, 300, 1], 0),
    ("f16", 15, 3, 128, 64, [100, 0, 511], 0), ("f16", 20, 4, 256, 16, [700, 90], 0), ("f16", 48, 1, 128, 32, [333], 0),
    ("q8", 8, 2, 128, 16, [400, 37, 5, 0, 64], 33), ("f16", 8, 2, 64, 16, [400, 37, 5, 0, 64], 1),
    ("q8", 4, 4, 64, 32, [1000, 129, 128, 127], 128), ("f16", 6, 2, 256, 16, [333, 16, 250], 250)]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("kind,heads,kv_heads,dim,tokens,lens,window", SHAPES)
def test_attention_against_oracle(kind, heads, kv_heads, dim, tokens, lens, window, f32):
    rng, c, table, q = _problem(kind, heads, kv_heads, dim, tokens, lens, heads * 100 + dim)
    out, lse = qg.paged_attention(upload(c), dev(q, np.float16), dev(table), dev(lens), window=window, out_f32=f32,
                                  return_lse=True)
    ref = paged.attention(c, 0, q, table, lens, 10 ** 9, dim ** -0.5, window)
    check_attention(out, lse, ref, max(lens), dim)


def test_q8_equals_f16_of_the_decoded_values():
    """int8 pages and fp16 pages that hold the decoded values give the same bits."""
    lens = [1, 77, 640, 0, 333]
    rng, c, table, q = _problem("q8", 16, 4, 128, 16, lens, 5)
    f = paged.Cache("f16", 1, c.pages, 4, 128, 16)
    for i in (0, 1):
        with np.errstate(all="ignore"):
            v = c.codes[i].astype(np.float64) * np.repeat(c.scales[i].astype(np.float64), 32, axis=-1)
            f.values[i] = np.clip(v, -65504, 65504).astype(np.float16)
    a = qg.paged_attention(upload(c), dev(q, np.float16), dev(table), dev(lens), return_lse=True)
    b = qg.paged_attention(upload(f), dev(q, np.float16), dev(table), dev(lens), return_lse=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_saturated_decode():
    """Scale 516 (a group's maximum above 65469): code +-127 decodes to +-65504, not to infinity."""
    c = paged.Cache("q8", 1, 2, 1, 64, 16)
    x = np.zeros((20, 64), np.float16)
    x[:, 0], x[:, 33], x[:, 1] = 65504.0, -65504.0, 500.0
    table = np.array([[1, 0]], np.int32)
    c.append(0, table, x * np.float16(1e-3), x, np.arange(20), np.zeros(20, np.int32))
    c.append(0, table, x, x * np.float16(1), [3, 7], [0, 0])
    assert float(c.scales[1][0, 1, 0, 3, 0]) == 516.0
    q = np.zeros((1, 1, 64), np.float16)
    q[0, 0, :2] = [1e-4, 1e-3]
    out, lse = qg.paged_attention(upload(c), dev(q, np.float16), dev(table), dev([20]), out_f32=True, return_lse=True)
    ref = paged.attention(c, 0, q, table, [20], 32, 0.125)
    assert np.all(np.isfinite(out.cpu().numpy()))
    check_attention(out, lse, ref, 20, 64)
    assert abs(float(out[0, 0, 0]) - 65504.0) < 1.0


def test_bad_pages_are_left_out():
    """Entries outside the pool, at the start, the middle and the end of a row, and a whole row of them."""
    lens = [90, 90, 40, 16]
    rng, c, table, q = _problem("q8", 8, 2, 64, 16, lens, 8)
    table[0, 0], table[0, 3], table[0, 5] = -1, c.pages, 2 ** 31 - 1
    table[1, 5] = -2 ** 31
    table[2, :] = -1
    for kind in ("q8", "f16"):
        if kind == "f16":
            _, c, _, _ = _problem("f16", 8, 2, 64, 16, lens, 8)
        out, lse = qg.paged_attention(upload(c), dev(q, np.float16), dev(table), dev(lens), out_f32=True, return_lse=True)
        ref = paged.attention(c, 0, q, table, lens, 96, 64 ** -0.5)
        assert np.isneginf(ref[1][2]).all() and not np.isneginf(ref[1][0]).any()
        check_attention(out, lse, ref, 90, 64)
        assert torch.all(out[2] == 0)


def test_lens_outside_and_max_len():
    """Lengths below 0 count as 0, past max_len as max_len; max_len need not be whole pages."""
    lens = [70, 70, 70, 70]
    rng, c, table, q = _problem("f16", 4, 2, 128, 16, lens, 21)
    asked = [-5, 2 ** 31 - 1, 50, -2 ** 31]
    out, lse = qg.paged_attention(upload(c), dev(q, np.float16), dev(table), dev(asked), max_len=61, out_f32=True,
                                  return_lse=True)
    check_attention(out, lse, paged.attention(c, 0, q, table, asked, 61, 128 ** -0.5), 61, 128)
    assert torch.all(out[0] == 0) and torch.all(out[3] == 0)


def test_max_len_zero_and_empty_batch():
    rng, c, table, q = _problem("q8", 4, 2, 64, 16, [5, 9], 3)
    pool = upload(c)
    out, lse = qg.paged_attention(pool, dev(q, np.float16), dev(table), dev([5, 9]), max_len=0, return_lse=True)
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))
    none = torch.empty((0, 4, 64), dtype=torch.float16, device="cuda")
    out = qg.paged_attention(pool, none, dev(table)[:0], torch.empty(0, dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 4, 64)


def test_strides_layers_and_fp16_scores():
    """q as a slice of a fused projection, out and the table as slices, the second of three layers, no lse."""
    lens = [100, 20, 64]
    rng, c, table, q = _problem("q8", 8, 2, 128, 32, lens, 31, layers=3)
    fused = torch.full((3, 8 * 128 + 2 * 2 * 128 + 8), 9.0, dtype=torch.float16, device="cuda")
    fused[:, 8:8 + 1024] = dev(q, np.float16).reshape(3, -1)
    wide = torch.full((3, 1024 + 16), 5.0, dtype=torch.float32, device="cuda")
    wt = torch.full((3, 9), -7, dtype=torch.int32, device="cuda")
    wt[:, 3:3 + table.shape[1]] = dev(table)
    out = wide[:, 4:4 + 1024].unflatten(1, (8, 128))
    got = qg.paged_attention(upload(c), fused[:, 8:8 + 1024].unflatten(1, (8, 128)), wt[:, 3:3 + table.shape[1]], dev(lens),
                             scale=0.3, out=out, layer=1)
    assert got.data_ptr() == out.data_ptr()
    ref = paged.attention(c, 1, q, table, lens, 10 ** 6, 0.3)
    check_attention(out, torch.from_numpy(ref[1]), ref, 100, 128)
    assert torch.all(wide[:, :4] == 5) and torch.all(wide[:, 4 + 1024:] == 5)


@pytest.mark.parametrize("scale", [0.0, -0.2, 4.0])
def test_scales_and_peaked_scores(scale):
    """A zero scale (plain mean), a negative one, and scores far apart in growing order (the running
    maximum moves at every step) and in falling order."""
    lens = [500, 500]
    rng, c, table, q = _problem("f16", 4, 1, 64, 16, lens, 77)
    for s, order in ((0, 1), (1, -1)):
        for j in range(500):
            page, off = table[s, j // 16], j % 16
            c.values[0][0, page, 0, off] = c.values[0][0, page, 0, off] * 0.01
            c.values[0][0, page, 0, off, 0] = np.float16((j if order > 0 else 500 - j) * 0.5)
    q[:, :, 0] = 2.0
    out, lse = qg.paged_attention(upload(c), dev(q, np.float16), dev(table), dev(lens), scale=scale, out_f32=True,
                                  return_lse=True)
    check_attention(out, lse, paged.attention(c, 0, q, table, lens, 512, scale), 500, 64)


@pytest.mark.parametrize("kind", ["q8", "f16"])
def test_infinite_and_nan_entries_stay_in_their_head(kind):
    """An infinite q makes its own head NaN or infinite as the formula says; other heads and
    sequences are untouched."""
    lens = [50, 50]
    rng, c, table, q = _problem(kind, 8, 2, 64, 16, lens, 12)
    clean = qg.paged_attention(upload(c), dev(q, np.float16), dev(table), dev(lens), return_lse=True)
    q2 = q.copy()
    q2[0, 3, 5] = np.inf
    q2[1, 6, 0] = np.nan
    out, lse = qg.paged_attention(upload(c), dev(q2, np.float16), dev(table), dev(lens), return_lse=True)
    keep = torch.ones((2, 8), dtype=torch.bool)
    keep[0, 3] = keep[1, 6] = False
    assert torch.equal(out.cpu()[keep], clean[0].cpu()[keep]) and torch.equal(lse.cpu()[keep], clean[1].cpu()[keep])
    assert torch.all(torch.isnan(out[1, 6])) and torch.isnan(lse[1, 6])
    assert not torch.any(torch.isfinite(out[0, 3]))


@pytest.mark.parametrize("kind", ["q8", "f16"])
@pytest.mark.parametrize("max_len", [64, 40000])
def test_rows_without_tokens_ignore_q(kind, max_len):
    """A padded batch's empty rows may hold anything in q: no token, so zeros and -inf. The same for
    a row whose pages are all missing, and a first page missing does not hide a NaN."""
    lens = [0, 40, 40, -3, 40, 64]
    rng, c, table, q = _problem(kind, 8, 2, 64, 16, lens, 13)
    wide = np.full((len(lens), max(max_len // 16, table.shape[1])), -1, np.int32)
    wide[:, :table.shape[1]] = table
    wide[2] = -1
    wide[5, :2] = -1
    q[0] = np.nan
    q[2] = np.inf
    q[3, :, 1::2] = -np.inf
    q[5, 6, 40] = np.nan
    out, lse = qg.paged_attention(upload(c), dev(q, np.float16), dev(wide), dev(lens), max_len=max_len, return_lse=True)
    for b in (0, 2, 3):
        assert torch.all(out[b] == 0) and torch.all(lse[b] == -float("inf")), b
    keep = torch.ones((len(lens), 8), dtype=torch.bool)
    keep[5, 6] = False
    assert torch.all(torch.isnan(out[5, 6])) and torch.isnan(lse[5, 6])
    assert torch.all(torch.isfinite(out.cpu()[keep]))


def _reference(pool_values, table, lens, q, scale):
    """fp64 torch reference on the GPU for long caches: pool_values (K, V) fp16 [pages, heads, T, D]."""
    batch, heads, dim = q.shape
    kv = pool_values[0].shape[1]
    tokens = pool_values[0].shape[2]
    out, bound = torch.zeros((2, batch, heads, dim), dtype=torch.float64, device="cuda")
    lse, reach = torch.zeros((2, batch, heads), dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        at = table[b, :-(-n // tokens)].long()
        k, v = (x[at].transpose(0, 1).flatten(1, 2)[:, :n].double() for x in pool_values)
        for h in range(heads):
            kh, vh, x = k[h * kv // heads], v[h * kv // heads], q[b, h].double()
            s = (kh * x).sum(-1) * scale
            w = torch.softmax(s, 0)[:, None]
            out[b, h], bound[b, h] = (w * vh).sum(0), (w * vh.abs()).sum(0)
            lse[b, h], reach[b, h] = torch.logsumexp(s, 0), ((kh * x).abs().sum(-1) * abs(scale)).max()
    return tuple(t.cpu().numpy() for t in (out, lse, bound, reach))


@pytest.mark.parametrize("kind,heads,kv_heads,dim,tokens,lens", [
    ("q8", 8, 2, 128, 16, [20011]), ("f16", 4, 1, 64, 256, [40000, 7, 13001]), ("q8", 16, 1, 256, 64, [9000, 1]),
    ("f16", 8, 8, 128, 32, [5000] * 3)])
def test_long_caches(kind, heads, kv_heads, dim, tokens, lens):
    gen = torch.Generator("cuda").manual_seed(dim)
    width = -(-max(lens) // tokens)
    pages = sum(-(-n // tokens) for n in lens) + 1
    rng = np.random.default_rng(dim)
    table = dev(random_table(rng, lens, tokens, pages, width))
    pool = qg.KVPool.zeros(kind, kv_heads, dim, tokens, pages)
    k, v = torch.randn((2, pages, tokens, kv_heads * dim), generator=gen, device="cuda").half()
    all_pages = torch.arange(pages, device="cuda", dtype=torch.int32)[:, None].contiguous()
    place = torch.arange(tokens, device="cuda", dtype=torch.int32).repeat(pages)
    seq = torch.arange(pages, device="cuda", dtype=torch.int32).repeat_interleave(tokens)
    qg.kv_append(pool, all_pages, k.flatten(0, 1), v.flatten(0, 1), place, seq)
    gk, gv = qg.kv_gather(pool, all_pages, place, seq)
    values = [x.view(pages, tokens, kv_heads, dim).transpose(1, 2) for x in (gk, gv)]
    q = (torch.randn((len(lens), heads, dim), generator=gen, device="cuda") * 1.5).half()
    for f32 in (True, False):
        out, lse = qg.paged_attention(pool, q, table, dev(lens), out_f32=f32, return_lse=True)
        check_attention(out, lse, _reference(values, table, lens, q, dim ** -0.5), max(lens), dim)
    again = qg.paged_attention(pool, q, table, dev(lens), return_lse=True)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)     # equal inputs, equal bits


def test_offsets_past_32_bits():
    """Pages beyond the first 4 GiB of a layer, and a layer beyond it: a 5 GiB pool written and read there."""
    pages, heads, dim, tokens = 20000, 8, 128, 128
    pool = qg.KVPool(torch.empty((pages, qg.kv_page_bytes("q8", heads, dim, tokens)), dtype=torch.uint8, device="cuda"), "q8",
                     heads, dim, tokens)
    assert pool.pages.numel() > 2 ** 32
    pool.pages[-3:] = 0
    pool.pages[:3] = 0x7C
    lens = [300]
    table = dev([[pages - 1, pages - 3, pages - 2]])
    gen = torch.Generator("cuda").manual_seed(1)
    k, v = torch.randn((2, 300, heads * dim), generator=gen, device="cuda").half()
    pos, seq = torch.arange(300, dtype=torch.int32, device="cuda"), torch.zeros(300, dtype=torch.int32, device="cuda")
    qg.kv_append(pool, table, k, v, pos, seq)
    gk, gv = qg.kv_gather(pool, table, pos, seq)
    q8, d8 = kvcache.quantize(k.cpu().numpy())
    assert np.array_equal(gk.cpu().numpy(), kvcache.dequantize_fp16(q8, d8))
    q = torch.randn((1, 16, dim), generator=gen, device="cuda").half()
    out, lse = qg.paged_attention(pool, q, table, dev(lens), out_f32=True, return_lse=True)
    kk, vv = (torch.cat([x, x.new_zeros(84, heads * dim)]).view(3, tokens, heads, dim).transpose(1, 2) for x in (gk, gv))
    check_attention(out, lse, _reference((kk, vv), dev([[0, 1, 2]]), lens, q, dim ** -0.5), 300, dim)
    qg.kv_copy_pages(pool, dev([pages - 1]), dev([pages // 2]))
    assert torch.equal(pool.pages[pages // 2], pool.pages[pages - 1])
