"""GPU tests of a decode step's operators against the oracle: places for tokens (extend and trim, whole
numbers, equal), and the norm and rotation of queries and keys, alone and on their way into the cache."""
import numpy as np
import pytest

import dequant_gemv_q4g32_amd as qg
from oracle import step

from paged_util import assert_same_bytes, dev, download, random_cache, random_table, upload

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


# ---- extend and trim ---------------------------------------------------------------------------

def small_pool(pages, tokens):
    return qg.KVPool.zeros("q8", 1, 64, tokens, pages)


def check_extend(pool, table, lens, refs, add, slots, starts=True):
    """One call against the oracle; both sides' tables, lengths and counts move on."""
    t, n, r = dev(table), dev(lens), dev(refs)
    first = torch.full((len(lens) + 1,), -7, dtype=torch.int32, device="cuda") if starts else None
    granted, seqs, pos = qg.kv_extend(pool, t, n, r, dev(add), slots, starts=first)
    want = step.extend(table, lens, refs, add, slots, pool.page_tokens)
    torch.cuda.synchronize()
    for name, got, ref in [("granted", granted, want[0]), ("seqs", seqs, want[2]), ("positions", pos, want[3]), ("table", t, table),
                           ("lens", n, lens), ("refs", r, refs)] + ([("starts", first, want[1])] if starts else []):
        assert np.array_equal(got.cpu().numpy(), ref), name


def filled(rng, rows, tokens, pages, width, most):
    """A table of rows of random lengths in a pool with free pages between theirs; the rows that the pool has no
    pages for are empty."""
    lens = rng.integers(0, most + 1, rows).astype(np.int32)
    lens[np.cumsum(-(-lens // tokens)) > pages - 1] = 0
    table = random_table(rng, lens, tokens, pages, width)
    refs = np.zeros(pages, np.int32)
    refs[table[table >= 0]] = 1
    return table, lens, refs


@pytest.mark.parametrize("rows,tokens,pages,width,most,add_most,slots", [
    (1, 16, 4, 3, 0, 1, 1), (1, 16, 1, 1, 15, 1, 1), (3, 16, 40, 8, 60, 40, 200), (64, 16, 700, 12, 100, 3, 130),
    (64, 32, 90, 4, 64, 64, 4096), (300, 16, 4097, 20, 200, 30, 5000), (1023, 16, 9000, 12, 100, 2, 3000),
    (1024, 64, 5000, 6, 300, 80, 50000), (1025, 16, 8192, 9, 90, 40, 20000), (5000, 16, 20000, 5, 60, 9, 30000),
    (9001, 16, 70000, 10, 100, 2, 20000), (65536, 16, 140000, 3, 30, 2, 70000), (17, 256, 33, 3, 700, 300, 2000)])
def test_extend(rows, tokens, pages, width, most, add_most, slots):
    rng = np.random.default_rng(rows + pages)
    table, lens, refs = filled(rng, rows, tokens, pages, width, most)
    pool = small_pool(pages, tokens)
    for k in range(3):                                    # until pages, slots or table rows run out
        check_extend(pool, table, lens, refs, rng.integers(-1, add_most + 1, rows).astype(np.int32), slots, starts=k != 1)


def test_extend_large_pool():
    """Many blocks of pages, all held but a few far apart."""
    rng = np.random.default_rng(5)
    pages, rows = 1 << 20, 700
    refs = np.ones(pages, np.int32)
    refs[rng.choice(pages, 1500, replace=False)] = 0
    refs[-1] = 0
    table, lens = np.full((rows, 40), -1, np.int32), np.zeros(rows, np.int32)
    pool = qg.KVPool(torch.empty((pages, qg.kv_page_bytes("q8", 1, 64, 16)), dtype=torch.uint8, device="cuda"), "q8", 1, 64, 16)
    for _ in range(3):
        check_extend(pool, table, lens, refs, rng.integers(0, 33, rows).astype(np.int32), 16384)


def test_extend_shared_pages_and_holes():
    """Rows whose partly filled page other rows hold, or which is no page, get none; whole shared pages do not matter."""
    table = np.array([[0, 1, -1, -1], [0, 2, -1, -1], [3, 3, -1, -1], [-1, -1, -1, -1], [9, 4, -1, -1], [6, 999, -1, -1]], np.int32)
    lens = np.array([32, 20, 31, 5, 17, 16], np.int32)
    refs = np.array([2, 1, 1, 2, 1, 0, 1, 0, -3, 0], np.int32)
    check_extend(small_pool(10, 16), table, lens, refs, np.full(6, 2, np.int32), 20)


def test_extend_odd_lengths_and_requests():
    """Lengths below 0 and past the table, requests past everything."""
    table = np.full((5, 2), -1, np.int32)
    lens = np.array([-9, 40, 2 ** 31 - 1, 0, 0], np.int32)
    check_extend(small_pool(12, 16), table, lens, np.zeros(12, np.int32), np.array([3, 1, 2 ** 31 - 1, 2 ** 31 - 1, 4], np.int32), 64)
    table, lens = np.full((3, 2), -1, np.int32), np.zeros(3, np.int32)
    check_extend(small_pool(12, 16), table, lens, np.zeros(12, np.int32), np.array([5, 6, 7], np.int32), 0)


def test_extend_no_rows_and_narrow_tables():
    pool = small_pool(12, 16)
    check_extend(pool, np.zeros((0, 3), np.int32), np.zeros(0, np.int32), np.zeros(12, np.int32), np.zeros(0, np.int32), 5)
    check_extend(pool, np.zeros((3, 0), np.int32), np.zeros(3, np.int32), np.zeros(12, np.int32), np.ones(3, np.int32), 5)


def test_extend_given_outputs_and_strided_table():
    rng = np.random.default_rng(8)
    table, lens, refs = filled(rng, 9, 16, 60, 6, 50)
    wide = torch.full((9, 11), 77, dtype=torch.int32, device="cuda")
    wide[:, 2:8] = dev(table)
    t, n, r, add = wide[:, 2:8], dev(lens), dev(refs), rng.integers(0, 30, 9).astype(np.int32)
    out = [torch.empty(k, dtype=torch.int32, device="cuda") for k in (9, 10, 300, 300)]
    got = qg.kv_extend(small_pool(60, 16), t, n, r, dev(add), 300, *out)
    assert got[0] is out[0] and got[1] is out[2] and got[2] is out[3]
    want = step.extend(table, lens, refs, add, 300, 16)
    torch.cuda.synchronize()
    for a, b in zip(out, want):
        assert np.array_equal(a.cpu().numpy(), b)
    assert np.array_equal(t.cpu().numpy(), table) and (wide[:, :2] == 77).all() and (wide[:, 8:] == 77).all()


@pytest.mark.parametrize("rows,tokens,pages,width,most", [(1, 16, 4, 3, 40), (37, 16, 300, 10, 150), (500, 64, 1500, 4, 250)])
def test_trim(rows, tokens, pages, width, most):
    rng = np.random.default_rng(rows)
    table, lens, refs = filled(rng, rows, tokens, pages, width, most)
    if rows > 4:                                          # shared and missing pages, a length past the table
        table[1], lens[1] = table[0], lens[0]
        for e in table[0][table[0] >= 0]:
            refs[e] += 1
        table[2, :2] = (-5, pages)
        lens[2] = width * tokens + 9
    to = rng.integers(-2, most + 2, rows).astype(np.int32)
    t, n, r = dev(table), dev(lens), dev(refs)
    qg.kv_trim(small_pool(pages, tokens), t, n, r, dev(to))
    step.trim(table, lens, refs, to, tokens)
    torch.cuda.synchronize()
    assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(n.cpu().numpy(), lens) and np.array_equal(r.cpu().numpy(), refs)


# ---- norm and rotation ---------------------------------------------------------------------------

def rope_tolerance(want, size, dim, norm):
    """How far a rotated head may be from the oracle's. e = 2^-24, half a step of fp32.

    Of an element's value: 2^-11 for the rounding to fp16 (2^-25 where that is subnormal). Of `size`, |y1| + |y2| times
    the factor: cosine and sine, from an angle reduced in fp64 (1e-7 turns at 2^31 tokens) to an fp32 part of a turn (e of at
    most half a turn: 2 pi e / 2 radians) by an instruction good to 2^-22, and the factor's product: 16 e together; two products and a
    sum: 3 e; the norm: a sum of `dim` squares in any order, dim e at most, halved by the root, its mean and the
    reciprocal root's one step (2 e), and two products: dim / 2 e + 6 e."""
    e = 2.0 ** -24
    return np.abs(want) * 2.0 ** -11 + 2.0 ** -25 + size * e * (20 + (dim / 2 + 6 if norm else 0))


def check_heads(got, x, positions, dim, freqs, weight, interleaved, factor, eps, skipped=None):
    """got, x: [count, heads * dim] arrays."""
    half = 0 if freqs is None else len(freqs)
    for i, p in enumerate(positions):
        for h in range(x.shape[1] // dim):
            at = slice(h * dim, (h + 1) * dim)
            if p < 0:
                assert np.array_equal(got[i, at].view(np.uint16), skipped[i, at].view(np.uint16))
                continue
            want = step.rotate(x[i, at], p, [] if half == 0 else freqs, interleaved, weight, eps, factor)
            y = np.abs(step.rotate(x[i, at], p, [], False, weight, eps))
            size = y.copy()
            for j in range(half):
                a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
                size[a] = size[b] = (y[a] + y[b]) * abs(factor)
            off = np.abs(got[i, at].astype(np.float64) - want)
            assert (off <= rope_tolerance(want, size, dim, weight is not None)).all(), (i, h, int(np.argmax(off)), off.max())


def heads_of(rng, count, heads, dim, ld):
    """A strided device tensor [count, heads * dim], its host values, channels of different size."""
    whole = (rng.standard_normal((count, ld)) * 1.5).astype(np.float16)
    t = dev(whole, np.float16)
    return t[:, :heads * dim], whole[:, :heads * dim]


ROPES = [
    # dim, rotary dim, interleaved, heads, kv heads, count, norms (q, k), factor
    (128, 128, False, 32, 8, 5, True, True, 1.0), (128, 128, True, 4, 4, 3, False, False, 1.0), (64, 64, False, 12, 12, 7, True, False, 1.0),
    (64, 16, False, 3, 1, 2, False, True, 0.5), (64, 48, True, 5, 1, 4, True, True, 1.0), (256, 64, True, 16, 2, 3, True, True, 1.0),
    (256, 256, False, 2, 1, 9, True, True, 1.25), (256, 48, False, 7, 7, 2, False, False, -2.0), (128, 0, False, 9, 3, 3, True, True, 1.0),
    (128, 112, False, 1, 1, 1, False, False, 1.0), (64, 32, True, 71, 1, 1, False, False, 1.0), (128, 0, True, 2, 2, 2, False, False, 3.0)]


@pytest.mark.parametrize("dim,rot,inter,heads,kv_heads,count,qn,kn,factor", ROPES)
def test_qk_rope(dim, rot, inter, heads, kv_heads, count, qn, kn, factor):
    rng = np.random.default_rng(dim + rot + heads)
    freqs = qg.rope_freqs(rot) if rot else None
    wq, wk = ((rng.random(dim) + 0.5).astype(np.float16) if on else None for on in (qn, kn))
    rotary = qg.Rotary(dim, freqs, inter, *(None if w is None else dev(w, np.float16) for w in (wq, wk)), eps=1e-5, factor=factor)
    q, qh = heads_of(rng, count, heads, dim, heads * dim + 24)
    k, kh = heads_of(rng, count, kv_heads, dim, kv_heads * dim + 8)
    pos = rng.integers(0, 100000, count).astype(np.int32)
    pos[0] = 0
    q_out, k_out = qg.qk_rope(rotary, q, k, dev(pos))
    assert q_out.is_contiguous() and k_out.is_contiguous()
    check_heads(q_out.cpu().numpy(), qh, pos, dim, freqs, wq, inter, factor, 1e-5)
    check_heads(k_out.cpu().numpy(), kh, pos, dim, freqs, wk, inter, factor, 1e-5)
    if rot == 0 and not qn:
        assert np.array_equal(q_out.cpu().numpy(), qh)    # nothing to do: the same bits
    # in place, into the strided rows themselves
    again = qg.qk_rope(rotary, q, k, dev(pos), q_out=q, k_out=k)
    assert again[0] is q and torch.equal(q.view(torch.int16), q_out.view(torch.int16)) and torch.equal(k.view(torch.int16), k_out.view(torch.int16))


def test_qk_rope_far_positions():
    """Angles of positions up to the last one, and of frequencies below zero and above a turn a token."""
    rng = np.random.default_rng(4)
    freqs = np.concatenate([qg.rope_freqs(16), [-0.3, 7.0, 100.25, 0.0, 1e-9, 3.1, 2.0, 1.0]])
    pos = np.array([1, 131071, 2 ** 24 + 1, 2 ** 31 - 1], np.int32)
    q, qh = heads_of(rng, 4, 2, 64, 128)
    out, none = qg.qk_rope(qg.Rotary(64, freqs), q, None, dev(pos))
    assert none is None
    for i, p in enumerate(pos):                           # the oracle's own product has 2^-53 of the angle
        check_heads(out.cpu().numpy()[i:i + 1], qh[i:i + 1], [p], 64, np.abs(freqs) * 0 + freqs, None, False, 1.0, 0.0)


def test_qk_rope_skipped_rows_and_odd_values():
    """Rows at positions below 0 stay as they were; NaN and infinity stay in their own head; zero heads norm to zeros."""
    rng = np.random.default_rng(6)
    q, qh = heads_of(rng, 6, 3, 128, 384)
    q[2, 5] = float("nan")
    q[3, 130] = float("inf")
    q[4, 256:] = 0
    qh = q.cpu().numpy()
    w = (rng.random(128) + 0.5).astype(np.float16)
    freqs = qg.rope_freqs(128)
    pos = np.array([5, -1, 7, 8, 9, -2 ** 31], np.int32)
    out = torch.full((6, 384), 9.0, dtype=torch.float16, device="cuda")
    qg.qk_rope(qg.Rotary(128, freqs, q_weight=dev(w, np.float16)), q, None, dev(pos), q_out=out)
    got = out.cpu().numpy()
    assert (got[[1, 5]] == 9).all()
    assert np.isnan(got[2, :128]).all() and np.isnan(got[3, 128:256]).any()
    assert np.isfinite(got[2, 128:]).all() and np.isfinite(got[3, :128]).all() and np.isfinite(got[3, 256:]).all() and (got[4, 256:] == 0).all()
    fine = [0, 4]
    check_heads(got[fine], qh[fine], pos[fine], 128, freqs, w, False, 1.0, 1e-6)


def test_qk_rope_many_tokens():
    """More tokens than a launch's own split of heads, a count that is no multiple of anything; three-dimensional heads."""
    rng = np.random.default_rng(9)
    count, dim = 2051, 64
    q = dev(rng.standard_normal((count, 40, dim)), np.float16)
    k = dev(rng.standard_normal((count, 2, dim)), np.float16)
    pos = dev(np.arange(count) * 37 % 5000)
    freqs = qg.rope_freqs(64)
    rotary = qg.Rotary(dim, freqs)
    out, k_out = qg.qk_rope(rotary, q, k, pos)
    assert out.shape == q.shape and k_out.shape == k.shape
    for i in (0, 1, 1023, 1024, 2050):
        check_heads(out[i].cpu().numpy().reshape(1, -1), q[i].cpu().numpy().reshape(1, -1), [int(pos[i])], dim, freqs, None, False, 1.0, 0.0)
        # a row's result is the same in any call
        alone = qg.qk_rope(rotary, q[i:i + 1], k[i:i + 1], pos[i:i + 1])
        assert torch.equal(alone[0][0], out[i]) and torch.equal(alone[1][0], k_out[i])
    whole = torch.stack([qg.qk_rope(rotary, q[i:i + 64], None, pos[i:i + 64])[0] for i in range(0, 2048, 64)]).flatten(0, 1)
    assert torch.equal(whole, out[:2048])


@pytest.mark.parametrize("kind", ["q8", "f16"])
@pytest.mark.parametrize("dim,rot,inter,heads,kv_heads,count,norm", [
    (128, 128, False, 32, 8, 9, True), (64, 32, True, 6, 3, 20, False), (256, 64, True, 8, 1, 5, True), (64, 64, False, 0, 12, 4, True),
    (128, 48, False, 5, 5, 1, False), (128, 128, False, 4, 1, 1500, False)])
def test_append_rope(kind, dim, rot, inter, heads, kv_heads, count, norm):
    """The same bytes as qk_rope and kv_append one after the other, for int8 pages with the keys as fp64 rounds them; rows
    without a place, and skipped ones."""
    rng = np.random.default_rng(dim + count)
    tokens, layers, rows = 16, 2, 7
    width = -(-count // (tokens * rows)) + 2
    pages = rows * width + 2
    c = random_cache(kind, layers, pages, kv_heads, dim, tokens, 2, poison=True)
    pool, other = upload(c), upload(c)
    table = random_table(rng, [width * tokens] * rows, tokens, pages, width)
    table[3, 0] = -1
    table[4, 1] = pages + 3
    places = rng.permutation(rows * width * tokens)[:count]
    seqs, pos = (places // (width * tokens)).astype(np.int32), (places % (width * tokens)).astype(np.int32)
    if count > 4:
        seqs[0], pos[1], pos[2], seqs[3] = -1, -1, width * tokens, rows
    fused = dev(rng.standard_normal((count, (heads + 2 * kv_heads) * dim + 8)), np.float16)
    q, k, v = fused[:, :heads * dim], fused[:, heads * dim:(heads + kv_heads) * dim], fused[:, (heads + kv_heads) * dim:(heads + 2 * kv_heads) * dim]
    w = [dev(rng.random(dim) + 0.5, np.float16) if norm else None for _ in range(2)]
    rotary = qg.Rotary(dim, qg.rope_freqs(rot, 10000.0, "linear", 2.0), inter, *w)
    before = torch.full((count, heads * dim), 3.0, dtype=torch.float16, device="cuda")
    got = qg.kv_append_rope(pool, dev(table), rotary, q if heads else None, k, v, dev(pos), dev(seqs), q_out=before.clone() if heads else None, layer=1)
    keys = k.cpu().numpy().reshape(count, kv_heads, dim)   # k itself is the output where it is dense
    want_q, want_k = qg.qk_rope(rotary, q, k, dev(pos), q_out=before.clone(), k_out=k.contiguous())
    if kind == "q8":
        freqs, weight = qg.rope_freqs(rot, 10000.0, "linear", 2.0), None if w[1] is None else w[1].cpu().numpy()
        exact = np.stack([[step.rotate(x, p, freqs, inter, weight, float(np.float32(1e-6))) for x in heads_] for heads_, p in zip(keys, pos)])
        want_k = dev(exact.astype(np.float32).reshape(count, -1), np.float16)
    qg.kv_append(other, dev(table), want_k, v, dev(pos), dev(seqs), layer=1)
    torch.cuda.synchronize()
    assert torch.equal(got, want_q) if heads else got is None
    assert_same_bytes(download(c, pool), download(c, other))


def test_append_rope_in_place_and_rows_by_number():
    """q itself as the output, seqs left out, queries as [count, heads, dim]."""
    rng = np.random.default_rng(3)
    c = random_cache("q8", 1, 6, 2, 64, 16, 1)
    pool, other = upload(c), upload(c)
    table, pos = dev([[0, 1], [2, 3], [4, 5]]), dev([0, 17, 31])
    q, k, v = (dev(rng.standard_normal((3, n, 64)), np.float16) for n in (6, 2, 2))
    rotary = qg.Rotary(64, qg.rope_freqs(64))
    want = qg.kv_append_rope(other, table, rotary, q, k.flatten(1), v.flatten(1), pos, dev([0, 1, 2]))
    got = qg.kv_append_rope(pool, table, rotary, q, k.flatten(1), v.flatten(1), pos, q_out=q)
    torch.cuda.synchronize()
    assert got is q and torch.equal(got, want)
    assert_same_bytes(download(c, pool), download(c, other))


def test_binding_refusals():
    pool = small_pool(4, 16)
    t, i = torch.zeros((3, 2), dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    refs = torch.zeros(4, dtype=torch.int32, device="cuda")
    q = torch.zeros((3, 128), dtype=torch.float16, device="cuda")
    k = torch.zeros((3, 64), dtype=torch.float16, device="cuda")
    rotary, wide = qg.Rotary(64, qg.rope_freqs(64)), qg.Rotary(128, qg.rope_freqs(64))
    for bad in (lambda: qg.kv_extend(pool, t, i, refs, i[:2], 4), lambda: qg.kv_extend(pool, t, i, refs[:3], i, 4),
                lambda: qg.kv_extend(pool, t, i.long(), refs, i, 4), lambda: qg.kv_extend(pool, t, i, refs, i.cpu(), 4),
                lambda: qg.kv_extend(pool, t, i, refs, i, 4, seqs=i), lambda: qg.kv_extend(pool, t, i, refs, i, 4, starts=i),
                lambda: qg.kv_extend(pool, t, i, refs, i, -1),
                lambda: qg.kv_trim(pool, t, i, refs, i[:1]), lambda: qg.kv_trim(pool, t.float(), i, refs, i),
                lambda: qg.qk_rope(rotary, q.float(), k, i), lambda: qg.qk_rope(rotary, q[:, :100], k, i),
                lambda: qg.qk_rope(rotary, q, k[:2], i), lambda: qg.qk_rope(rotary, q, k, i[:2]), lambda: qg.qk_rope(rotary, q, k, i, q_out=k),
                lambda: qg.kv_append_rope(pool, t, wide, q, k, k, i), lambda: qg.kv_append_rope(pool, t, rotary, q[:2], k, k, i),
                lambda: qg.kv_append_rope(pool, t, rotary, q, q, k, i), lambda: qg.kv_append_rope(pool, t, rotary, q, k, k, i, q_out=k)):
        with pytest.raises(ValueError):
            bad()


def test_outputs_of_other_heads():
    q, k, wide = (torch.zeros((2, n), dtype=torch.float16, device="cuda") for n in (128, 64, 192))
    i = dev([0, 1])
    rotary = qg.Rotary(64, qg.rope_freqs(64))
    for bad in (lambda: qg.qk_rope(rotary, q, k, i, q_out=wide), lambda: qg.qk_rope(rotary, q, k, i, k_out=q), lambda: qg.qk_rope(rotary, q, None, i, k_out=k),
                lambda: qg.qk_rope(rotary, q, k, i, q_out=q.view(2, 1, 128))):
        with pytest.raises(ValueError):
            bad()
    out = qg.qk_rope(rotary, q, k, i, q_out=wide[:, 64:])
    assert out[0].data_ptr() == wide.data_ptr() + 128 and out[1].shape == k.shape
