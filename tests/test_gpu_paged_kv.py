"""GPU tests of the paged cache's writes, reads and page operations against oracle/paged.py.

Bar: every byte of the pool, the tables, the counts and the gathered rows equals the oracle's:
the codec's codes and scales have one right answer, and everything else is moved, not computed.
Pools start as random bytes, so a write outside the named places shows as a difference.
"""
import numpy as np
import pytest

import dequant_gemv_q4g32_amd as qg
from oracle import paged

from paged_util import assert_same_bytes, dev, download, random_cache, random_table, upload

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _rows(rng, count, cols, ld):
    x = rng.standard_normal((count, cols)) * rng.choice([1e-4, 0.05, 1.0, 40.0], size=(count, 1))
    x.reshape(-1)[:: max(1, x.size // 7)] *= 50.0
    x = np.clip(x, -65000, 65000).astype(np.float16)
    buf = torch.full((count, ld), 3.0, dtype=torch.float16, device="cuda")
    buf[:, :cols] = torch.from_numpy(x).cuda()
    return x, buf[:, :cols]


CASES = [  # kind, heads, dim, tokens, layers, rows appended, ld beyond the columns
    ("q8", 1, 64, 16, 1, 1, 0), ("q8", 8, 128, 16, 2, 37, 8), ("q8", 3, 256, 64, 1, 20, 0), ("q8", 5, 64, 256, 3, 300, 24),
    ("f16", 1, 64, 16, 1, 1, 0), ("f16", 8, 128, 32, 2, 37, 8), ("f16", 2, 256, 128, 1, 150, 0)]


@pytest.mark.parametrize("kind,heads,dim,tokens,layers,count,extra", CASES)
def test_append_and_gather(kind, heads, dim, tokens, layers, count, extra):
    rng = np.random.default_rng(count * 31 + dim)
    lens = [tokens * 2 + 3, 1, 0, count + tokens]
    width = -(-max(lens) // tokens) + 1
    c = random_cache(kind, layers, 4 * width + 2, heads, dim, tokens, 5, poison=True)
    pool = upload(c)
    table = random_table(rng, lens, tokens, c.pages, width)
    table[0, 1] = c.pages                               # an entry past the pool: names no page
    # rows at distinct places, and rows without one: negative and far positions, bad rows, holes
    places = [(s, p) for s in range(4) for p in range(width * tokens)]
    pick = [places[i] for i in rng.permutation(len(places))[:count]]
    bad = [(-1, 0), (4, 0), (0, -1), (3, width * tokens), (3, 2 ** 31 - 1), (2 ** 31 - 1, 0), (0, -2 ** 31)]
    seqs, pos = (np.array(x, np.int32) for x in zip(*(pick + bad)))
    cols = heads * dim
    xk, k = _rows(rng, len(pos), cols, cols + extra)
    xv, v = _rows(rng, len(pos), cols, cols + extra)
    layer = layers - 1
    qg.kv_append(pool, dev(table), k, v, dev(pos), dev(seqs), layer=layer)
    c.append(layer, table, xk, xv, pos, seqs)
    torch.cuda.synchronize()
    assert_same_bytes(download(c, pool), c, "pool")
    # back, with repeated rows, into strided buffers
    again = np.concatenate([np.arange(len(pos)), np.arange(len(pos))[::-1][: 5]])
    outs = [torch.full((len(again), cols + 8), 7.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    qg.kv_gather(pool, dev(table), dev(pos[again]), dev(seqs[again]), k=outs[0][:, :cols], v=outs[1][:, :cols], layer=layer)
    want = c.gather(layer, table, pos[again], seqs[again])
    for i in (0, 1):
        got = outs[i].cpu().numpy()
        assert np.array_equal(got[:, :cols].view(np.uint16), want[i].view(np.uint16)), f"gathered {'kv'[i]}"
        assert np.all(got[:, cols:] == 7.0)


def test_append_without_seqs_is_row_by_row():
    """The decode form: row i is sequence i, padded rows have position -1."""
    rng = np.random.default_rng(3)
    c = random_cache("q8", 1, 12, 2, 128, 16, 6, poison=True)
    pool = upload(c, layers_dim=False)
    pos = np.array([0, 15, -1, 16, 31], np.int32)
    table = random_table(rng, pos + 1, 16, 12, 2)
    xk, k = _rows(rng, 5, 256, 256)
    xv, v = _rows(rng, 5, 256, 256)
    qg.kv_append(pool, dev(table), k, v, dev(pos))
    c.append(0, table, xk, xv, pos)
    gk, gv = qg.kv_gather(pool, dev(table), dev(pos))
    want = c.gather(0, table, pos)
    assert_same_bytes(download(c, pool), c)
    assert np.array_equal(gk.cpu().numpy(), want[0]) and np.array_equal(gv.cpu().numpy(), want[1])
    assert np.all(want[:, 2] == 0)


def test_append_special_groups():
    """The codec's corner cases in a page: ties, the fp16 maximum, subnormals, empty groups."""
    import json
    import os
    groups = json.load(open(os.path.join(os.path.dirname(__file__), "golden", "kvcache_groups.json")))["groups"]
    n = len(groups) + len(groups) % 2
    x = np.zeros((n, 32), np.float16)
    for i, g in enumerate(groups):
        for j, val in g["values"].items():
            x[i, int(j)] = val
    x = x.reshape(-1, 64)
    count = x.shape[0]
    c = random_cache("q8", 1, 3, 1, 64, 16, 9, poison=True)
    assert count <= 48
    table = np.array([[2, 0, 1]], np.int32)
    pool = upload(c)
    pos, seqs = np.arange(count, dtype=np.int32), np.zeros(count, np.int32)
    k = torch.from_numpy(x).cuda()
    qg.kv_append(pool, dev(table), k, k.flip(0), dev(pos), dev(seqs))
    c.append(0, table, x, x[::-1], pos, seqs)
    gk, gv = qg.kv_gather(pool, dev(table), dev(pos), dev(seqs))
    want = c.gather(0, table, pos, seqs)
    assert_same_bytes(download(c, pool), c)
    assert np.array_equal(gk.cpu().numpy().view(np.uint16), want[0].view(np.uint16))
    assert np.array_equal(gv.cpu().numpy().view(np.uint16), want[1].view(np.uint16))
    assert np.all(np.isfinite(want.astype(np.float32)))


def test_empty_calls_change_nothing():
    c = random_cache("q8", 1, 4, 1, 64, 16, 2, poison=True)
    pool = upload(c)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    rows = torch.empty((0, 64), dtype=torch.float16, device="cuda")
    table, lens, refs = dev([[0, 1]]), dev([20]), dev([1, 1, 0, 0])
    qg.kv_append(pool, table, rows, rows, none)
    k, v = qg.kv_gather(pool, table, none)
    qg.kv_copy_pages(pool, none, none)
    qg.kv_fork(pool, table, lens, refs, none, none, none)
    qg.kv_free(pool, table, lens, refs, none)
    assert k.shape == v.shape == (0, 64)
    assert_same_bytes(download(c, pool), c)
    assert table.tolist() == [[0, 1]] and lens.tolist() == [20] and refs.tolist() == [1, 1, 0, 0]


@pytest.mark.parametrize("kind,heads,dim,tokens,layers,pages", [
    ("q8", 1, 64, 16, 1, 9), ("q8", 8, 128, 16, 3, 40), ("f16", 3, 256, 256, 2, 12), ("f16", 1, 64, 16, 5, 33)])
def test_copy_pages(kind, heads, dim, tokens, layers, pages):
    rng = np.random.default_rng(pages)
    c = random_cache(kind, layers, pages, heads, dim, tokens, 4, poison=True)
    pool = upload(c)
    order = rng.permutation(pages)
    n = pages // 3
    src, dst = list(order[:n]) + [order[0]], list(order[n:2 * n + 1])          # one page copied twice
    bad = [(-1, int(order[-1])), (int(order[-1]), -1), (pages, int(order[-1])), (int(order[-1]), pages), (2 ** 31 - 1, 0)]
    src, dst = (np.array(a, np.int32) for a in zip(*(list(zip(src, dst)) + bad + [(order[-2], order[-2])])))
    qg.kv_copy_pages(pool, dev(src), dev(dst))
    for s, d in zip(src, dst):
        if 0 <= s < pages and 0 <= d < pages:
            c.copy_page(s, d)
    assert_same_bytes(download(c, pool), c)


def _state(kind, heads, dim, tokens, layers, lens, spare, width, seed):
    rng = np.random.default_rng(seed)
    pages = sum(-(-n // tokens) for n in lens) + spare
    c = random_cache(kind, layers, pages, heads, dim, tokens, seed, poison=True)
    table = random_table(rng, lens, tokens, pages, width)
    refs = np.zeros(pages, np.int32)
    refs[table[table >= 0]] = 1
    return rng, c, table, np.array(lens, np.int32), refs


@pytest.mark.parametrize("kind,heads,dim,tokens,layers,lens", [
    ("q8", 2, 128, 16, 2, [33, 16, 1, 0, 48, 40, 17, 0]), ("f16", 1, 64, 32, 1, [700, 0, 32, 9999, 64]),
    ("f16", 8, 128, 64, 3, [65, 127, 128, 1])])
def test_fork_and_free(kind, heads, dim, tokens, layers, lens):
    width = -(-max(lens) // tokens) + 2
    rng, c, table, lens, refs = _state(kind, heads, dim, tokens, layers, lens, 6, width, 11)
    pool, t, n, r = upload(c), dev(table), dev(lens), dev(refs)
    free_pages = np.flatnonzero(refs == 0).astype(np.int32)
    rows = len(lens)

    def same(what):
        torch.cuda.synchronize()
        assert_same_bytes(download(c, pool), c, what)
        assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(n.cpu().numpy(), lens), what
        assert np.array_equal(r.cpu().numpy(), refs), what

    def step(src, dst, fresh, gone, what):
        src, dst, fresh, gone = (np.array(x, np.int32) for x in (src, dst, fresh, gone))
        qg.kv_free(pool, t, n, r, dev(gone))
        paged.free(c, table, lens, refs, gone)
        same(what + " free")
        qg.kv_fork(pool, t, n, r, dev(src), dev(dst), dev(fresh))
        paged.fork(c, table, lens, refs, src, dst, fresh)
        same(what + " fork")

    step([0, 0], [rows - 1, rows - 2], free_pages[:2], [rows - 1, rows - 2], "two of one")
    step([rows - 1], [1], free_pages[2:3], [1, 1, rows, -1, 2 ** 31 - 1], "of a fork, row freed twice, rows outside")
    # skipped: rows outside, a row onto itself, a row that is a source, a row named twice, pages outside or named twice
    step([0, 0, 0, 0, 0, 0, -1, rows], [rows, -1, 0, 2, 2, 1, 2, 2],
         [free_pages[3], free_pages[4], free_pages[4], c.pages, free_pages[5], free_pages[5], 0, 0], [2, 1], "skipped")
    step([], [], [], np.arange(rows), "everything")
    assert np.all(refs <= 1) and np.all(lens <= 0)


def test_fork_lens_and_entries_outside():
    """Lengths below 0 and past the table, holes in the source row, a row filled to its last entry."""
    rng, c, table, lens, refs = _state("f16", 1, 64, 16, 1, [32, 20, 7, 0, 0, 0], 4, 2, 5)
    table[1, 0] = -1
    table[2, 0] = 99
    lens[0], lens[5] = 1000, -4
    pool, t, n, r = upload(c), dev(table), dev(lens), dev(refs)
    fresh = np.flatnonzero(refs == 0).astype(np.int32)[:4]
    src, dst = np.array([0, 1, 2], np.int32), np.array([3, 4, 5], np.int32)
    qg.kv_fork(pool, t, n, r, dev(src), dev(dst), dev(fresh[:3]))
    paged.fork(c, table, lens, refs, src, dst, fresh[:3])
    assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(n.cpu().numpy(), lens)
    assert np.array_equal(r.cpu().numpy(), refs)
    assert_same_bytes(download(c, pool), c)


@pytest.mark.parametrize("kind,heads,dim,tokens,layers,pages,share,in_place", [
    ("q8", 1, 64, 16, 1, 1, 1.0, False), ("q8", 1, 64, 16, 1, 5, 0.0, False), ("f16", 2, 64, 16, 2, 64, 0.5, False),
    ("q8", 8, 128, 16, 3, 77, 0.7, True), ("f16", 1, 64, 16, 1, 1024, 0.3, True), ("q8", 1, 64, 16, 2, 2500, 0.6, False),
    ("f16", 1, 64, 16, 1, 9001, 0.45, True), ("q8", 2, 128, 16, 1, 300, 1.0, False)])
def test_compact(kind, heads, dim, tokens, layers, pages, share, in_place):
    rng = np.random.default_rng(pages)
    c = random_cache(kind, layers, pages, heads, dim, tokens, 8, poison=True)
    refs = (rng.random(pages) < share).astype(np.int32) * rng.integers(1, 5, pages).astype(np.int32)
    refs[refs == 0] = rng.choice([0, 0, -3], int((refs == 0).sum()))
    table = rng.integers(-2, pages + 2, (7, 41)).astype(np.int32)
    table[0, :2] = [2 ** 31 - 1, -2 ** 31]
    pool, t, r = upload(c), dev(table), dev(refs)
    out = qg.kv_compact(pool, t, r, table_out=t if in_place else None, refs_out=r if in_place else None)
    want = paged.compact(c, table, refs)
    torch.cuda.synchronize()
    for got, ref, name in zip(out, want, ("table", "refs", "remap", "live")):
        assert np.array_equal(got.cpu().numpy().reshape(np.shape(ref)), ref), name
    if not in_place:
        assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(r.cpu().numpy(), refs)
    assert_same_bytes(download(c, pool), c)


def test_strided_tables_and_layers():
    """A table that is a slice of a wider one, and layers with a gap between them."""
    rng, c, table, lens, refs = _state("q8", 2, 64, 16, 2, [20, 5, 0, 0], 3, 3, 17)
    packed = torch.from_numpy(c.pack()).cuda()
    wide = torch.full((2, c.pages + 3, packed.shape[2]), 0x5A, dtype=torch.uint8, device="cuda")
    wide[:, :c.pages] = packed
    pool = qg.KVPool(wide[:, :c.pages], "q8", 2, 64, 16)
    wt = torch.full((4, 8), 77, dtype=torch.int32, device="cuda")
    wt[:, 2:5] = dev(table)
    t = wt[:, 2:5]
    n, r = dev(lens), dev(refs)
    fresh = np.flatnonzero(refs == 0).astype(np.int32)
    src, dst = np.array([0, 1], np.int32), np.array([2, 3], np.int32)
    qg.kv_fork(pool, t, n, r, dev(src), dev(dst), dev(fresh[:2]))
    paged.fork(c, table, lens, refs, src, dst, fresh[:2])
    assert_same_bytes(download(c, pool), c, "fork")
    gone = np.array([0], np.int32)
    qg.kv_free(pool, t, n, r, dev(gone))
    paged.free(c, table, lens, refs, gone)
    out = qg.kv_compact(pool, t, r, table_out=t, refs_out=r)
    table, refs, remap, live = paged.compact(c, table, refs)
    assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(r.cpu().numpy(), refs)
    assert_same_bytes(download(c, pool), c, "compact")
    assert np.all(wide[:, c.pages:].cpu().numpy() == 0x5A) and np.all(wt[:, [0, 1, 5, 6, 7]].cpu().numpy() == 77)
