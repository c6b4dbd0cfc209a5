"""Refusals of the paged-cache entry points: every argument check runs on the host before any
launch, so it is tested here on the CPU with addresses that are never read."""
import ctypes

import pytest

import dequant_gemv_q4g32_amd as qg

NULL, FMT, SHAPE, ALIGN, RANGE, WORK = -1, -6, -2, -3, -5, -9
P = 0x1000000          # a well-aligned address


def pool(**kw):
    d = dict(pages=P, num_pages=10, layers=2, layer_stride=10 * 34816, kind=1, kv_heads=8, head_dim=128, page_tokens=16)
    d.update(kw)
    return qg._Pool(**d)


BAD_POOLS = [(dict(pages=None), NULL), (dict(pages=P + 8), ALIGN), (dict(num_pages=0), SHAPE), (dict(num_pages=2 ** 31), SHAPE),
             (dict(layers=0), SHAPE), (dict(layers=65536), SHAPE), (dict(layer_stride=10 * 34816 - 16), SHAPE),
             (dict(layer_stride=10 * 34816 + 8), ALIGN), (dict(kind=0), FMT), (dict(kind=3), FMT), (dict(kv_heads=0), SHAPE),
             (dict(kv_heads=1025), SHAPE), (dict(head_dim=32), SHAPE), (dict(head_dim=96), SHAPE), (dict(page_tokens=8), SHAPE),
             (dict(page_tokens=48), SHAPE), (dict(page_tokens=512), SHAPE)]


def rows(name, pl, layer=0, table=P, ld=4, trows=3, tpages=4, k=P, ldk=1024, v=P, ldv=1024, seqs=P, pos=P, count=5):
    return getattr(qg.lib, name)(ctypes.addressof(pl) if pl else None, layer, table, ld, trows, tpages, k, ldk, v, ldv, seqs,
                                 pos, count, None)


def attn(pl, layer=0, q=P, ldq=4096, table=P, ld=512, lens=P, batch=3, heads=32, max_len=8192, window=0, scale=0.1, out=P,
         ldo=4096, f32=0, lse=P, ws=P, size=None):
    ref = ctypes.addressof(pl) if pl else None
    if size is None:
        got = ctypes.c_int64()
        size = got.value if qg.lib.qg_paged_attention_bytes(ref, batch, heads, max_len, ctypes.byref(got)) == 0 else 0
        size = got.value
    return qg.lib.qg_paged_attention(ref, layer, q, ldq, table, ld, lens, batch, heads, max_len, window, scale, out, ldo, f32,
                                     lse, ws, size, None)


def fork(pl, table=P, ld=4, trows=3, tpages=4, lens=P, refs=P, src=P, dst=P, new=P, count=2):
    return qg.lib.qg_kv_fork(ctypes.addressof(pl) if pl else None, table, ld, trows, tpages, lens, refs, src, dst, new, count,
                             None)


def free(pl, table=P, ld=4, trows=3, tpages=4, lens=P, refs=P, rows_=P, count=2):
    return qg.lib.qg_kv_free(ctypes.addressof(pl) if pl else None, table, ld, trows, tpages, lens, refs, rows_, count, None)


def copy(pl, src=P, dst=P, count=2):
    return qg.lib.qg_kv_copy_pages(ctypes.addressof(pl) if pl else None, src, dst, count, None)


def compact(pl, table=P, ld=4, out=P, ldo=4, trows=3, tpages=4, refs=P, refs_out=P, remap=P, live=P, ws=P, size=1 << 20):
    return qg.lib.qg_kv_compact(ctypes.addressof(pl) if pl else None, table, ld, out, ldo, trows, tpages, refs, refs_out, remap,
                                live, ws, size, None)


CALLS = [lambda p, **k: rows("qg_kv_append", p, **k), lambda p, **k: rows("qg_kv_gather", p, **k), attn, fork, free, copy, compact]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("bad,status", BAD_POOLS)
def test_entry_point_pools(call, bad, status):
    assert call(pool(**bad)) == status


@pytest.mark.parametrize("call", CALLS)
def test_entry_point_no_pool(call):
    assert call(None) == NULL


@pytest.mark.parametrize("name", ["qg_kv_append", "qg_kv_gather"])
@pytest.mark.parametrize("bad,status", [
    (dict(layer=-1), SHAPE), (dict(layer=2), SHAPE), (dict(table=None), NULL), (dict(table=P + 2), ALIGN), (dict(ld=3), SHAPE),
    (dict(trows=-1), SHAPE), (dict(tpages=-1), SHAPE), (dict(k=None), NULL), (dict(v=None), NULL), (dict(pos=None), NULL),
    (dict(k=P + 8), ALIGN), (dict(v=P + 2), ALIGN), (dict(seqs=P + 1), ALIGN), (dict(pos=P + 1), ALIGN), (dict(ldk=1020), SHAPE),
    (dict(ldv=1028), ALIGN), (dict(count=-1), SHAPE), (dict(count=2 ** 24 + 1), SHAPE)])
def test_entry_point_rows(name, bad, status):
    assert rows(name, pool(), **bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(layer=2), SHAPE), (dict(q=None), NULL), (dict(lens=None), NULL), (dict(out=None), NULL), (dict(ws=None), NULL),
    (dict(table=None), NULL), (dict(q=P + 8), ALIGN), (dict(out=P + 4), ALIGN), (dict(lens=P + 2), ALIGN), (dict(lse=P + 2), ALIGN),
    (dict(ws=P + 8), ALIGN), (dict(ldq=4095), SHAPE), (dict(ldq=4100), ALIGN), (dict(ldo=4090), SHAPE), (dict(ldo=4100), ALIGN),
    (dict(ldo=4102, f32=1), ALIGN), (dict(heads=0), SHAPE), (dict(heads=33), SHAPE), (dict(batch=-1), SHAPE),
    (dict(batch=2 ** 20), SHAPE), (dict(max_len=-1), SHAPE), (dict(max_len=2 ** 30 + 1), SHAPE), (dict(max_len=8193), SHAPE),
    (dict(window=-1), SHAPE), (dict(scale=float("inf")), RANGE), (dict(scale=float("nan")), RANGE), (dict(size=0), WORK)])
def test_entry_point_attention(bad, status):
    assert attn(pool(), **bad) == status


def test_entry_point_attention_workspace_one_byte_short():
    got = ctypes.c_int64()
    p = pool()
    assert qg.lib.qg_paged_attention_bytes(ctypes.addressof(p), 3, 32, 8192, ctypes.byref(got)) == 0 and got.value > 0
    assert attn(p, size=got.value - 1) == WORK
    assert qg.lib.qg_paged_attention_bytes(ctypes.addressof(p), 3, 32, 128, None) == NULL
    assert qg.lib.qg_paged_attention_bytes(ctypes.addressof(p), 3, 31, 128, ctypes.byref(got)) == SHAPE
    assert qg.lib.qg_paged_attention_bytes(ctypes.addressof(p), 3, 32, 128, ctypes.byref(got)) == 0 and got.value == 0


@pytest.mark.parametrize("call,names", [(fork, ["lens", "refs", "src", "dst", "new"]), (free, ["lens", "refs", "rows_"]),
                                        (copy, ["src", "dst"])])
def test_entry_point_page_operations(call, names):
    for n in names:
        assert call(pool(), **{n: None}) == NULL, n
        assert call(pool(), **{n: P + 2}) == ALIGN, n
    assert call(pool(), count=-1) == SHAPE
    assert call(pool(), count=4097 if call is fork else 2 ** 23 + 1) == SHAPE
    if call is not copy:
        assert call(pool(), ld=3) == SHAPE
        assert call(pool(), table=None) == NULL


def test_entry_point_compact():
    for n in ("refs", "refs_out", "remap", "live", "ws", "table", "out"):
        assert compact(pool(), **{n: None}) == NULL, n
        assert compact(pool(), **{n: P + 2}) == ALIGN, n
    assert compact(pool(), ld=3) == SHAPE and compact(pool(), ldo=3) == SHAPE
    got = ctypes.c_int64()
    p = pool()
    assert qg.lib.qg_kv_compact_bytes(ctypes.addressof(p), ctypes.byref(got)) == 0
    assert compact(p, size=got.value - 1) == WORK
    big = pool(num_pages=2 ** 24 + 1, layers=1)
    assert compact(big) == SHAPE and qg.lib.qg_kv_compact_bytes(ctypes.addressof(big), ctypes.byref(got)) == SHAPE


@pytest.mark.parametrize("call,kw", [(lambda p, **k: rows("qg_kv_append", p, **k), dict(count=0, k=None, v=None, pos=None)),
                                     (lambda p, **k: rows("qg_kv_gather", p, **k), dict(count=0, k=None, v=None, pos=None)),
                                     (attn, dict(batch=0, q=None, out=None, lens=None, table=None)),
                                     (fork, dict(count=0, src=None)), (free, dict(trows=0, table=None)),
                                     (copy, dict(count=0, src=None, dst=None))])
def test_entry_point_nothing_to_do(call, kw):
    assert call(pool(), **kw) == 0


def test_workspace_status_text():
    assert qg.lib.qg_strerror(-9) != b"unknown status"


@pytest.mark.parametrize("scale", [3.0e38, -3.0e38])
def test_entry_point_attention_scale_past_fp32(scale):
    """scale * log2(e) has to be a number: 2.4e38 is the largest scale."""
    assert attn(pool(), scale=scale) == RANGE
