"""Refusals of the attention over shared prefixes, on the CPU: every argument is checked before any
launch, so the addresses are never read."""
import ctypes
import types

import pytest

import dequant_gemv_q4g32_amd as qg

torch = pytest.importorskip("torch")

NULL, FMT, SHAPE, ALIGN, RANGE, WORK = -1, -6, -2, -3, -5, -9
P = 0x1000000          # a well-aligned address


def pool(**kw):
    d = dict(pages=P, num_pages=10, layers=2, layer_stride=10 * 34816, kind=1, kv_heads=8, head_dim=128, page_tokens=16)
    d.update(kw)
    return qg._Pool(**d)


def need(pl, batch=6, heads=32, groups=2, max_len=8192, max_tail=100):
    got = ctypes.c_int64(-1)
    return qg.lib.qg_prefix_attention_bytes(ctypes.addressof(pl) if pl else None, batch, heads, groups, max_len, max_tail,
                                            ctypes.byref(got)), got.value


def call(pl, layer=0, q=P, ldq=4096, table=P, ld=512, lens=P, starts=P, prefix=P, groups=2, batch=6, heads=32, max_len=8192,
         max_tail=100, scale=0.1, out=P, ldo=4096, f32=0, lse=P, ws=P, size=None):
    if size is None:
        size = max(0, need(pl, batch, heads, groups, max_len, max_tail)[1])
    return qg.lib.qg_prefix_attention(ctypes.addressof(pl) if pl else None, layer, q, ldq, table, ld, lens, starts, prefix, groups,
                                      batch, heads, max_len, max_tail, scale, out, ldo, f32, lse, ws, size, None)


def test_pools():
    for bad, status in [(dict(pages=None), NULL), (dict(pages=P + 8), ALIGN), (dict(num_pages=0), SHAPE), (dict(layers=0), SHAPE),
                        (dict(layer_stride=10 * 34816 - 16), SHAPE), (dict(kind=3), FMT), (dict(kv_heads=0), SHAPE),
                        (dict(head_dim=96), SHAPE), (dict(page_tokens=48), SHAPE)]:
        assert call(pool(**bad)) == status and need(pool(**bad))[0] == status, bad
    assert call(None) == NULL and need(None)[0] == NULL
    assert qg.lib.qg_prefix_attention_bytes(ctypes.addressof(pool()), 6, 32, 2, 100, 100, None) == NULL


@pytest.mark.parametrize("bad,status", [
    (dict(layer=2), SHAPE), (dict(layer=-1), SHAPE), (dict(q=None), NULL), (dict(lens=None), NULL), (dict(out=None), NULL),
    (dict(ws=None), NULL), (dict(table=None), NULL), (dict(starts=None), NULL), (dict(prefix=None), NULL), (dict(q=P + 8), ALIGN),
    (dict(out=P + 4), ALIGN), (dict(lens=P + 2), ALIGN), (dict(lse=P + 2), ALIGN), (dict(ws=P + 8), ALIGN), (dict(starts=P + 2), ALIGN),
    (dict(prefix=P + 1), ALIGN), (dict(ldq=4095), SHAPE), (dict(ldq=4100), ALIGN), (dict(ldo=4090), SHAPE), (dict(ldo=4100), ALIGN),
    (dict(ldo=4102, f32=1), ALIGN), (dict(heads=0), SHAPE), (dict(heads=33), SHAPE), (dict(batch=-1), SHAPE), (dict(batch=2 ** 20), SHAPE),
    (dict(max_len=-1), SHAPE), (dict(max_len=2 ** 30 + 1), SHAPE), (dict(max_len=8193), SHAPE), (dict(max_tail=-1), SHAPE),
    (dict(max_tail=2 ** 30 + 1), SHAPE), (dict(groups=-1), SHAPE), (dict(groups=7), SHAPE), (dict(scale=float("inf")), RANGE),
    (dict(scale=float("nan")), RANGE), (dict(scale=3e38), RANGE), (dict(size=0), WORK)])
def test_arguments(bad, status):
    assert call(pool(), **bad) == status


def test_sizes():
    status, size = need(pool())
    assert status == 0 and call(pool(), size=size - 1) == WORK
    assert need(pool(), batch=5000, groups=1024)[0] == SHAPE and need(pool(), batch=5000, groups=1023)[0] == 0
    # the line of tiles stays below 2^31
    assert need(pool(kv_heads=1, num_pages=2 ** 31 - 1, layers=1), batch=2 ** 16, heads=64, groups=1, max_len=2 ** 20)[0] == SHAPE
    # more of anything never needs less
    for name, values in [("batch", (2, 6, 40, 300)), ("max_len", (16, 100, 3000, 8192)), ("max_tail", (0, 10, 1000, 8192))]:
        sizes = [need(pool(), **{name: v})[1] for v in values]
        assert sizes == sorted(sizes), (name, sizes)
    assert call(pool(), batch=0, groups=0, q=None, out=None, lens=None, table=None, starts=None) == 0


def test_workspace_of_many_groups():
    """Partial results: 256 rows for each workgroup and 16 for each of 2048 waves, and of every query row one of its
    shared tokens in either place and one of its own; 500 groups of two rows need no more than one of 1000."""
    rows = 4 * (128 + 2)
    for groups in (1, 500):
        size = need(pool(kv_heads=16, layer_stride=10 * 69632), batch=1000, heads=64, groups=groups)[1]
        assert size < 1.05 * rows * (256 * 256 + 2048 * 16 + 2 * 1000 * 64 + 4 * 2048 + 1000 * 64), (groups, size)


def test_stream_of_another_device_is_refused():
    pl = types.SimpleNamespace(device=torch.device("cuda", 0), _index=0)
    other = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=64)
    with pytest.raises(ValueError, match="stream"):
        qg.prefix_attention(pl, None, None, None, None, None, stream=other)
