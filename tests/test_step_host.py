"""Refusals of a decode step's entry points (places for tokens, norm and rotation) and the host's
frequencies, on the CPU: every argument is checked before any launch, so the addresses are never read."""
import ctypes
import types

import numpy as np
import pytest

import dequant_gemv_q4g32_amd as qg
from oracle import step

torch = pytest.importorskip("torch")

NULL, FMT, SHAPE, ALIGN, RANGE, WORK = -1, -6, -2, -3, -5, -9
P = 0x1000000          # a well-aligned address


def pool(**kw):
    d = dict(pages=P, num_pages=10, layers=2, layer_stride=10 * 34816, kind=1, kv_heads=8, head_dim=128, page_tokens=16)
    d.update(kw)
    return qg._Pool(**d)


def rotary(**kw):
    d = dict(freqs=P, q_weight=P, k_weight=P, eps=1e-6, factor=1.0, rotary_dim=128, interleaved=0)
    d.update(kw)
    return qg._Rotary(**d)


def ref(s):
    return ctypes.addressof(s) if s else None


def extend(pl, table=P, ld=4, trows=3, tpages=4, lens=P, refs=P, add=P, granted=P, starts=P, seqs=P, pos=P, slots=7, ws=P, size=1 << 20):
    return qg.lib.qg_kv_extend(ref(pl), table, ld, trows, tpages, lens, refs, add, granted, starts, seqs, pos, slots, ws, size, None)


def trim(pl, table=P, ld=4, trows=3, tpages=4, lens=P, refs=P, to=P):
    return qg.lib.qg_kv_trim(ref(pl), table, ld, trows, tpages, lens, refs, to, None)


def append(pl, rot=rotary(), layer=0, table=P, ld=4, trows=3, tpages=4, heads=32, q=P, ldq=6144, k=P, ldk=1024, v=P, ldv=1024,
           seqs=P, pos=P, count=5, out=P, ldo=4096):
    return qg.lib.qg_kv_append_rope(ref(pl), layer, table, ld, trows, tpages, ref(rot), heads, q, ldq, k, ldk, v, ldv, seqs, pos,
                                    count, out, ldo, None)


def dense(rot=rotary(), dim=128, heads=32, kv_heads=8, q=P, ldq=6144, k=P, ldk=1024, pos=P, count=5, out=P, ldo=4096, kout=P, ldko=1024):
    return qg.lib.qg_qk_rope(ref(rot), dim, heads, kv_heads, q, ldq, k, ldk, pos, count, out, ldo, kout, ldko, None)


BAD_POOLS = [(dict(pages=None), NULL), (dict(pages=P + 8), ALIGN), (dict(num_pages=0), SHAPE), (dict(layers=0), SHAPE),
             (dict(layer_stride=10 * 34816 - 16), SHAPE), (dict(kind=3), FMT), (dict(kv_heads=0), SHAPE), (dict(head_dim=96), SHAPE),
             (dict(page_tokens=48), SHAPE)]


@pytest.mark.parametrize("call", [extend, trim, append])
def test_pools(call):
    for bad, status in BAD_POOLS:
        assert call(pool(**bad)) == status, bad
    assert call(None) == NULL
    for bad, status in [(dict(table=None), NULL), (dict(table=P + 2), ALIGN), (dict(ld=3), SHAPE), (dict(trows=-1), SHAPE),
                        (dict(tpages=-1), SHAPE)]:
        assert call(pool(), **bad) == status, bad


def test_extend():
    for n in ("refs", "lens", "add", "granted", "seqs", "pos", "ws"):
        assert extend(pool(), **{n: None}) == NULL, n
        assert extend(pool(), **{n: P + 2}) == ALIGN, n
    assert extend(pool(), starts=P + 2) == ALIGN
    assert extend(pool(), slots=-1) == SHAPE and extend(pool(), slots=2 ** 26 + 1) == SHAPE
    assert extend(pool(), trows=65537) == SHAPE and extend(pool(num_pages=2 ** 24 + 1, layers=1)) == SHAPE
    got = ctypes.c_int64()
    p = pool()
    assert qg.lib.qg_kv_extend_bytes(ref(p), 3, ctypes.byref(got)) == 0 and got.value > 0
    assert extend(p, size=got.value - 1) == WORK
    assert qg.lib.qg_kv_extend_bytes(ref(p), 3, None) == NULL
    assert qg.lib.qg_kv_extend_bytes(ref(p), 65537, ctypes.byref(got)) == SHAPE
    assert qg.lib.qg_kv_extend_bytes(ref(p), -1, ctypes.byref(got)) == SHAPE


def test_trim():
    for n in ("refs", "lens", "to"):
        assert trim(pool(), **{n: None}) == NULL, n
        assert trim(pool(), **{n: P + 2}) == ALIGN, n
    assert trim(pool(), trows=0, table=None, lens=None) == 0
    assert trim(pool(), trows=65537) == SHAPE


ROTARIES = [(dict(freqs=None), NULL), (dict(freqs=P + 4), ALIGN), (dict(q_weight=P + 8), ALIGN), (dict(k_weight=P + 8), ALIGN),
            (dict(rotary_dim=130), SHAPE), (dict(rotary_dim=144), SHAPE), (dict(rotary_dim=24), SHAPE), (dict(rotary_dim=-16), SHAPE),
            (dict(eps=0.0), RANGE), (dict(eps=-1.0), RANGE), (dict(eps=float("nan")), RANGE), (dict(eps=float("inf")), RANGE),
            (dict(eps=1e-40), RANGE), (dict(eps=0.0, q_weight=None), RANGE), (dict(factor=float("inf")), RANGE),
            (dict(factor=float("nan")), RANGE)]


def test_rotaries():
    for bad, status in ROTARIES:
        assert append(pool(), rotary(**bad)) == status, bad
        assert dense(rotary(**bad)) == status, bad
    assert append(pool(), None) == NULL and dense(None) == NULL


def test_append_rows():
    for bad, status in [(dict(layer=-1), SHAPE), (dict(layer=2), SHAPE), (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL),
                        (dict(out=None), NULL), (dict(pos=None), NULL), (dict(q=P + 8), ALIGN), (dict(k=P + 2), ALIGN), (dict(v=P + 8), ALIGN),
                        (dict(out=P + 8), ALIGN), (dict(pos=P + 1), ALIGN), (dict(seqs=P + 2), ALIGN), (dict(ldq=4088), SHAPE),
                        (dict(ldq=4100), ALIGN), (dict(ldk=1020), SHAPE), (dict(ldv=1028), ALIGN), (dict(ldo=4088), SHAPE),
                        (dict(ldo=4100), ALIGN), (dict(count=-1), SHAPE), (dict(count=2 ** 23 + 1), SHAPE), (dict(heads=-1), SHAPE),
                        (dict(heads=65537), SHAPE)]:
        assert append(pool(), **bad) == status, bad
    assert append(pool(), count=0, q=None, k=None, pos=None) == 0


def test_dense_rows():
    for bad, status in [(dict(dim=96), SHAPE), (dict(q=None), NULL), (dict(k=None), NULL), (dict(out=None), NULL), (dict(kout=None), NULL),
                        (dict(pos=None), NULL), (dict(q=P + 8), ALIGN), (dict(k=P + 8), ALIGN), (dict(out=P + 2), ALIGN),
                        (dict(kout=P + 2), ALIGN), (dict(pos=P + 2), ALIGN), (dict(ldq=4088), SHAPE), (dict(ldk=1028), ALIGN),
                        (dict(ldo=4100), ALIGN), (dict(ldko=1016), SHAPE), (dict(count=-1), SHAPE), (dict(count=2 ** 23 + 1), SHAPE),
                        (dict(heads=-1), SHAPE), (dict(kv_heads=-1), SHAPE), (dict(kv_heads=65537), SHAPE)]:
        assert dense(**bad) == status, bad
    assert dense(count=0, q=None) == 0 and dense(heads=0, kv_heads=0, q=None, k=None, pos=None) == 0


@pytest.mark.parametrize("kind,args", [("plain", {}), ("linear", dict(scale=4.0)), ("base", dict(scale=8.0)),
                                       ("turns", dict(scale=8.0, context=8192, low=1.0, high=4.0)),
                                       ("parts", dict(scale=16.0, context=4096, low=1.0, high=32.0)),
                                       ("parts", dict(scale=2.0, context=10, low=1.0, high=32.0))])
@pytest.mark.parametrize("dim,base", [(64, 10000.0), (128, 500000.0), (48, 10000.0), (6, 10.0)])
def test_freqs_match_oracle(kind, args, dim, base):
    """Both sides are fp64; a power of base up to 2^19 carries |exponent| * 2^-52 relative, 32 steps with room."""
    got, want = qg.rope_freqs(dim, base, kind, **args), step.freqs(kind, dim, base, **args)
    assert got.dtype == np.float64 and np.allclose(got, want, rtol=2.0 ** -47, atol=0)


def test_freqs_refusals():
    out = (ctypes.c_double * 64)()
    call = lambda kind=4, dim=64, base=1e4, scale=2.0, context=4096.0, low=1.0, high=32.0, to=out: qg.lib.qg_rope_freqs(
        kind, dim, base, scale, context, low, high, to)
    assert call() == 0
    for bad, status in [(dict(to=None), NULL), (dict(kind=-1), FMT), (dict(kind=5), FMT), (dict(dim=0), SHAPE), (dict(dim=63), SHAPE),
                        (dict(dim=-2), SHAPE), (dict(kind=2, dim=2), SHAPE), (dict(base=1.0), RANGE), (dict(base=float("inf")), RANGE),
                        (dict(base=float("nan")), RANGE), (dict(scale=0.0), RANGE), (dict(scale=float("nan")), RANGE),
                        (dict(context=0.0), RANGE), (dict(context=float("inf")), RANGE), (dict(low=0.0), RANGE),
                        (dict(high=1.0), RANGE), (dict(high=float("inf")), RANGE), (dict(low=float("nan")), RANGE)]:
        assert call(**bad) == status, bad
    assert call(kind=0, scale=float("nan"), context=0.0) == 0    # not read by the plain frequencies
    with pytest.raises(qg.QGError):
        qg.rope_freqs(63)


def test_stream_of_another_device_is_refused():
    pl = types.SimpleNamespace(device=torch.device("cuda", 0), _index=0)
    other = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=64)
    x = None
    for call in (lambda: qg.kv_extend(pl, x, x, x, x, 4, stream=other), lambda: qg.kv_trim(pl, x, x, x, x, stream=other),
                 lambda: qg.kv_append_rope(pl, x, x, x, x, x, x, stream=other)):
        with pytest.raises(ValueError, match="stream"):
            call()


def test_rotary_refusals():
    for bad in (dict(freqs=np.ones(8), device="cpu"), dict(q_weight=torch.ones(64)), dict(q_weight=torch.ones(32, dtype=torch.float16)),
                dict(q_weight=torch.ones(64, dtype=torch.float16)), dict(freqs=torch.ones(8))):
        with pytest.raises(ValueError):
            qg.Rotary(64, **bad)
    with pytest.raises(ValueError, match="GPU"):
        qg.qk_rope(None, torch.ones(2, 64, dtype=torch.float16), None, None)
