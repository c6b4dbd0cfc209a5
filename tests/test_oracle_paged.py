"""The paged-cache oracle (oracle/paged.py) against hand-worked cases, and its record layout
against the sizes the library states. CPU only."""
import numpy as np
import pytest

import dequant_gemv_q4g32_amd as qg
from oracle import kvcache, paged


@pytest.mark.parametrize("kind", ["q8", "f16"])
def test_pack_layout_and_round_trip(kind):
    c = paged.Cache(kind, 2, 3, 2, 64, 16)
    rng = np.random.default_rng(1)
    for a in c._arrays:
        a.view(np.uint8)[...] = rng.integers(0, 256, a.view(np.uint8).shape, dtype=np.uint8)
    p = c.pack()
    assert p.shape == (2, 3, qg.kv_page_bytes(kind, 2, 64, 16))
    again = paged.Cache(kind, 2, 3, 2, 64, 16).unpack(p)
    for a, b in zip(c._arrays, again._arrays):
        assert np.array_equal(a.view(np.uint8), b.view(np.uint8))
    head = p[1, 2].reshape(2, -1)[1]                     # layer 1, page 2, head 1
    if kind == "q8":
        assert np.array_equal(head[5 * 64:6 * 64].view(np.int8), c.codes[0][1, 2, 1, 5])
        assert np.array_equal(head[1024 + 5 * 64:1024 + 6 * 64].view(np.int8), c.codes[1][1, 2, 1, 5])
        scales = head[2048:].view(np.uint16)
        assert scales[5 * 2 + 1] == c.scales[0].view(np.uint16)[1, 2, 1, 5, 1]
        assert scales[32 + 1 * 16 + 5] == c.scales[1].view(np.uint16)[1, 2, 1, 5, 1]
    else:
        assert np.array_equal(head[2 * 5 * 64:2 * 6 * 64].view(np.uint16), c.values[0].view(np.uint16)[1, 2, 1, 5])


def test_page_bytes():
    assert qg.kv_page_bytes("q8", 8, 128, 16) == 8 * 16 * (2 * 128 + 2 * 2 * 4)
    assert qg.kv_page_bytes("f16", 3, 256, 64) == 3 * 64 * 2 * 2 * 256
    for bad in [(0, 8, 128, 16), (3, 8, 128, 16), (1, 0, 128, 16), (1, 1025, 128, 16), (1, 8, 96, 16), (1, 8, 32, 16),
                (1, 8, 512, 16), (1, 8, 128, 8), (1, 8, 128, 24), (1, 8, 128, 512)]:
        import ctypes
        out = ctypes.c_int64(-5)
        assert qg.lib.qg_kv_page_bytes(*bad, ctypes.byref(out)) == (-6 if bad[0] in (0, 3) else -2)
        assert out.value == -5
    assert qg.lib.qg_kv_page_bytes(1, 8, 128, 16, None) == -1


def test_append_gather_attention_by_hand():
    c = paged.Cache("q8", 1, 2, 1, 64, 16)
    table = np.array([[1, -1], [0, 7]], np.int32)
    k = np.zeros((4, 64), np.float16)
    v = np.zeros((4, 64), np.float16)
    k[0, 0], v[0, :] = 127, 2                    # sequence 0, token 0
    k[1, 0], v[1, :] = 0, 4                      # sequence 0, token 1
    k[2, 0], v[2, :] = 127, 8                    # sequence 1, token 15
    v[3, :] = 99                                 # no place: position -1
    c.append(0, table, k, v, [0, 1, 15, -1], [0, 0, 1, 1])
    assert c.codes[0][0, 1, 0, 0, 0] == 127 and c.scales[0][0, 1, 0, 0, 0] == 1.0
    got = c.gather(0, table, [15, 0, 16, 16], [1, 0, 1, 0])
    assert got[0, 0, 0] == 127 and got[0, 1, 0] == 127
    assert np.all(got[1, 0] == kvcache.dequantize_fp16(*kvcache.quantize(v[2:3]))[0]) and np.all(got[:, 2:] == 0)
    q = np.zeros((2, 1, 64), np.float16)
    q[0, 0, 0] = np.float16(np.log(3.0) / 127 * 0.5)
    out, lse, bound, _ = paged.attention(c, 0, q, table, [2, 0], 32, 2.0)
    e = np.exp(2.0 * 127 * float(q[0, 0, 0]))                 # weight of token 0 against token 1's 1
    v0, v1 = (float(c.token(0, 1, 1, t)[0, 0]) for t in (0, 1))
    assert np.allclose(out[0, 0], (e * v0 + v1) / (e + 1), rtol=1e-12) and np.isclose(lse[0, 0], np.log(e + 1))
    assert np.all(out[1] == 0) and lse[1, 0] == -np.inf
    out, _, _, _ = paged.attention(c, 0, q, table, [2, 0], 32, 2.0, window=1)
    assert np.all(out[0, 0] == v1)


def test_fork_free_compact_by_hand():
    c = paged.Cache("f16", 1, 6, 1, 64, 16)
    for p in range(6):
        c.values[0][0, p] = p
    table = np.array([[5, 3, -1], [-1, -1, -1], [-1, -1, -1]], np.int32)
    lens, refs = np.array([20, 0, 0], np.int32), np.array([0, 0, 0, 1, 0, 1], np.int32)
    paged.fork(c, table, lens, refs, [0, 0, 0], [1, 1, 2], [4, 2, 4])      # the second names row 1 again, the third page 4
    assert table.tolist() == [[5, 3, -1], [5, 4, -1], [-1, -1, -1]] and lens.tolist() == [20, 20, 0]
    assert refs.tolist() == [0, 0, 0, 1, 1, 2] and np.all(c.values[0][0, 4] == 3)
    paged.free(c, table, lens, refs, [0, 0, 9])
    assert refs.tolist() == [0, 0, 0, 0, 1, 1] and lens.tolist() == [0, 20, 0] and table[0].tolist() == [-1] * 3
    t, r, remap, live = paged.compact(c, table, refs)
    assert live == 2 and remap.tolist() == [-1, -1, -1, -1, 0, 1] and r.tolist() == [1, 1, 0, 0, 0, 0]
    assert t[1].tolist() == [1, 0, -1] and np.all(c.values[0][0, 0] == 3) and np.all(c.values[0][0, 1] == 5)
