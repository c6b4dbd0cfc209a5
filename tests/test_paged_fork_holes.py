"""Forks of a row whose partly filled last page is no page of the pool (a table entry outside it): the
new row holds the same tokens as its source and no others, so it has no page there either, and the
page that was offered for the copy stays free."""
import numpy as np
import pytest

import dequant_gemv_q4g32_amd as qg
from oracle import paged

torch = pytest.importorskip("torch")


def _state(kind="f16"):
    c = paged.Cache(kind, 2, 8, 2, 64, 16)
    for a in c._arrays:
        a[...] = np.random.default_rng(1).integers(-9, 10, a.shape)
    table = np.array([[5, -1, -1], [3, 99, -1], [-1, -1, 6], [-1, -1, -1], [-1, -1, -1], [7, 2, 2]], np.int32)
    lens = np.array([20, 30, 41, 0, 0, 0], np.int32)
    refs = np.zeros(8, np.int32)
    refs[[5, 3, 6]] = 1
    # of a row whose last page is missing, of another with the same offered page, of a whole row
    src, dst, fresh = (np.array(x, np.int32) for x in ([0, 1, 2], [3, 4, 5], [4, 4, 4]))
    return c, table, lens, refs, src, dst, fresh


def test_oracle_fork_of_a_missing_last_page():
    c, table, lens, refs, src, dst, fresh = _state()
    fresh[2] = 1
    before = [a.copy() for a in c._arrays]
    paged.fork(c, table, lens, refs, src, dst, fresh)
    assert table[3].tolist() == [5, -1, -1] and table[4].tolist() == [3, 99, -1] and table[5].tolist() == [-1, -1, 1]
    assert lens[3:].tolist() == [20, 30, 41] and refs.tolist() == [0, 1, 0, 2, 0, 2, 1, 0]
    for a, b in zip(c._arrays, before):
        b[:, 1] = b[:, 6]
        assert np.array_equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["q8", "f16"])
@pytest.mark.parametrize("offered", [4, -1, 8])
def test_fork_of_a_missing_last_page(kind, offered):
    """Every byte, entry and count as the oracle's, the new rows' tokens and attention as their sources'. An
    offered page that is not needed may be any number, and the same for several forks."""
    from paged_util import assert_same_bytes, dev, download, upload
    c, table, lens, refs, src, dst, fresh = _state(kind)
    fresh[:2], fresh[2] = offered, 1
    for a in c._arrays:                                   # the offered page holds what a former row left there
        a.view(np.uint8)[:, 4] = 0x7E
    pool, t, n, r = upload(c), dev(table), dev(lens), dev(refs)
    qg.kv_fork(pool, t, n, r, dev(src), dev(dst), dev(fresh))
    paged.fork(c, table, lens, refs, src, dst, fresh)
    assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(n.cpu().numpy(), lens)
    assert np.array_equal(r.cpu().numpy(), refs) and refs[4] == 0
    assert_same_bytes(download(c, pool), c)
    place = dev(np.tile(np.arange(48), 3))
    rows = [qg.kv_gather(pool, t, place, dev(np.repeat(x, 48)), layer=1) for x in (src, dst)]
    assert torch.equal(rows[0][0][:96], rows[1][0][:96]) and torch.equal(rows[0][1][:96], rows[1][1][:96])
    q = torch.randn((3, 4, 64), generator=torch.Generator("cuda").manual_seed(2), device="cuda").half().repeat(2, 1, 1)
    out, lse = qg.paged_attention(pool, q, t, n, return_lse=True)
    assert torch.isfinite(out).all() and torch.equal(out[:3], out[3:]) and torch.equal(lse[:3], lse[3:])
