"""Extend serves rows in order, and a row that the free pages do not suffice for counts for the rows behind it: by
the definition (on the CPU), and on the device."""
import numpy as np
import pytest

from oracle import step

# 3 free pages of 16 tokens, empty rows: (tokens asked for, tokens granted, pages in the table afterwards)
ORDERS = [([80, 32], [0, 0], []), ([32, 80], [32, 0], [0, 1]), ([80, 0, 1], [0, 0, 0], []), ([32, 32, 16], [32, 0, 0], [0, 1]),
          ([32, 16, 80], [32, 16, 0], [0, 1, 2]), ([129, 32], [0, 32], [0, 1])]   # 129: past the row's 8 pages, and not counted


def rows_of(add):
    return np.full((len(add), 8), -1, np.int32), np.zeros(len(add), np.int32), np.zeros(3, np.int32), np.array(add, np.int32)


@pytest.mark.parametrize("add,granted,pages", ORDERS)
def test_by_definition(add, granted, pages):
    table, lens, refs, asked = rows_of(add)
    got = step.extend(table, lens, refs, asked, 512, 16)
    assert got[0].tolist() == granted and lens.tolist() == granted and table[table >= 0].tolist() == pages
    assert refs.tolist() == [1] * len(pages) + [0] * (3 - len(pages))


@pytest.mark.gpu
@pytest.mark.parametrize("add,granted,pages", ORDERS)
def test_on_the_device(add, granted, pages):
    import dequant_gemv_q4g32_amd as qg
    from paged_util import dev
    table, lens, refs, asked = (dev(x) for x in rows_of(add))
    got = qg.kv_extend(qg.KVPool.zeros("q8", 1, 64, 16, 3), table, lens, refs, asked, 512)
    assert got[0].tolist() == granted and lens.tolist() == granted and table[table >= 0].tolist() == pages
    assert refs.tolist() == [1] * len(pages) + [0] * (3 - len(pages))
