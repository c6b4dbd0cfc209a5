"""The largest sizes paged attention takes, as include/qgemv.h states them (host checks only)."""
import ctypes

import pytest

import dequant_gemv_q4g32_amd as qg


@pytest.mark.parametrize("batch,heads,max_len,status", [
    (2 ** 17, 32, 511 * 32, 0), (2 ** 17, 32, 511 * 32 + 1, -2), (2 ** 22, 1, 511 * 32, 0), (2 ** 22, 1, 512 * 32, -2),
    (2 ** 22 + 1, 1, 32, -2), (2 ** 22, 1, 0, 0), (1, 63, 2 ** 30, 0), (1, 64, 2 ** 30, -2), (1, 1, 2 ** 30 + 1, -2)])
def test_product_of_batch_heads_and_steps(batch, heads, max_len, status):
    """batch * heads * ceil(max_len / 32) below 2^31, batch * heads up to 2^22, max_len up to 2^30."""
    pool = qg._Pool(0x1000000, 10, 1, 0, qg.KV_KINDS["f16"], 1, 64, 16)
    got = ctypes.c_int64()
    assert qg.lib.qg_paged_attention_bytes(ctypes.addressof(pool), batch, heads, max_len, ctypes.byref(got)) == status
