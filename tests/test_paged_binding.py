"""The paged-cache binding's streams (on the CPU, with stand-ins for what needs a GPU)."""
import types

import pytest

import dequant_gemv_q4g32_amd as qg

torch = pytest.importorskip("torch")


def test_stream_of_another_device_is_refused():
    """A torch stream belongs to a device; on any other than the pool's a call must not run elsewhere."""
    pool = types.SimpleNamespace(device=torch.device("cuda", 0), _index=0)
    other = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=64)
    x = None
    for call in (lambda: qg.kv_append(pool, x, x, x, x, stream=other), lambda: qg.kv_gather(pool, x, x, stream=other),
                 lambda: qg.paged_attention(pool, x, x, x, stream=other), lambda: qg.kv_copy_pages(pool, x, x, stream=other),
                 lambda: qg.kv_fork(pool, x, x, x, x, x, x, stream=other), lambda: qg.kv_free(pool, x, x, x, x, stream=other),
                 lambda: qg.kv_compact(pool, x, x, stream=other)):
        with pytest.raises(ValueError, match="stream"):
            call()
