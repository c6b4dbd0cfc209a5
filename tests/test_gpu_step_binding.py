"""GPU tests of what the decode step's calls refuse."""
import pytest

import dequant_gemv_q4g32_amd as qg

from paged_util import dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_an_output_without_its_input():
    """q_out is for q's rows: without queries nothing would be written there."""
    pool = qg.KVPool.zeros("q8", 1, 64, 16, 4)
    k = torch.zeros((1, 64), dtype=torch.float16, device="cuda")
    args = [pool, dev([[0]]), qg.Rotary(64, qg.rope_freqs(64))]
    with pytest.raises(ValueError, match="q_out"):
        qg.kv_append_rope(*args, None, k, k, dev([0]), q_out=torch.zeros_like(k))
    assert qg.kv_append_rope(*args, None, k, k, dev([0])) is None
