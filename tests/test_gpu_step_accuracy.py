"""GPU tests of how exactly queries and keys are normed and rotated."""
import numpy as np
import pytest

import dequant_gemv_q4g32_amd as qg
from oracle import step

from paged_util import dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,rot,inter", [(64, 32, False), (128, 128, True), (256, 0, False), (256, 192, True)])
def test_norm_of_a_head_with_an_infinity(dim, rot, inter):
    """Its root is infinite: what is finite becomes zero, the infinity itself NaN, and so does its pair's other half."""
    rng = np.random.default_rng(dim)
    w = (rng.random(dim) + 0.5).astype(np.float16)
    freqs = qg.rope_freqs(rot) if rot else None
    rotary = qg.Rotary(dim, freqs, inter, dev(w, np.float16), dev(w, np.float16))
    x = rng.standard_normal((3, 4, dim)).astype(np.float16)
    x[0, 1, 5], x[1, 0, dim - 1], x[2, 3, 0], x[2, 3, 9] = np.inf, -np.inf, np.inf, -np.inf
    pos = np.array([0, 3, 100000], np.int32)
    with np.errstate(invalid="ignore"):
        want = np.stack([[step.rotate(h, p, [] if freqs is None else freqs, inter, w, 1e-6) for h in heads] for heads, p in zip(x, pos)])
    got = qg.qk_rope(rotary, dev(x, np.float16), dev(x, np.float16), dev(pos))
    for out in got:
        out = out.cpu().numpy().astype(np.float64)
        assert np.array_equal(np.isnan(out), np.isnan(want))
        odd = ~np.isfinite(x).all(-1)
        assert (out[odd][~np.isnan(want[odd])] == 0).all() and (want[odd][~np.isnan(want[odd])] == 0).all()
