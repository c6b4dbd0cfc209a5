"""Frequencies and bases that leave fp64 are refused, on the CPU."""
import ctypes

import numpy as np
import pytest

import dequant_gemv_q4g32_amd as qg

RANGE = -5


@pytest.mark.parametrize("kind,dim,base,scale", [
    ("base", 64, 1e4, 1e300), ("base", 4, 1e4, 1e160), ("base", 64, 1.5, 1e-320), ("linear", 64, 1e4, 1e-320), ("linear", 128, 2.0, 5e-324),
    ("turns", 64, 1e4, 1e-320), ("parts", 64, 1e4, 1e-320)])
def test_out_of_fp64(kind, dim, base, scale):
    out = (ctypes.c_double * 64)()
    assert qg.lib.qg_rope_freqs(qg.ROPE_KINDS[kind], dim, base, scale, 4096.0, 1.0, 32.0, out) == RANGE
    with pytest.raises(qg.QGError):
        qg.rope_freqs(dim, base, kind, scale, 4096.0)


@pytest.mark.parametrize("kind,dim,base,scale", [("base", 64, 1e4, 1e250), ("base", 4, 1e4, 1e150), ("linear", 64, 1e4, 1e-300)])
def test_just_inside(kind, dim, base, scale):
    assert np.isfinite(qg.rope_freqs(dim, base, kind, scale)).all()
