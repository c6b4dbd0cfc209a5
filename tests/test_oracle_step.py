"""The oracle of a decode step's operators: hand-worked cases and invariants."""
import math

import numpy as np
import pytest

from oracle import step


def test_extend_by_hand():
    """Pages of 4 tokens, pages 0 to 5, of which 1, 3 and 4 are free."""
    table = np.array([[0, -1, -1], [2, -1, -1], [5, -1, -1]], np.int32)
    lens = np.array([4, 3, 2], np.int32)
    refs = np.array([1, 0, 1, 0, 0, 1], np.int32)
    granted, starts, seqs, pos = step.extend(table, lens, refs, np.array([1, 1, 6], np.int32), 9, 4)
    assert granted.tolist() == [1, 1, 6] and starts.tolist() == [0, 1, 2, 8] and lens.tolist() == [5, 4, 8]
    assert table.tolist() == [[0, 1, -1], [2, -1, -1], [5, 3, -1]] and refs.tolist() == [1, 1, 1, 1, 0, 1]
    assert seqs.tolist() == [0, 1, 2, 2, 2, 2, 2, 2, -1] and pos.tolist() == [4, 3, 2, 3, 4, 5, 6, 7, -1]


def test_extend_refusals_by_hand():
    """Row 0 lacks more pages than are free, row 1 needs none, row 2 needs one and stands behind row 0, row 3's
    partly filled page is shared, row 4 passes its table row."""
    table = np.array([[0, -1, -1], [1, -1, -1], [-1, -1, -1], [2, -1, -1], [3, 4, 5]], np.int32)
    lens = np.array([4, 1, 0, 2, 12], np.int32)
    refs = np.array([1, 1, 2, 1, 1, 1, 0], np.int32)
    t0, r0 = table.copy(), refs.copy()
    granted, starts, seqs, pos = step.extend(table, lens, refs, np.array([5, 3, 1, 1, 1], np.int32), 20, 4)
    assert granted.tolist() == [0, 3, 0, 0, 0] and starts.tolist() == [0, 5, 8, 9, 10, 11] and lens.tolist() == [4, 4, 0, 2, 12]
    assert np.array_equal(table, t0) and np.array_equal(refs, r0)
    assert seqs.tolist() == [-1] * 5 + [1] * 3 + [-1] * 12 and pos.tolist() == [-1] * 5 + [1, 2, 3] + [-1] * 12


def test_extend_slots_by_hand():
    """The third row's tokens pass the slot map: it and what follows get none."""
    table, lens = np.full((4, 2), -1, np.int32), np.zeros(4, np.int32)
    refs = np.zeros(8, np.int32)
    granted, starts, seqs, pos = step.extend(table, lens, refs, np.array([2, -5, 3, 1], np.int32), 4, 4)
    assert granted.tolist() == [2, 0, 0, 0] and starts.tolist() == [0, 2, 2, 4, 4]
    assert seqs.tolist() == [0, 0, -1, -1] and refs.tolist() == [1] + [0] * 7


def test_trim_undoes_extend():
    rng = np.random.default_rng(1)
    table, lens, refs = np.full((5, 6), -1, np.int32), np.zeros(5, np.int32), np.zeros(40, np.int32)
    step.extend(table, lens, refs, np.array([3, 9, 0, 16, 1], np.int32), 64, 4)
    before = [x.copy() for x in (table, lens, refs)]
    step.extend(table, lens, refs, rng.integers(0, 8, 5).astype(np.int32), 64, 4)
    step.trim(table, lens, refs, before[1], 4)
    assert all(np.array_equal(a, b) for a, b in zip((table, lens, refs), before))
    step.trim(table, lens, refs, np.array([-1, 100, 0, 0, 0], np.int32), 4)
    assert lens.tolist() == [3, 9, 0, 0, 0] and refs.sum() == 4


def test_rotate_by_hand():
    x = np.array([1.0, 2.0, 3.0, 4.0, 7.0, -9.0])
    half = step.rotate(x, 1, [math.pi / 2, math.pi])
    assert np.allclose(half, [-3, -2, 1, -4, 7, -9])
    inter = step.rotate(x, 1, [math.pi / 2, math.pi], interleaved=True, factor=2.0)
    assert np.allclose(inter, [-4, 2, -6, -8, 7, -9])
    normed = step.rotate([3.0, 4.0], 5, [], weight=[1.0, 2.0], eps=0.0)
    assert np.allclose(normed, np.array([3.0, 8.0]) / math.sqrt(12.5))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotated_products_depend_on_the_distance_alone(interleaved):
    rng = np.random.default_rng(2)
    f = step.freqs("plain", 16, 10000.0)
    a, b = rng.standard_normal((2, 24))
    near = step.rotate(a, 7, f, interleaved) @ step.rotate(b, 3, f, interleaved)
    far = step.rotate(a, 1007, f, interleaved) @ step.rotate(b, 1003, f, interleaved)
    assert abs(near - far) < 1e-10
    assert abs(np.linalg.norm(step.rotate(a, 123456, f, interleaved)) - np.linalg.norm(a)) < 1e-10


def test_frequencies():
    plain = step.freqs("plain", 64, 10000.0)
    assert plain[0] == 1.0 and abs(plain[16] - 0.01) < 1e-15
    assert np.allclose(step.freqs("linear", 64, 10000.0, 4.0), plain / 4)
    ntk = step.freqs("base", 64, 10000.0, 4.0)
    assert ntk[0] == 1.0 and abs(ntk[-1] - plain[-1] / 4) < 1e-15
    for kind in ("turns", "parts"):
        f = step.freqs(kind, 64, 10000.0, 8.0, 4096, 1.0, 32.0)
        turns = 4096 * plain / (2 * math.pi)
        # `parts` rounds the pairs that make `high` and `low` turns outwards, by less than one pair each
        wide = 1.0 if kind == "turns" else 10000.0 ** (2 / 64)
        assert np.allclose(f[turns > 32 * wide], plain[turns > 32 * wide])
        assert np.allclose(f[turns < 1 / wide], plain[turns < 1 / wide] / 8)
        assert (f <= plain * (1 + 1e-15)).all() and (f >= plain / 8 * (1 - 1e-15)).all() and (np.diff(f) < 0).all()
