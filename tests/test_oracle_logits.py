"""Pins of the plain implementations of the logits operators: values worked out
by hand, and the identities that the formulas imply."""
import numpy as np
import pytest

import oracle
from logits_util import pack_masks

O = oracle.logits


def test_w4_by_hand():
    # two rows of four weights, groups of two: w = [1 2 | 3 15], [0 8 | 9 4]
    w = np.array([[0x21, 0xF3], [0x80, 0x49]], dtype=np.uint8)
    assert O.unpack_w4(w).tolist() == [[1, 2, 3, 15], [0, 8, 9, 4]]
    s = np.array([[0.5, 2.0], [1.0, 0.25]])
    x = np.array([[1.0, -1.0, 2.0, 0.5]])
    # zeros 8: 0.5 * (-7 + 6) + 2 * (-10 + 3.5) = -13.5; 1 * (-8 - 0) + 0.25 * (2 - 2) = -8
    assert O.w4_product(x, w, s).tolist() == [[-13.5, -8.0]]
    # zeros [1 3], [0 5] (their high bits ignored): 0.5 * -1 + 2 * (0 + 6) = 11.5; -8 + 0.25 * (8 - 0.5) = -6.125
    z = np.array([[0x11, 0x03], [0xF0, 0x05]], dtype=np.uint8)
    assert O.w4_product(x, w, s, z).tolist() == [[11.5, -6.125]]
    assert (O.w4_error_bound(x, w, s, z) > 0).all()


def test_history_by_hand():
    h = O.TokenHistory(3, 5)
    h.append([[1, 1, -1, 4]])
    h.append([[4, 2, 5], [0, 0, -7]], slots=[0, 9], prompt=True)
    assert h.counts().tolist() == [[0, 2, 0x80000000, 0, 0x80000001], [0] * 5, [0] * 5]
    assert h.num().tolist() == [3, 0, 0]
    h.reset([0, 5])
    assert h.num().tolist() == [0, 0, 0]


@pytest.mark.parametrize("f", [lambda *a, **k: O.process_rows(*a, **k)[0], O.process_rows_f32])
def test_process_by_hand(f):
    h = O.TokenHistory(1, 6)
    h.append([[0, 2]], prompt=True)
    h.append([[2, 3]])
    z = np.array([[[2.0, 4.0, -2.0, 3.0, 1.0, 0.0]] * 2])
    got = f(z, history=h, drafts=[[3, 3]], first=0, repetition=[2.0], presence=[0.5], frequency=[0.25],
            bias_ids=[[4, 1, 4]], bias_values=[[1.0, -np.inf, 0.5]])
    # position 0: counts 2:1, 3:1; position 1 also the draft 3
    assert got[0, 0].tolist() == [1.0, -np.inf, -4.75, 0.75, 2.5, 0.0]
    assert got[0, 1].tolist() == [1.0, -np.inf, -4.75, 0.5, 2.5, 0.0]


def test_masks_rows_and_bad_values():
    allowed = np.array([[True, False, True] + [False] * 30 + [True], [False] * 34])
    z = np.arange(3 * 34, dtype=float).reshape(1, 3, 34)
    got, _ = O.process_rows(z, masks=pack_masks(allowed), mask_rows=[[0, -1, 1]], rows=[2])
    assert np.isneginf(got[0, 0]).tolist() == (~allowed[0]).tolist()
    assert (got[0, 1:] == z[0, 1:]).all()
    got, _ = O.process_rows(z, masks=pack_masks(allowed), mask_rows=[[1, 2, -2]])
    assert np.isneginf(got[0, 0]).all() and np.isnan(got[0, 1:]).all()
    assert np.isnan(O.process_rows(z, repetition=[0.0])[0]).all()


def test_neutral_values_change_nothing():
    rng = np.random.default_rng(0)
    h = O.TokenHistory(2, 50)
    h.append(rng.integers(0, 50, (2, 30)))
    z = rng.standard_normal((2, 3, 50)).astype(np.float32)
    assert (O.process_rows_f32(z, history=h, drafts=rng.integers(0, 50, (2, 2)), repetition=[1, 1], presence=[0, 0]) == z).all()
