"""The min-p oracle by hand, and against the definition p(v) >= min_p max p."""
import numpy as np
import pytest

from oracle import minp, verify


def test_by_hand():
    z = np.log(np.array([0.5, 0.25, 0.125, 0.125]))
    assert np.isfinite(minp.cut(z, 1.0, 0.6)).tolist() == [True, False, False, False]
    assert np.isfinite(minp.cut(z, 1.0, 0.4)).tolist() == [True, True, False, False]
    assert np.isfinite(minp.cut(z, 1.0, 0.2)).tolist() == [True] * 4
    assert np.isfinite(minp.cut(z, 0.5, 0.2)).tolist() == [True, True, False, False]   # ratios 1, 1/4, 1/16
    assert minp.cut(z, 0.0, 0.5) is z and minp.cut(z, 1.0, 0.0) is z
    t, p, _ = minp.sample(z[None], [0.7], [1.0], [0], [1.0], [0.4])
    assert t[0] == 1 and np.isclose(p[0], 1 / 3)
    assert minp.sample(z[None], [0.7], [1.0], [0], [1.0], [1.5])[0][0] == -1
    assert minp.sample(z[None], [0.7], [1.0], [0], [1.0], [np.nan])[0][0] == -1


@pytest.mark.parametrize("T,min_p", [(1.0, 0.05), (0.3, 0.5), (2.0, 0.01), (1.0, 1.0)])
def test_against_probabilities(T, min_p):
    rng = np.random.default_rng(3)
    z = 3 * rng.standard_normal(2000)
    p = verify.process(z, T, 0, 1.0).prob
    assert (np.isfinite(minp.cut(z, T, min_p)) == (p >= min_p * p.max() * (1 - 1e-12))).all()


def test_order_is_min_p_then_top_k_then_top_p():
    """top_p counts the mass of what min-p and top-k left."""
    z = np.log(np.array([0.4, 0.3, 0.2, 0.1]))
    pr = verify.process(minp.cut(z, 1.0, 0.6), 1.0, 0, 0.55)     # 4/7, 3/7: the first alone reaches 0.55
    assert pr.kept.tolist() == [True, False, False, False]
    assert verify.process(z, 1.0, 0, 0.55).kept.tolist() == [True, True, False, False]
    pr = verify.process(minp.cut(z, 1.0, 0.6), 1.0, 1, 1.0)
    assert pr.kept.tolist() == [True, False, False, False]
