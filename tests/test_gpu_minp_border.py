"""min-p's border, z >= zmax + T ln(min_p), where exp((z - zmax) / T) no longer tells the two sides apart: whichever
launch takes the row, what is below the border is not kept."""
import numpy as np
import pytest

from oracle import minp
from speculative_sampling_verification_verify_amd import binding
from logits_util import TYPES, dev
from test_gpu_minp import bits, sample

import torch

pytestmark = pytest.mark.gpu


def check(z, dtype, T, min_p, hints):
    """Rows z [R, V]: every kept value is drawn by some uniform, with its probability, and no other."""
    R, V = z.shape
    t = dev(z, TYPES[dtype])
    T, min_p = np.broadcast_to(np.float32(T), R).copy(), np.broadcast_to(np.float32(min_p), R).copy()
    off = dict(T=T, min_p=min_p, top_k=np.zeros(R, np.int32), top_p=np.ones(R, np.float32))
    rows = bits(t)
    for u in (0.01, 0.24, 0.49, 0.51, 0.76, 0.99):
        us = np.full(R, u, np.float32)
        tok, prob = sample(t, us, off, hints)
        want, p, margin = minp.sample(rows, us, T, off["top_k"], off["top_p"], min_p)
        assert (margin > 1e-6).all(), (u, margin)
        assert (tok == want).all(), (u, np.argwhere(tok != want)[:4], tok[:4], want[:4])
        np.testing.assert_allclose(prob, p, rtol=2.0 ** -23)


@pytest.mark.parametrize("hints", [0, binding.SV_HINT_ALL_MIN_P])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_min_p_of_one_keeps_the_largest_alone(dtype, hints):
    """Values so close to the largest, next to T, that their exponential rounds to 1."""
    z = np.full((4, 1000), -50.0)
    z[0, 7], z[0, 3] = 0.0, -1e-17
    z[1, 500], z[1, [2, 999]] = 1e-20, 0.0
    z[2, 4], z[2, 900] = 1.0, 1 - 2.0 ** -8
    z[3, 10:20], z[3, 15] = -1e-30, 1e-30
    check(z, dtype, np.array([1.0, 0.5, 1e20, 2.0]), 1.0, hints)


@pytest.mark.parametrize("hints", [0, binding.SV_HINT_ALL_MIN_P])
def test_below_a_border_close_to_the_largest(hints):
    """min_p next to 1, a largest value of 0 and one value so close to the border, on either side, that its
    exponential rounds as the border's does."""
    rng = np.random.default_rng(1)
    T = rng.uniform(0.5, 2, 200000).astype(np.float32)
    k = rng.integers(3, 40, len(T))
    min_p = (1 - k * 2.0 ** -24).astype(np.float32)
    border = T.astype(np.float64) * np.log(min_p.astype(np.float64))
    v = border.astype(np.float32).astype(np.float64)
    off = np.abs(v / border - 1)
    near = np.nonzero((off < 4e-10 / k) & (off > 1e-13))[0][:60]
    below = v[near] < border[near]
    assert len(near) == 60 and 10 < below.sum() < 50
    z = np.full((60, 300), -1.0)
    z[:, 40], z[:, 30] = 0.0, v[near]
    check(z, "fp32", T[near], min_p[near], hints)


def test_the_same_in_every_launch():
    """A row's border does not depend on whether its lists hold what is kept: such rows with and without
    2000 more values that are."""
    z = np.tile(-50 - 0.01 * np.arange(5000), (6, 1))
    z[:, 4000] = 0.0
    z[:, 3] = -1e-17
    z[3:, 1000:3000] = 0.0
    for hints in (0, binding.SV_HINT_ALL_MIN_P):
        R = len(z)
        off = dict(T=np.ones(R, np.float32), min_p=np.ones(R, np.float32), top_k=np.zeros(R, np.int32), top_p=np.ones(R, np.float32))
        tok, prob = sample(dev(z, torch.float32), np.zeros(R, np.float32), off, hints)
        assert tok.tolist() == [4000] * 3 + [1000] * 3
        np.testing.assert_allclose(prob, [1.0] * 3 + [1 / 2001] * 3, rtol=2.0 ** -23)
