"""min-p calls whose tokens and counts are really compared: the checks of test_gpu_minp.py leave out what the oracle
decides within its margin, so here uniforms keep away from borders and the share compared is asserted."""
import numpy as np
import pytest
import torch

from speculative_sampling_verification_verify_amd import binding
from logits_util import TYPES, dev
from test_gpu_minp import check_sample, check_verify, logits, settings, verify_inputs

pytestmark = pytest.mark.gpu
HINTS = [0, binding.SV_HINT_ALL_MIN_P]


@pytest.mark.parametrize("hints", HINTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,G,V", [(1, 1, 1), (5, 3, 2), (12, 8, 4099), (6, 5, 40000), (3, 64, 500), (2, 2, 152064), (3, 7, 70001)])
def test_verify(B, G, V, dtype, hints):
    """Every sequence, or all but one of three and more."""
    rng = np.random.default_rng(B * 100 + G + 1)
    p, q, draft, u, gamma, s = verify_inputs(rng, B, G, V, dtype)
    assert check_verify(p, q, draft, 0.05 + 0.9 * u, gamma, s, hints) >= (1 if B < 3 else 1 - 1.01 / B)


def test_verify_many():
    rng = np.random.default_rng(9)
    args = verify_inputs(rng, 100, 3, 20011, "bf16")
    assert check_verify(*args, lenience=rng.random(100).astype(np.float32)) > 0.9


@pytest.mark.parametrize("hints", HINTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_lists_that_overflow(dtype, hints):
    """Rows around what a part's and a row's lists hold, drawn inside of them.  (The values kept are all apart or
    all the same: a nucleus ends far from top_p or in a tie.)"""
    rng = np.random.default_rng(2)
    V = 50000
    z = np.full((8, V), -20.0)
    z[0] = 1.0
    for r, n in ((1, 511), (2, 512), (3, 513), (4, 1023), (5, 1024), (6, 1025)):
        z[r, rng.permutation(V)[:n]] = 2.0 + 0.5 * rng.random(n)
    z[7, 4000:4600] = 3.0
    R = len(z)
    t = dev(z, TYPES[dtype])
    full = lambda v, d=np.float32: np.full(R, v, d)
    for top_k, top_p, T in ((0, 1.0, 1.0), (40, 1.0, 1.0), (2000, 0.7, 1.0), (0, 0.9, 2.0), (0, 1.0, 0.0)):
        s = dict(T=full(T), top_k=full(top_k, np.int32), top_p=full(top_p), min_p=full(0.1))
        for u in (0.0137, 0.3701, 0.9873):
            assert check_sample(t, full(u), s, hints) > 0.8, (top_k, top_p, T, u)


@pytest.mark.parametrize("hints", HINTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_part_far_below_the_largest_overflows(dtype, hints):
    """A flat bulk, whose parts' lists overflow though nothing of them is kept, beside a few likely tokens."""
    rng = np.random.default_rng(4)
    B, G, V = 4, 2, 152064
    p = dev(1.5 * rng.standard_normal((B, G + 1, V)), TYPES[dtype])
    for b in range(B):
        p[b, :, dev(rng.integers(0, V, 20))] = dev(14 + 2 * rng.random((G + 1, 20)), TYPES[dtype])
    q = (p[:, :G].float() + dev(0.2 * rng.standard_normal((B, G, V)), torch.float32)).to(TYPES[dtype])
    one = lambda v, d=np.float32: np.full(B, v, d)
    s = dict(T=one(1.5), top_k=np.array([0, 10, 0, 5], np.int32), top_p=np.array([1, 1, 0.9, 0.8], np.float32), min_p=one(0.05))
    draft = q.argmax(2).int().cpu().numpy()
    u = (0.05 + 0.9 * rng.random((B, G + 1))).astype(np.float32)
    assert check_verify(p, q, draft, u, one(G, np.int32), s, hints) > 0.7
    assert check_sample(p[:, 0].contiguous(), u[:, 0], s, hints) > 0.7


def test_rows_with_masks():
    """Masked values and the type's lowest ones."""
    rng = np.random.default_rng(3)
    R, V = 24, 5003
    for dtype in ("bf16", "fp32"):
        z = logits(rng, (R, V), dtype)
        s = settings(rng, R)
        z[:, ::3] = -torch.inf
        z[1::2, 1::3] = torch.finfo(z.dtype).min
        z[3, 1:] = -torch.inf
        z[4, :-1] = -torch.inf
        for hints in HINTS:
            assert check_sample(z, (0.05 + 0.9 * rng.random(R)).astype(np.float32), s, hints) > 0.9, (dtype, hints)


def test_odd_bases():
    rng = np.random.default_rng(14)
    for dtype in ("bf16", "fp32"):
        for lead in range(1, 9):
            R, V = 5, 6000 + lead
            z = torch.empty(R * V + lead, dtype=TYPES[dtype], device="cuda")[lead:].view(R, V)
            z.copy_(logits(rng, (R, V), dtype))
            assert check_sample(z, (0.05 + 0.9 * rng.random(R)).astype(np.float32), settings(rng, R)) >= 0.8, (dtype, lead)
