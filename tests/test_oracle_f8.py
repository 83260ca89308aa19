"""The oracle of the 8-bit quantiser and product, against torch's own conversion
and by hand, and the refusals of its entry points that no library is needed for."""
import numpy as np
import pytest
import torch

import oracle
from oracle import f8


def test_codes_are_the_format():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(f8.VALUES, want, equal_nan=True)


def test_encode_rounds_to_nearest_even():
    v = np.concatenate([f8.VALUES[:127], (f8.VALUES[:126] + f8.VALUES[1:127]) / 2, np.linspace(0, 448, 5001),
                        2.0 ** -np.arange(1, 30)]).astype(np.float32)
    v = np.concatenate([v, -v])
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(f8.encode(v), want)


@pytest.mark.parametrize("rows", [1, 128])
def test_quantize(rows):
    rng = np.random.default_rng(rows)
    x = rng.standard_normal((130, 300)).astype(np.float32)
    x[:, 128:256] = 0
    q, s = f8.quantize(x, rows)
    assert s.shape == (130 if rows == 1 else 2, 3) and (s[:, 1] == f8.TINY).all() and (q[:, 128:256] == 0).all()
    back = f8.VALUES[q] * np.repeat(np.repeat(s, rows, 0)[:130], 128, 1)[:, :300]
    # half a step of 8-bit values, or of their subnormals
    tol = np.abs(x) * 2.0 ** -4 + np.repeat(np.repeat(s, rows, 0)[:130], 128, 1)[:, :300] * 2.0 ** -10
    assert (np.abs(back - x) <= tol * (1 + 1e-6)).all()
    # each block's largest value takes the largest code
    assert (f8.VALUES[q].reshape(130, 300)[:, :128].max() == 448) or (np.abs(f8.VALUES[q])[:, :128].max() == 448)


def test_product_by_hand():
    codes = f8.encode(np.array([[1, 2, 0.5, -4]]))
    weights = f8.encode(np.array([[1, 1, 1, 1], [2, -2, 8, 0.25]]))
    out, bound = oracle.f8.product(codes, np.array([[0.5]], dtype=np.float32), weights, np.array([[4]], dtype=np.float32))
    assert np.array_equal(out, [[-1.0, 2.0]]) and (bound < 3e-3).all()   # 2 * 132 * 2^-22 * 32 and little else
