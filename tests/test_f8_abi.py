"""The 8-bit entry points refuse bad arguments on the host before touching the
GPU (no compute calls here)."""
import pytest
import torch

from speculative_sampling_verification_verify_amd import logits as L
from speculative_sampling_verification_verify_amd.binding import (SV_BF16, SV_ERR_ARG, SV_ERR_UNSUPPORTED, SV_ERR_WORKSPACE,
                                                                  SV_FP32, SV_OK)
from test_logits_abi import FAKE, _lib


def quant(x=FAKE, xt=SV_BF16, rows=1, R=2, K=128, q=2 * FAKE, s=4 * FAKE):
    return _lib().spec_quantize_f8(x, xt, rows, R, K, q, s, None)


def f8(x=FAKE, xt=SV_BF16, xs=None, w=FAKE, s=FAKE, R=2, K=128, N=10, out=1 << 40, ot=SV_FP32, ws=None, wsb=0):
    return _lib().spec_logits_f8(x, xt, xs, w, s, R, K, N, out, ot, ws, wsb, None)


def test_quantize_refusals():
    assert quant(R=0) == quant(R=0, x=None) == SV_OK
    assert quant(xt=2) == quant(xt=-1) == quant(rows=64) == quant(rows=0) == SV_ERR_UNSUPPORTED
    assert quant(R=L.SL_MAX_ROWS + 1) == quant(K=L.SL_MAX_K + 1) == quant(R=1 << 18, K=1 << 16) == SV_ERR_UNSUPPORTED
    assert quant(R=-1) == quant(K=0) == SV_ERR_ARG
    for k in ("x", "q", "s"):
        assert quant(**{k: None}) == SV_ERR_ARG, k
    assert quant(x=FAKE + 1) == quant(x=FAKE + 2, xt=SV_FP32) == quant(s=FAKE * 4 + 2) == SV_ERR_ARG
    assert quant(q=FAKE + 511) == quant(q=FAKE - 255) == quant(s=FAKE + 508) == quant(s=2 * FAKE + 252) == SV_ERR_ARG


def test_product_refusals():
    assert f8(R=0) == f8(R=0, x=None, w=None) == SV_OK
    assert f8(xt=3) == f8(xt=-1) == f8(ot=2) == SV_ERR_UNSUPPORTED
    assert f8(R=L.SL_MAX_ROWS + 1) == f8(N=(1 << 20) + 1) == f8(K=L.SL_MAX_K + 16) == SV_ERR_UNSUPPORTED
    assert f8(R=1 << 18, K=1 << 16) == f8(R=1 << 20, N=1 << 14) == SV_ERR_UNSUPPORTED
    assert f8(R=-1) == f8(K=0) == f8(N=0) == f8(K=8) == f8(K=120) == SV_ERR_ARG
    assert f8(xt=L.SL_F8) == f8(xs=FAKE) == SV_ERR_ARG
    for k in ("x", "w", "s", "out"):
        assert f8(**{k: None}) == SV_ERR_ARG, k
    assert f8(x=FAKE + 8) == f8(w=FAKE + 8) == f8(s=FAKE + 2) == f8(out=FAKE + 2) == SV_ERR_ARG
    assert f8(xt=L.SL_F8, xs=FAKE + 2) == f8(out=FAKE + 1, ot=SV_BF16) == SV_ERR_ARG


def test_an_output_over_an_input_is_refused():
    at = {"x": 1 << 40, "w": 1 << 41, "s": 1 << 42, "xs": 1 << 43}
    R, K, N = 2, 128, 10
    size = {"x": R * K, "w": N * K, "s": 4, "xs": R * 4}
    for k in at:
        for out in (at[k], at[k] + size[k] - 4, at[k] - R * N * 4 + 4):
            assert f8(**at, xt=L.SL_F8, R=R, K=K, N=N, out=out) == SV_ERR_ARG, (k, hex(out))


def test_workspace():
    need = _lib().spec_logits_f8_workspace_bytes
    assert need(SV_BF16, 1, 4096) == need(SV_FP32, 0, 4096) == need(SV_BF16, -1, 4096) == need(SV_FP32, 16, 4096) == 0
    for bad in ((SV_BF16, 320, 100), (SV_BF16, 320, 1 << 20), (SV_FP32, 1 << 21, 4096), (SV_FP32, 1 << 18, 1 << 16),
                (3, 320, 4096)):
        assert need(*bad) == 0
    for R in (17, 33, 320, 1000, 1 << 18):
        for K in (16, 256, 4096, 65520):
            for out, size in ((SV_BF16, 1 if R > 64 else 2), (SV_FP32, 2)):
                assert need(out, R, K) >= size * R * K + 4 * R * ((K + 127) // 128), (R, K)
    n = need(SV_FP32, 100, 128)
    for ws, wsb in ((None, n), (FAKE, n - 1), (FAKE + 128, n)):
        assert f8(R=100, ws=ws, wsb=wsb) == SV_ERR_WORKSPACE


def test_host_tensors_are_refused():
    z = torch.zeros
    with pytest.raises(ValueError, match="GPU memory"):
        L.spec_quantize_f8(z(2, 128))
    with pytest.raises(ValueError, match="GPU memory"):
        L.spec_logits_f8(z(2, 128), z((4, 128), dtype=torch.uint8), z(1, 1))
