"""A head that no call would take is refused when it is made (no compute calls here)."""
import pytest
import torch

from speculative_sampling_verification_verify_amd import logits as L


@pytest.mark.parametrize("K", [1, 8, 100, 120, L.SL_MAX_K + 16])
def test_k(K):
    with pytest.raises(ValueError, match="K"):
        L.F8Head(torch.zeros((10, K), dtype=torch.uint8), torch.zeros((1, (K + 127) // 128)))
    with pytest.raises(ValueError, match="K"):
        L.F8Head.quantize(torch.zeros((10, K)))   # before anything is quantised


def test_shapes():
    w = torch.zeros((200, 256), dtype=torch.uint8)
    assert (L.F8Head(w, torch.zeros((2, 2))).N, L.F8Head(w, torch.zeros((2, 2))).K) == (200, 256)
    for weights, scales in ((w, torch.zeros((2, 3))), (w, torch.zeros((1, 2))), (w[0], torch.zeros((2, 2))), (w, torch.zeros(2))):
        with pytest.raises(ValueError):
            L.F8Head(weights, scales)
    with pytest.raises(ValueError):
        L.F8Head.quantize(torch.zeros((2, 10, 256)))
