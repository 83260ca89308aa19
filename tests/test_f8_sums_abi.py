"""The 8-bit head's choice of products: types and workspaces, on the host (no
compute calls here)."""
from speculative_sampling_verification_verify_amd import logits as L
from speculative_sampling_verification_verify_amd.binding import SV_BF16, SV_ERR_ARG, SV_ERR_UNSUPPORTED, SV_ERR_WORKSPACE, SV_FP32
from test_f8_abi import FAKE, f8
from test_logits_abi import _lib


def test_workspace_of_each_form():
    """Rows as bf16 where sums are in float32, whatever the output's type; as codes for 8-bit products."""
    need = _lib().spec_logits_f8_workspace_bytes
    for R in (65, 128, 320, 448, 1000, 1 << 18):
        for K in (16, 256, 4096, 65520):
            scales = 4 * R * ((K + 127) // 128)
            assert need(SV_BF16, R, K) == need(SV_FP32, R, K) >= 2 * R * K + scales, (R, K)
            assert R * K + scales <= need(L.SL_BF16_F8, R, K) < need(SV_BF16, R, K), (R, K)
    for R in (1, 16, 17, 64):
        assert need(L.SL_BF16_F8, R, 4096) == need(SV_BF16, R, 4096), R
    for R in range(17, 600):   # a workspace also serves fewer rows
        assert need(SV_BF16, R, 256) <= need(SV_BF16, R + 1, 256), R


def test_types():
    # (each of these ends before a launch)
    assert f8(ot=L.SL_BF16_F8, R=100) == f8(ot=SV_BF16, R=100) == SV_ERR_WORKSPACE
    assert f8(ot=5) == f8(ot=8) == f8(xt=L.SL_BF16_F8) == SV_ERR_UNSUPPORTED
    assert f8(ot=L.SL_BF16_F8, out=FAKE + 1) == f8(ot=L.SL_BF16_F8, out=None) == SV_ERR_ARG
    n = _lib().spec_logits_f8_workspace_bytes(L.SL_BF16_F8, 100, 128)
    for ws, wsb in ((None, n), (FAKE, n - 1), (FAKE + 128, n)):
        assert f8(ot=L.SL_BF16_F8, R=100, ws=ws, wsb=wsb) == SV_ERR_WORKSPACE
    # the output is bf16: its last byte lies before a hidden row that begins behind it
    at = 1 << 40
    assert f8(ot=L.SL_BF16_F8, R=100, N=8, out=at - 100 * 8 * 2, x=at) == SV_ERR_WORKSPACE
    assert f8(ot=L.SL_BF16_F8, R=2, N=8, out=at - 2 * 8 * 2 + 2, x=at) == SV_ERR_ARG
