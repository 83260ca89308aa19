"""The shapes of test_gpu_f8_forms.py reach every tile kernel of the 8-bit product (no compute calls here)."""
from speculative_sampling_verification_verify_amd import logits as L
from speculative_sampling_verification_verify_amd.binding import SV_BF16
from f8_forms import LONG, SHAPES, form, row_blocks
from test_logits_abi import _lib


def test_every_kernel_is_reached():
    every = {(cn, mt, f8) for cn in (1, 2) for mt in range(1, 6) for f8 in (False, True) if f8 or mt <= 2}
    assert {form(R, N, f8) for R, K, N, f8 in SHAPES} == every
    assert {form(R, N, f8)[0] for R, N, f8 in LONG} == {2} and {form(R, N, f8)[2] for R, N, f8 in LONG} == {False, True}


def test_the_rule_is_the_librarys():
    """As far as the workspace shows it: its row tiles."""
    need = _lib().spec_logits_f8_workspace_bytes
    for R in (*range(17, 2100, 7), 5000, 1 << 18):
        for K in (16, 128, 1040):
            KB = -(-K // 128)
            assert need(SV_BF16, R, K) == row_blocks(R, False) * KB * (8192 + 128), (R, K)
            if R > 64:
                assert need(L.SL_BF16_F8, R, K) == row_blocks(R, True) * KB * (4096 + 128), (R, K)
