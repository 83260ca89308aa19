"""spec_logits_w4 at the borders of its forms: the longest rows that stay in
LDS and the next longer ones, for every count of rows that changes the limit,
and 17 to 32 such rows with several column tiles a workgroup in every group
size.  Bounds as in test_gpu_w4."""
import numpy as np
import pytest
import torch

import oracle
from speculative_sampling_verification_verify_amd import logits as L
from speculative_sampling_verification_verify_amd.binding import SV_BF16, SV_FP32
from logits_util import HALF, TYPES, dev, head_arrays, host, make_head

pytestmark = pytest.mark.gpu

# (type of the hidden states, group, rows, the longest K without a workspace)
LIMITS = [("bf16", 128, 32, 2432), ("bf16", 64, 17, 2304), ("bf16", 32, 20, 2304), ("fp32", 128, 32, 768), ("fp32", 32, 24, 768),
          ("bf16", 128, 16, 4864), ("bf16", 32, 9, 4608), ("fp32", 128, 16, 1536), ("fp32", 32, 12, 1536), ("bf16", 64, 8, 9344),
          ("fp32", 128, 5, 3200), ("fp32", 64, 4, 6272), ("bf16", 128, 2, 35456)]


def check(R, K, N, group, x, scale, out, exact):
    rng = np.random.default_rng(R * 1009 + K + N)
    if exact:     # every float32 sum is a whole number (times a power of two) below 2^24
        most = max(1, min(255 if x == "bf16" else 2047, int(2 ** 21 / (31 * K))))
        h = rng.integers(-most, most + 1, (R, K)).astype(np.float64)
    else:
        h = host(dev(rng.standard_normal((R, K)) + 0.3, TYPES[x]))
    w, s, z = make_head(rng, N, K, group, scale, zeros=(R + K // 128) % 2 == 0, power=exact)
    arrays = head_arrays(w, s, z)
    got = host(L.spec_logits_w4(dev(h, TYPES[x]), w, s, z, out_dtype=TYPES[out]))
    ref = oracle.logits.w4_product(h, *arrays)
    if exact:
        want = torch.from_numpy(ref).float().to(TYPES[out]).double().numpy()
        assert (got == want).all(), (R, K, N, group)
        return
    bound = oracle.logits.w4_error_bound(h, *arrays, parts=3 if x == "fp32" else 1)
    assert (np.abs(got - ref) <= bound + HALF[out] * (np.abs(ref) + bound)).all(), (R, K, N, group)


@pytest.mark.parametrize("exact", [True, False])
@pytest.mark.parametrize("x,group,R,most", LIMITS)
def test_longest_rows_in_lds(x, group, R, most, exact):
    need = L.lib().spec_logits_w4_workspace_bytes
    code = SV_BF16 if x == "bf16" else SV_FP32
    step = max(group, 128)
    assert need(code, group, R, most) == 0 and need(code, group, R, most + step) > 0
    for K in (most, most + step):
        check(R, K, 37, group, x, "bf16" if R % 2 else "fp32", "fp32", exact)


@pytest.mark.parametrize("x,scale", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("R", [17, 25, 32])
def test_several_column_tiles_a_workgroup(R, group, x, scale):
    check(R, 768, 9001, group, x, scale, "bf16", exact=True)
    check(R, 512, 5003, group, x, scale, "fp32", exact=False)
