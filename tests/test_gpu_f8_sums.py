"""How the product of the 8-bit head is summed: in float32 whatever the number of
rows and the output's type, unless the caller asks for the matrix cores' 8-bit
products."""
import numpy as np
import pytest
import torch

from oracle import f8
from speculative_sampling_verification_verify_amd import logits as L
from logits_util import HALF, TYPES, dev, host
from test_gpu_f8 import SHAPES, head

pytestmark = pytest.mark.gpu

MANY = [s for s in SHAPES if s[0] > 64]


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("R", [1, 16, 17, 64, 65, 130, 200, 320])
def test_small_products_beside_large_ones(R, out):
    """In each 8 of k, two products of 448^2 cancel and six of 1 are left: 6 K / 8.  What a float32 sum
    may drop is 2^-23 of 448^2's binade in each of a block's 132 additions, 2^-6 each."""
    K, N = 1024, 300
    x, w = np.ones((R, K)), np.ones((N, K))
    x[:, 0::8] = x[:, 1::8] = w[:, 0::8] = 448
    w[:, 1::8] = -448
    one = lambda n: torch.ones((n, K // 128), device="cuda")
    got = host(L.spec_logits_f8(dev(f8.encode(x)).view(torch.float8_e4m3fn), dev(f8.encode(w)), one(3), one(R), out_dtype=TYPES[out]))
    want, tol = 6 * K / 8, K / 128 * 132 * 2.0 ** -6
    assert np.abs(got - want).max() <= tol + HALF[out] * (want + tol), (got.min(), got.max())


@pytest.mark.parametrize("x", ["bf16", "fp32"])
@pytest.mark.parametrize("R,K,N", MANY)
def test_many_rows_in_bf16(R, K, N, x):
    """Real values, within the bound of float32 sums."""
    rng = np.random.default_rng(R * 104729 + K * 17 + N)
    h = dev(rng.standard_normal((R, K)) * np.where(rng.random(K) < 0.02, 20, 1), TYPES[x])
    w, s = head(rng, N, K)
    got = host(L.spec_logits_f8(h, w, s, out_dtype=torch.bfloat16))
    ref, bound = f8.product(*f8.quantize(host(h).astype(np.float32)), w.cpu().numpy(), s.cpu().numpy())
    assert (np.abs(got - ref) <= bound + HALF["bf16"] * (np.abs(ref) + bound)).all()


@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_a_row_does_not_depend_on_the_others(out):
    """The same bits for a row in calls of 17 rows and more, and of 1 to 16."""
    rng = np.random.default_rng(3)
    h = dev(rng.standard_normal((700, 400)), torch.bfloat16)
    w, s = head(rng, 1000, 400)
    all_ = L.spec_logits_f8(h, w, s, out_dtype=TYPES[out])
    for R in (17, 64, 65, 128, 130, 192, 200, 256, 320, 448):
        assert torch.equal(L.spec_logits_f8(h[:R], w, s, out_dtype=TYPES[out]), all_[:R]), R
    few = L.spec_logits_f8(h[:16], w, s, out_dtype=TYPES[out])
    for R in (1, 2, 3, 9):
        assert torch.equal(L.spec_logits_f8(h[:R], w, s, out_dtype=TYPES[out]), few[:R]), R


@pytest.mark.parametrize("x", ["bf16", "fp32"])
@pytest.mark.parametrize("R,K,N", SHAPES)
def test_f8_products(R, K, N, x):
    """The caller's 8-bit products: within their bound from 65 rows on, the same call up to 64."""
    rng = np.random.default_rng(R * 104729 + K * 17 + N)
    h = dev(rng.standard_normal((R, K)) * np.where(rng.random(K) < 0.02, 20, 1), TYPES[x])
    w, s = head(rng, N, K)
    out = torch.full((R, N), -7.0, dtype=torch.bfloat16, device="cuda")
    assert L.spec_logits_f8(h, w, s, out=out, f8_products=True) is out
    if R <= 64:
        assert torch.equal(out, L.spec_logits_f8(h, w, s, out_dtype=torch.bfloat16))
    got = host(out)
    ref, bound = f8.product(*f8.quantize(host(h).astype(np.float32)), w.cpu().numpy(), s.cpu().numpy(), codes_as_they_are=R > 64)
    assert (np.abs(got - ref) <= bound + HALF["bf16"] * (np.abs(ref) + bound)).all()


def test_a_head_of_f8_products():
    """The head's choice goes with every call of it; an output in fp32 is refused."""
    rng = np.random.default_rng(4)
    h = dev(rng.standard_normal((2, 40, 256)), torch.bfloat16)
    weights = dev(rng.standard_normal((500, 256)), torch.bfloat16)
    plain, fast = L.F8Head.quantize(weights), L.F8Head.quantize(weights, f8_products=True)
    want = L.spec_logits_f8(h, plain.weights, plain.scales, f8_products=True)
    assert torch.equal(fast(h), want) and torch.equal(plain(h), L.spec_logits_f8(h, plain.weights, plain.scales))
    assert not torch.equal(plain(h), want)
    for bad in (lambda: fast(h, out_dtype=torch.float32), lambda: fast(h.float()),
                lambda: L.spec_logits_f8(h.float(), plain.weights, plain.scales, f8_products=True)):
        with pytest.raises(ValueError):
            bad()


def test_f8_products_captured_with_a_workspace_of_their_own():
    """One graph with both forms, replayed with new rows between eager calls."""
    rng = np.random.default_rng(5)
    h = dev(rng.standard_normal((130, 640)), torch.bfloat16)
    w, s = head(rng, 385, 640)
    outs = [torch.empty((130, 385), dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    def both():
        for o, fast in zip(outs, (False, True)):
            L.spec_logits_f8(h, w, s, out=o, f8_products=fast)

    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for _ in range(3):
        h.copy_(dev(rng.standard_normal((130, 640)), torch.bfloat16))
        both()
        want = [o.clone() for o in outs]
        for o in outs:
            o.fill_(-9)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
