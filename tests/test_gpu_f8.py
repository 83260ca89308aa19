"""The 8-bit floating-point quantiser and product on the GPU against the oracle.

Codes and scales are defined to the last bit, so they have to be equal.  The
product is checked on two kinds of inputs: codes of small integers with scales
that are powers of two, where every float32 partial sum is exact and the result
is the correctly rounded exact product; and real values, where it may be off by
the roundings of float32 sums (oracle.f8.product) and half a step of the
output's type."""
import numpy as np
import pytest
import torch

import oracle
from oracle import f8
from speculative_sampling_verification_verify_amd import logits as L
from logits_util import HALF, TYPES, dev, host

pytestmark = pytest.mark.gpu

# (R, K, N): one value of everything, tails of rows, columns and blocks, odd N, both sides of every change of form.
SHAPES = [(1, 16, 1), (1, 128, 16), (3, 144, 17), (2, 256, 33), (16, 240, 50), (17, 400, 129), (5, 528, 1000), (33, 512, 100),
          (64, 384, 257), (65, 128, 300), (100, 1040, 64), (130, 640, 385), (1, 8192, 130), (16, 9600, 40), (16, 10240, 40),
          (4, 1088, 2049), (1, 512, 32000), (129, 272, 513), (257, 256, 770), (700, 144, 3001), (8, 4096, 4111)]


def codes_of(t):
    return t.view(torch.uint8).cpu().numpy()


def spread(rng, shape):
    """Values over many binades, some of them zero."""
    x = rng.standard_normal(shape) * np.exp(2 * rng.standard_normal(shape))
    return np.where(rng.random(shape) < 0.05, 0, x)


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("x", ["bf16", "fp32"])
@pytest.mark.parametrize("R,K", [(1, 1), (1, 128), (3, 130), (129, 1000), (200, 264), (5, 4096), (128, 128), (257, 129)])
def test_quantize(R, K, x, rows):
    rng = np.random.default_rng(R * 1000 + K)
    t = dev(spread(rng, (R, K)), TYPES[x])
    if R > 100:
        t[:128, :min(K, 128)] = 0          # a block of zeros
    q, s = L.spec_quantize_f8(t, rows)
    want, ws = f8.quantize(host(t).astype(np.float32), rows)
    assert q.dtype == torch.float8_e4m3fn and np.array_equal(s.cpu().numpy(), ws)
    assert np.array_equal(codes_of(q), want)


def test_quantize_every_border():
    """Quotients on, just above and just below every border between two codes
    (the block's scale is 1, by a value of 448)."""
    mid = (f8.VALUES[:126] + f8.VALUES[1:127]) / 2
    mid = mid.astype(np.float32)
    v = np.concatenate([mid, np.nextafter(mid, np.float32(1000)), np.nextafter(mid, np.float32(0)), f8.VALUES[:127]])
    v = np.concatenate([v, -v]).astype(np.float32)
    v = np.concatenate([v, np.zeros(-len(v) % 127, dtype=np.float32)]).reshape(-1, 127)
    v = np.concatenate([v, np.full((len(v), 1), 448, dtype=np.float32)], 1)
    q, s = L.spec_quantize_f8(dev(v))
    assert (s == 1).all() and np.array_equal(codes_of(q), f8.encode(v))


def test_quantize_extremes():
    """The largest and smallest values, NaN and infinities; tensors without rows
    and with more than two dimensions; unaligned tensors."""
    v = np.zeros((6, 256), dtype=np.float32)
    v[0, :] = 3.4e38
    v[1, :] = 1e-45
    v[2, :128], v[2, 128:] = 1e-38, -3e-38
    v[3, 5], v[3, 6] = np.nan, 2.0
    v[4, 130], v[4, 131] = np.inf, 2.0
    v[5, 7] = -np.inf
    q, s = L.spec_quantize_f8(dev(v))
    c, s = f8.VALUES[codes_of(q)], s.cpu().numpy()
    want, ws = f8.quantize(v[:3])
    assert np.array_equal(codes_of(q)[:3], want) and np.array_equal(s[:3], ws)
    assert np.isnan(c[3, 5]) and c[3, 6] == 448 and s[3, 0] == np.float32(2) * (np.float32(1) / np.float32(448))
    assert np.isnan(c[4, 130]) and c[4, 131] == 0 and np.isinf(s[4, 1]) and np.isnan(c[5, 7])
    q, s = L.spec_quantize_f8(torch.empty((0, 300), device="cuda"))
    assert q.shape == (0, 300) and s.shape == (0, 3)
    t = torch.randn((2, 3, 200), device="cuda")
    q, s = L.spec_quantize_f8(t)
    assert q.shape == (2, 3, 200) and s.shape == (2, 3, 2)
    odd = torch.randn(1 + 3 * 256, device="cuda")[1:].view(3, 256)
    q, s = L.spec_quantize_f8(odd)
    want, ws = f8.quantize(odd.cpu().numpy())
    assert np.array_equal(codes_of(q), want) and np.array_equal(s.cpu().numpy(), ws)


def head(rng, N, K, power=False):
    """Codes [N, K] and scales of a head, on the GPU."""
    w = f8.encode(np.clip(100 * rng.standard_normal((N, K)), -448, 448).astype(np.float32))
    shape = (-(-N // 128), -(-K // 128))
    s = 2.0 ** rng.integers(-3, 2, shape) if power else 0.001 * np.exp(rng.standard_normal(shape))
    return dev(w), dev(s, torch.float32)


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("R,K,N", SHAPES)
def test_exact_integers(R, K, N, out):
    """Codes of the integers -8..8 with hidden scales of 1, 2 and 4: a block's sums stay within 2^13, and every
    later partial sum is a multiple of 2^-3 of at most 2^24 such steps (with codes up to 3 where there are more blocks)."""
    rng = np.random.default_rng(R * 7919 + K * 31 + N)
    KB = -(-K // 128)
    most = 8 if KB <= 32 else 3
    h = f8.encode(rng.integers(-most, most + 1, (R, K)).astype(np.float32))
    w = f8.encode(rng.integers(-most, most + 1, (N, K)).astype(np.float32))
    hs = (2.0 ** rng.integers(0, 3, (R, KB))).astype(np.float32)
    ws = (2.0 ** rng.integers(-3, 2, (-(-N // 128), KB))).astype(np.float32)
    assert 128 * most * most * 4 * 2 * KB * 8 <= 2 ** 24
    got = L.spec_logits_f8(dev(h).view(torch.float8_e4m3fn), dev(w), dev(ws), dev(hs), out_dtype=TYPES[out])
    ref = f8.product(h, hs, w, ws)[0]
    assert torch.equal(got.cpu(), torch.from_numpy(ref).float().to(TYPES[out])), (R, K, N)


@pytest.mark.parametrize("x,out", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("R,K,N", SHAPES)
def test_real_values(R, K, N, x, out):
    rng = np.random.default_rng(R * 104729 + K * 17 + N)
    h = dev(rng.standard_normal((R, K)) * np.where(rng.random(K) < 0.02, 20, 1), TYPES[x])
    w, s = head(rng, N, K)
    got = host(L.spec_logits_f8(h, w.view(torch.float8_e4m3fn), s, out_dtype=TYPES[out]))
    codes, hs = f8.quantize(host(h).astype(np.float32))
    ref, bound = f8.product(codes, hs, w.cpu().numpy(), s.cpu().numpy(), codes_as_they_are=out == "bf16" and R > 64)
    tol = bound + HALF[out] * (np.abs(ref) + bound)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (R, K, N, np.argwhere(bad)[:4], np.abs(got - ref).max())


@pytest.mark.parametrize("R,out", [(1, "bf16"), (2, "fp32"), (70, "bf16")])
def test_the_longest_k(R, out):
    """K = 2^16: not even one row fits the streaming kernel's LDS.  Integers, as above."""
    rng = np.random.default_rng(R)
    K, N = L.SL_MAX_K, 140
    KB = K // 128
    h, w = (f8.encode(rng.integers(-2, 3, (n, K)).astype(np.float32)) for n in (R, N))
    hs = (2.0 ** rng.integers(0, 3, (R, KB))).astype(np.float32)
    ws = (2.0 ** rng.integers(-3, 2, (2, KB))).astype(np.float32)
    assert 128 * 2 * 2 * 4 * 2 * KB * 8 <= 2 ** 24
    got = L.spec_logits_f8(dev(h).view(torch.float8_e4m3fn), dev(w), dev(ws), dev(hs), out_dtype=TYPES[out])
    assert torch.equal(got.cpu(), torch.from_numpy(f8.product(h, hs, w, ws)[0]).float().to(TYPES[out]))


@pytest.mark.parametrize("R", [3, 40, 300])
def test_given_codes_are_the_same_call(R):
    """Hidden states quantised before the call give the same bits."""
    rng = np.random.default_rng(R)
    h = dev(rng.standard_normal((R, 400)), torch.bfloat16)
    hd = L.F8Head.quantize(dev(rng.standard_normal((515, 400)), torch.bfloat16))
    q, s = L.spec_quantize_f8(h)
    a = hd(h, out_dtype=torch.float32)
    b = L.spec_logits_f8(q, hd.weights, hd.scales, s, out_dtype=torch.float32)
    assert torch.equal(a, b) and L.spec_logits_f8(q, hd.weights, hd.scales, s).dtype == torch.bfloat16
    # every code of the head is within half a step of what it was made from, so logits are near
    assert hd.weights.shape == (515, 400) and hd.scales.shape == (5, 4)


@pytest.mark.parametrize("R", [4, 70])
def test_nan_stays_in_its_row(R):
    rng = np.random.default_rng(R)
    h = dev(rng.standard_normal((R, 300 // 16 * 16)), torch.float32)
    w, s = head(rng, 200, 288)
    good = L.spec_logits_f8(h, w, s)
    h[1, 7], h[3, 200] = float("nan"), float("inf")
    got = L.spec_logits_f8(h, w, s)
    bad = torch.zeros(R, dtype=torch.bool, device="cuda")
    bad[[1, 3]] = True
    assert got[bad].isnan().all() and torch.equal(got[~bad], good[~bad])
    w[9, 100] = 0x7F
    col = L.spec_logits_f8(h, w, s)
    assert col[:, 9].isnan().all() and torch.equal(col[~bad][:, 10:], good[~bad][:, 10:])


@pytest.mark.parametrize("R", [1, 16, 20, 200])
def test_writes_its_output_only(R):
    """A guarded output, and rows that the workgroups' tiles go beyond."""
    rng = np.random.default_rng(R)
    w, s = head(rng, 333, 160)
    h = dev(rng.standard_normal((R, 160)), torch.bfloat16)
    buf = torch.full((R * 333 + 64,), -7.0, dtype=torch.bfloat16, device="cuda")
    L.spec_logits_f8(h, w, s, out=buf[32:32 + R * 333].view(R, 333))
    assert (buf[:32] == -7).all() and (buf[32 + R * 333:] == -7).all()
    assert torch.equal(buf[32:32 + R * 333].view(R, 333), L.spec_logits_f8(h, w, s))


def test_empty_and_3d():
    rng = np.random.default_rng(0)
    w, s = head(rng, 50, 64)
    assert L.spec_logits_f8(torch.empty((0, 64), device="cuda"), w, s).shape == (0, 50)
    h = torch.randn((2, 3, 64), device="cuda")
    assert torch.equal(L.spec_logits_f8(h, w, s), L.spec_logits_f8(h.view(6, 64), w, s).view(2, 3, 50))


@pytest.mark.parametrize("R", [1, 40])
def test_captured_and_on_a_stream(R):
    """A captured call replayed with new values, and a call on a stream of its own."""
    rng = np.random.default_rng(5)
    w, s = head(rng, 700, 256)
    h = dev(rng.standard_normal((R, 256)), torch.bfloat16)
    out = torch.empty((R, 700), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    L.spec_logits_f8(h, w, s, out=out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, L.spec_logits_f8(h, w, s))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.spec_logits_f8(h, w, s, out=out)
        q, qs = L.spec_quantize_f8(h)
    for i in range(3):
        h.copy_(dev(rng.standard_normal((R, 256)), torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, L.spec_logits_f8(h, w, s)), i
        assert torch.equal(qs, L.spec_quantize_f8(h)[1]), i
        assert torch.equal(q.view(torch.uint8), L.spec_quantize_f8(h)[0].view(torch.uint8)), i


def test_binding_refusals():
    z = lambda *shape, dtype=torch.float32: torch.zeros(shape, dtype=dtype, device="cuda")
    w, s, h = z(40, 64, dtype=torch.uint8), z(1, 1), z(3, 64)
    L.spec_logits_f8(h, w, s)
    for bad in (lambda: L.spec_logits_f8(h, w, z(2, 1)), lambda: L.spec_logits_f8(h, w, z(1, 2)),
                lambda: L.spec_logits_f8(z(3, 48), w, s), lambda: L.spec_logits_f8(h, w, s, out=z(3, 41)),
                lambda: L.spec_logits_f8(h, w[:, ::2], s), lambda: L.spec_logits_f8(h.half(), w, s),
                lambda: L.spec_logits_f8(h, w.int(), s), lambda: L.spec_logits_f8(h, w, s.double()),
                lambda: L.spec_logits_f8(h, w, s, hidden_scales=z(3, 1)), lambda: L.spec_logits_f8(h, w, s.cpu()),
                lambda: L.spec_logits_f8(h, w, s, out=z(3, 40), out_dtype=torch.bfloat16),
                lambda: L.spec_logits_f8(z(3, 64, dtype=torch.uint8), w, s),
                lambda: L.spec_quantize_f8(h, rows=64), lambda: L.spec_quantize_f8(z(2, 3, 64), rows=128),
                lambda: L.spec_quantize_f8(h.half()), lambda: L.spec_quantize_f8(h, codes=z(3, 63, dtype=torch.uint8)),
                lambda: L.spec_quantize_f8(h, scales=z(3, 2)), lambda: L.spec_quantize_f8(h.t())):
        with pytest.raises((ValueError, TypeError)):
            bad()
    with pytest.raises(L.SpecLogitsError):      # K is no multiple of 16
        L.spec_logits_f8(z(3, 72), z(40, 72, dtype=torch.uint8), s)
    with pytest.raises(L.SpecLogitsError):      # the output is the input
        L.spec_logits_f8(h, z(64, 64, dtype=torch.uint8), s, out=h)
