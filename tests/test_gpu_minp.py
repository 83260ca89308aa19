"""spec_sample_min_p and spec_verify_min_p on the GPU against the float64 oracle.

Probabilities and masses are held in 64 bits on both sides (a mass as a multiple
of 2^-42), so tokens and counts have to be equal wherever the oracle's
decision margin is at least that of V masses, 4 V 2^-42 with a factor to spare, and
there probabilities agree within their rounding to float32 (2^-24)."""
import numpy as np
import pytest
import torch

import oracle
from oracle import minp
from speculative_sampling_verification_verify_amd import binding
from logits_util import TYPES, dev

pytestmark = pytest.mark.gpu
margin_of = lambda V: 4 * (V + 1000) * 2.0 ** -42
NEAR = dict(rtol=2.0 ** -23, atol=1e-12)


def code(dtype):
    return binding.SV_BF16 if dtype == "bf16" else binding.SV_FP32


def bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16) if t.dtype == torch.bfloat16 else t.cpu().numpy()


def logits(rng, shape, dtype, scale=3.0):
    z = scale * rng.standard_normal(shape) - np.log1p(shape[-1] * rng.random(shape))
    return dev(z, TYPES[dtype])


def settings(rng, n):
    """A row's parameters: every filter on and off, argmax, far and near temperatures."""
    return dict(T=rng.choice([0.0, 0.6, 1.0, 1.0, 1.7, 30.0, 1e-3], n).astype(np.float32),
                top_k=rng.choice([0, 0, 1, 5, 50, 700, 1 << 21], n).astype(np.int32),
                top_p=rng.choice([1.0, 1.0, 0.9, 0.5, 0.999, 0.0], n).astype(np.float32),
                min_p=rng.choice([0.05, 0.05, 0.3, 0.001, 1.0, 0.0, -1.0, 1e-9], n).astype(np.float32))


def sample(z, u, s, hints=0):
    R, V = z.shape
    call = binding.Sampler(R, V, code("bf16" if z.dtype == torch.bfloat16 else "fp32"), hints=hints, min_p=True)
    t = call(z, dev(u), dev(s["T"]), dev(s["top_k"]), dev(s["top_p"]), min_p=dev(s["min_p"]))
    return t.cpu().numpy(), call.prob.cpu().numpy()


def check_sample(z, u, s, hints=0):
    tok, prob = sample(z, u, s, hints)
    rt, rp, margin = minp.sample(bits(z), u, s["T"], s["top_k"], s["top_p"], s["min_p"])
    far = margin >= margin_of(z.shape[1])
    assert (tok[far] == rt[far]).all(), np.argwhere(far & (tok != rt))[:4]
    np.testing.assert_allclose(prob[far], rp[far], **NEAR)
    return far.mean()


VOCABS = [1, 2, 7, 64, 1000, 4095, 4097, 16385, 32001, 70001, 152064]


@pytest.mark.parametrize("hints", [0, binding.SV_HINT_ALL_MIN_P])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", VOCABS)
def test_sample(V, dtype, hints):
    rng = np.random.default_rng(V)
    R = 60 if V < 5000 else 24
    s = settings(rng, R)
    assert check_sample(logits(rng, (R, V), dtype), rng.random(R).astype(np.float32), s, hints) > 0.9


@pytest.mark.parametrize("hints", [0, binding.SV_HINT_ALL_MIN_P])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_the_longest_rows(dtype, hints):
    """2^20 values: a row alone has more parts than a position's workgroup has threads."""
    rng = np.random.default_rng(5)
    R, V = 3, 1 << 20
    z = logits(rng, (R, V), dtype)
    s = dict(T=np.array([1.0, 0.7, 1.0], np.float32), top_k=np.array([0, 40, 0], np.int32),
             top_p=np.array([1.0, 0.9, 0.95], np.float32), min_p=np.array([0.1, 0.02, 0.0], np.float32))
    z[:, -1] = z[:, 5] = 16.0   # kept in the first and in the last part
    for r in range(R):          # (one row, whose parts are the shortest, and three)
        one = {k: v[r:r + 1] for k, v in s.items()}
        assert check_sample(z[r:r + 1].contiguous(), rng.random(1).astype(np.float32), one, hints) == 1.0
    u = np.array([0.99, 0.01, 0.5], np.float32)
    check_sample(z, u, s, hints)


def test_a_workspace_of_more_sequences():
    """The C calls take a larger batch's workspace, whose parts are longer."""
    rng = np.random.default_rng(6)
    V, big, R = 32001, 700, 9
    ws = torch.empty(binding.spec_verify_min_p_workspace_bytes(big, 0, V, binding.SV_BF16), dtype=torch.uint8, device="cuda")
    z, s, u = logits(rng, (R, V), "bf16"), settings(rng, R), rng.random(R).astype(np.float32)
    want = sample(z, u, s)
    call = binding.Sampler(R, V, min_p=True)
    call.min_p_workspace = ws
    got = call(z, dev(u), dev(s["T"]), dev(s["top_k"]), dev(s["top_p"]), min_p=dev(s["min_p"]))
    assert (got.cpu().numpy() == want[0]).all()
    np.testing.assert_array_equal(call.prob.cpu().numpy(), want[1])


def test_calls_on_two_streams_at_once():
    """Each with its own workspace, while the other runs."""
    rng = np.random.default_rng(8)
    R, V = 300, 32001
    cases = []
    for _ in range(2):
        z, s, u = logits(rng, (R, V), "bf16"), settings(rng, R), rng.random(R).astype(np.float32)
        cases.append((z, [dev(u), dev(s["T"]), dev(s["top_k"]), dev(s["top_p"])], dev(s["min_p"]), sample(z, u, s)))
    calls = [binding.Sampler(R, V, min_p=True) for _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for (z, args, mp, _), call, st in zip(cases, calls, streams):
            call(z, *args, min_p=mp, stream=st)
    torch.cuda.synchronize()
    for (_, _, _, want), call in zip(cases, calls):
        assert (call.tokens.cpu().numpy() == want[0]).all()
        np.testing.assert_array_equal(call.prob.cpu().numpy(), want[1])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_sample_many_rows(dtype):
    """Enough rows for the longer parts."""
    rng = np.random.default_rng(1)
    R, V = 700, 33000
    s = settings(rng, R)
    assert check_sample(logits(rng, (R, V), dtype), rng.random(R).astype(np.float32), s) > 0.9


@pytest.mark.parametrize("hints", [0, binding.SV_HINT_ALL_MIN_P])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_lists_that_overflow(dtype, hints):
    """Equal values, flat rows and rows that keep just below and just above what
    the lists hold (512 of a part, 1024 of a row)."""
    rng = np.random.default_rng(2)
    V = 50000
    z = np.full((9, V), -20.0)
    z[0] = 1.0                                            # every value the same
    z[1] = 0.01 * rng.standard_normal(V)
    for r, n in ((2, 511), (3, 512), (4, 513), (5, 1023), (6, 1024), (7, 1025)):
        z[r, rng.permutation(V)[:n]] = 2.0 + 0.5 * rng.random(n)
    z[8, 4000:4600] = 3.0                                 # 600 of one part
    R = len(z)
    s = dict(T=np.full(R, 1.0, np.float32), top_k=np.zeros(R, np.int32), top_p=np.full(R, 1.0, np.float32),
             min_p=np.full(R, 0.1, np.float32))
    for top_k, top_p, T in ((0, 1.0, 1.0), (40, 1.0, 1.0), (2000, 0.7, 1.0), (0, 0.9, 2.0), (0, 1.0, 0.0)):
        s.update(top_k=np.full(R, top_k, np.int32), top_p=np.full(R, top_p, np.float32), T=np.full(R, T, np.float32))
        for u in (0.0, 0.37, 0.99999994):
            check_sample(dev(z, TYPES[dtype]), np.full(R, u, np.float32), s, hints)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_masked_and_bad_rows(dtype):
    """Masked values (-inf and the type's lowest), rows with nothing left, NaN
    of both signs and infinities, signed zeros, bad parameters: each row by itself."""
    rng = np.random.default_rng(3)
    V = 5003
    z = logits(rng, (20, V), dtype)
    s = settings(rng, 20)
    s["T"][:], s["min_p"][:], s["top_p"][:], s["top_k"][:] = 1.0, 0.05, 1.0, 0
    low = torch.finfo(z.dtype).min
    z[0, 1:] = -torch.inf
    z[1, :-1] = -torch.inf
    z[2] = -torch.inf
    z[3, ::2], z[4] = low, low
    z[5, 3], z[6, V - 1], z[7, 4096] = torch.nan, -torch.tensor(torch.nan), torch.inf
    z[8] = -torch.inf
    z[8, 100], z[8, 200], z[8, 300] = -0.0, 0.0, -0.0
    z[9] = torch.where(z[9] > -3, -torch.inf, z[9])
    for r, name, v in ((10, "T", -1.0), (11, "T", np.nan), (12, "top_p", np.nan), (13, "min_p", np.nan), (14, "min_p", 1.5),
                       (15, "T", 1e-38), (16, "T", 1e38), (17, "min_p", 1.0)):
        s[name][r] = v
    u = rng.random(20).astype(np.float32)
    u[18], u[19] = 1.0, np.nan
    for hints in (0, binding.SV_HINT_ALL_MIN_P):
        check_sample(z, u, s, hints)
    tok, prob = sample(z, u, s)
    invalid = [2, 5, 6, 7, 10, 11, 12, 13, 14, 18, 19]
    assert (tok[invalid] == -1).all() and np.isnan(prob[invalid]).all()
    assert (np.delete(tok, invalid) >= 0).all()
    s["T"][:] = 0
    check_sample(z, u, s)
    # of a negative NaN's two zeros, the first is the argmax
    assert sample(z, u, s)[0][8] == 100


def test_infinite_temperature():
    """T = inf: every finite value the same (min_p keeps them all)."""
    z = torch.full((2, 1000), -torch.inf, device="cuda")
    z[:, 10:20] = torch.arange(10, device="cuda", dtype=torch.float32)
    s = dict(T=np.full(2, np.inf, np.float32), top_k=np.zeros(2, np.int32), top_p=np.ones(2, np.float32),
             min_p=np.array([0.5, 1.0], np.float32))
    tok, prob = sample(z, np.array([0.05, 0.95], np.float32), s)
    assert tok.tolist() == [10, 19] and np.allclose(prob, 0.1)


def verify_inputs(rng, B, G, V, dtype):
    p = logits(rng, (B, G + 1, V), dtype)
    q = (p[:, :G].float() + dev(0.7 * rng.standard_normal((B, G, V)), torch.float32)).to(TYPES[dtype])
    s = settings(rng, B)
    kept = lambda z, T, m: z >= z.max() + (T * np.log(m) if m > 0 else -np.inf)
    draft = np.zeros((B, G), np.int32)
    qb = bits(q)
    for b in range(B):
        for i in range(G):   # mostly what a sampler of the same settings may have drawn
            z = oracle.decode_row(qb[b, i])
            ids = np.nonzero(kept(z, s["T"][b], s["min_p"][b]))[0]
            draft[b, i] = rng.integers(V) if rng.random() < 0.05 else ids[np.argmax(z[ids] + max(s["T"][b], 1e-6) * rng.gumbel(size=len(ids)))]
    gamma = rng.integers(1, G + 1, B).astype(np.int32)
    u = (rng.random((B, G + 1)) * 0.9).astype(np.float32)
    return p, q, draft, u, gamma, s


def check_verify(p, q, draft, u, gamma, s, hints=0, lenience=None):
    B, G, V = q.shape
    ver = binding.Verifier(B, G, V, code("bf16" if p.dtype == torch.bfloat16 else "fp32"), hints=hints, min_p=True)
    tok, n, alpha, pq = [t.cpu().numpy() for t in ver(
        p, q, dev(draft), dev(u), dev(s["T"]), dev(s["top_k"]), dev(s["top_p"]), dev(gamma), min_p=dev(s["min_p"]),
        lenience=None if lenience is None else dev(lenience))]
    ref = minp.verify(bits(p), bits(q), draft, u, s["T"], s["top_k"], s["top_p"], s["min_p"], gamma, lenience)
    far = 0
    for b, r in enumerate(ref):
        if r.n < 0:
            assert n[b] == -1 and (tok[b] == -1).all() and np.isnan(alpha[b]).all() and np.isnan(pq[b]).all(), b
            continue
        if r.margin >= margin_of(V):
            far += 1
            assert n[b] == r.n and (tok[b] == r.tokens).all(), (b, n[b], r.n, tok[b], r.tokens)
        ok = r.topp_pos >= margin_of(V)
        np.testing.assert_allclose(alpha[b][ok], r.alpha[ok], **NEAR)
        np.testing.assert_allclose(pq[b][ok], r.pq[ok], **NEAR)
    return far / B


@pytest.mark.parametrize("hints", [0, binding.SV_HINT_ALL_MIN_P])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,G,V", [(1, 1, 1), (5, 3, 2), (40, 4, 257), (12, 8, 4099), (6, 5, 40000), (3, 64, 500), (2, 2, 152064)])
def test_verify(B, G, V, dtype, hints):
    rng = np.random.default_rng(B * 100 + G)
    assert check_verify(*verify_inputs(rng, B, G, V, dtype), hints) > 0.85 or B < 10


def test_verify_many():
    """Enough rows for the longer parts, with lenience."""
    rng = np.random.default_rng(9)
    args = verify_inputs(rng, 100, 3, 20011, "bf16")
    check_verify(*args, lenience=rng.random(100).astype(np.float32))


def test_verify_bad_sequences():
    """Bad data in one sequence leaves the others alone."""
    rng = np.random.default_rng(10)
    p, q, draft, u, gamma, s = verify_inputs(rng, 12, 4, 3001, "fp32")
    s["T"][:], s["min_p"][:] = 1.0, 0.05
    gamma[:] = 4
    p[0, 4, 7] = torch.nan
    p[1, 1] = -torch.inf
    q[2, 3, 0] = torch.inf
    draft[3, 2], draft[4, 0] = 3001, -1
    u[5, 1], u[6, 4] = 1.0, np.nan
    s["min_p"][7], s["min_p"][8], s["T"][9] = 1.01, np.nan, -1
    gamma[10] = 2
    p[10, 3:], q[10, 2:], draft[10, 2:] = torch.nan, torch.nan, -5      # padding is not read
    u[10, 2:4] = 7
    check_verify(p, q, draft, u, gamma, s)
    gamma[11] = 5
    ver = binding.Verifier(12, 4, 3001, binding.SV_FP32, min_p=True)
    n = ver(p, q, dev(draft), dev(u), dev(s["T"]), gamma_len=dev(gamma), min_p=dev(s["min_p"]))[1].cpu().numpy()
    assert (n[[0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 11]] == -1).all() and n[10] >= 0


def test_without_min_p_it_is_the_verify():
    """min_p = 0 everywhere gives spec_verify's results (whose dense rows are in 32 bits)."""
    rng = np.random.default_rng(11)
    p, q, draft, u, gamma, s = verify_inputs(rng, 30, 3, 2000, "bf16")
    s["min_p"][:] = 0
    assert check_verify(p, q, draft, u, gamma, s) > 0.8
    ver = binding.Verifier(30, 3, 2000, min_p=True)
    args = (p, q, dev(draft), dev(u), dev(s["T"]), dev(s["top_k"]), dev(s["top_p"]), dev(gamma))
    a = [t.clone() for t in ver(*args)]
    b = ver(*args, min_p=dev(s["min_p"]))
    ref = minp.verify(bits(p), bits(q), draft, u, s["T"], s["top_k"], s["top_p"], s["min_p"], gamma)
    far = torch.tensor([r.margin >= 1e-5 for r in ref], device="cuda")
    assert torch.equal(a[0][far], b[0][far]) and torch.equal(a[1][far], b[1][far])


def test_distribution_of_the_draw():
    """Uniforms on a grid: each token as often as its probability says."""
    rng = np.random.default_rng(12)
    R, V = 4096, 300
    row = logits(rng, (1, V), "fp32")
    z = row.expand(R, V).contiguous()
    s = dict(T=np.full(R, 1.2, np.float32), top_k=np.full(R, 40, np.int32), top_p=np.full(R, 0.95, np.float32),
             min_p=np.full(R, 0.04, np.float32))
    tok, _ = sample(z, ((np.arange(R) + 0.5) / R).astype(np.float32), s)
    pr = oracle.process(minp.cut(row[0].double().cpu().numpy(), float(s["T"][0]), s["min_p"][0]), float(s["T"][0]), 40,
                        float(s["top_p"][0])).prob
    assert np.abs(np.bincount(tok, minlength=V) / R - pr).max() <= 1.01 / R    # a grid of R uniforms


@pytest.mark.parametrize("hints", [0, binding.SV_HINT_ALL_MIN_P])
def test_captured_calls(hints):
    """A sampler and a verifier captured into one graph, replayed with new inputs
    between eager calls of the same objects; lists overflow in some replays only."""
    rng = np.random.default_rng(13)
    B, G, V = 5, 2, 9001
    sam, ver = binding.Sampler(B, V, min_p=True, hints=hints), binding.Verifier(B, G, V, min_p=True, hints=hints)
    p, q, draft, u, gamma, s = verify_inputs(rng, B, G, V, "bf16")
    s["T"][:], s["min_p"][:] = 1.0, 0.05
    d = {k: dev(v) for k, v in dict(draft=draft, u=u, gamma=gamma, **s).items()}
    z, us = p[:, 0].contiguous(), dev(u[:, 0].copy())

    def both():
        a = sam(z, us, d["T"], d["top_k"], d["top_p"], min_p=d["min_p"])
        return (a, sam.prob, *ver(p, q, d["draft"], d["u"], d["T"], d["top_k"], d["top_p"], d["gamma"], min_p=d["min_p"]))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for i in range(4):
        n = verify_inputs(rng, B, G, V, "bf16")
        flat = 0.001 if i == 2 else 1.0
        p.copy_(n[0] * flat), q.copy_(n[1] * flat), z.copy_(p[:, 0])
        d["draft"].copy_(dev(n[2]))
        if i == 3:
            d["min_p"][1] = 0.0
        want = [t.clone() for t in both()]
        for t in (sam.tokens, ver.tokens, ver.n_accepted):
            t.fill_(-9)
        sam.prob.fill_(-9), ver.alpha.fill_(-9), ver.pq.fill_(-9)
        graph.replay()
        torch.cuda.synchronize()
        got = (sam.tokens, sam.prob, ver.tokens, ver.n_accepted, ver.alpha, ver.pq)
        for a, b in zip(got, want):
            assert torch.equal(a, b), i


def test_on_a_stream_and_odd_bases():
    """Another stream, and logits whose base is aligned to an element only."""
    rng = np.random.default_rng(14)
    for dtype in ("bf16", "fp32"):
        R, V = 3, 6000
        flat = torch.empty(R * V + 3, dtype=TYPES[dtype], device="cuda")
        z = flat[3:].view(R, V)
        z.copy_(logits(rng, (R, V), dtype))
        s = settings(rng, R)
        check_sample(z, rng.random(R).astype(np.float32), s)
    call = binding.Sampler(R, V, binding.SV_FP32, min_p=True)
    args = [dev(v) for v in (rng.random(R).astype(np.float32), s["T"], s["top_k"], s["top_p"])]
    want = call(z, *args, min_p=dev(s["min_p"])).clone()
    m = dev(s["min_p"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call.tokens.fill_(-9)
    side.wait_stream(torch.cuda.current_stream())
    call(z, *args, min_p=m, stream=side)
    side.synchronize()
    assert torch.equal(call.tokens, want)


def test_binding_refusals():
    z, f = torch.zeros((2, 100), device="cuda"), torch.full((2,), 0.5, device="cuda")
    sam = binding.Sampler(2, 100, binding.SV_FP32, min_p=True)
    sam(z, f, f, min_p=f)
    plain = binding.Sampler(2, 100, binding.SV_FP32)
    for bad in (lambda: plain(z, f, f, min_p=f), lambda: sam(z, f, f, min_p=f[:1]), lambda: sam(z, f, f, min_p=f.double()),
                lambda: binding.Sampler(2, 100, binding.SV_FP32, hints=1, min_p=True)(z, f, f, min_p=f),
                lambda: sam(z, f, f, min_p=f.cpu())):
        with pytest.raises((ValueError, TypeError)):
            bad()
    p, q = torch.zeros((2, 3, 100), device="cuda"), torch.zeros((2, 2, 100), device="cuda")
    d, u = torch.zeros((2, 2), dtype=torch.int32, device="cuda"), torch.full((2, 3), 0.5, device="cuda")
    ver = binding.Verifier(2, 2, 100, binding.SV_FP32, min_p=True)
    ver(p, q, d, u, f, min_p=f)
    for bad in (lambda: binding.Verifier(2, 2, 100, binding.SV_FP32)(p, q, d, u, f, min_p=f),
                lambda: ver(p, q, d, u, f, min_p=f[:1])):
        with pytest.raises((ValueError, TypeError)):
            bad()
    # the hint for calls with min_p is none for calls without
    binding.Verifier(2, 2, 100, binding.SV_FP32, min_p=True, hints=binding.SV_HINT_ALL_MIN_P)(p, q, d, u, f)
