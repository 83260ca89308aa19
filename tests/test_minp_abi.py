"""The min-p entry points refuse bad arguments on the host before touching the
GPU (no compute calls here)."""
import pytest

from speculative_sampling_verification_verify_amd import binding as Bn
from test_abi import _ensure_built

FAKE = 0x100000   # never dereferenced: every case below ends on the host


def need(B=2, G=3, V=64, dt=Bn.SV_BF16):
    _ensure_built()
    return Bn.spec_verify_min_p_workspace_bytes(B, G, V, dt)


def verify(p=FAKE, q=FAKE, dt=Bn.SV_BF16, draft=FAKE, gamma=None, u=FAKE, T=FAKE, k=None, tp=None, mp=FAKE, l=None, hints=0,
           B=2, G=3, V=64, tokens=FAKE, n=FAKE, alpha=FAKE, pq=None, ws=FAKE, wsb=None):
    wsb = need() if wsb is None else wsb
    return _ensure_built().spec_verify_min_p(p, q, dt, draft, gamma, u, T, k, tp, mp, l, hints, B, G, V, tokens, n, alpha, pq,
                                             ws, wsb, None)


def sample(z=FAKE, dt=Bn.SV_BF16, u=FAKE, T=FAKE, mp=FAKE, hints=0, R=2, V=64, tokens=FAKE, prob=None, ws=FAKE, wsb=None):
    wsb = need(2, 0) if wsb is None else wsb
    return _ensure_built().spec_sample_min_p(z, dt, u, T, None, None, mp, hints, R, V, tokens, prob, ws, wsb, None)


def test_workspace():
    for dt in (Bn.SV_BF16, Bn.SV_FP32):
        for V in (1, 7, 1000, 16384, 16385, 152064, 1 << 20):
            for G in (0, 1, 8, 64):
                for B in (1, 7, 256):
                    # a record of 32 bytes a position, and a list for each row
                    assert need(B, G, V, dt) >= B * (G + 1) * 32 + B * (2 * G + 1) * 2048, (B, G, V, dt)
    assert need(0) > 0
    for bad in ((-1, 3, 64, 0), (2, -1, 64, 0), (2, 65, 64, 0), (2, 3, 0, 0), (2, 3, (1 << 20) + 1, 0), (2, 3, 64, 5)):
        assert need(*bad) == 0, bad


def test_workspace_serves_smaller_batches():
    """Also where a smaller batch is cut into shorter parts, which take more lists."""
    for dt in (Bn.SV_BF16, Bn.SV_FP32):
        for G, V in ((0, 1), (0, 32000), (4, 128256), (7, 152064), (64, 1000), (1, 1 << 20), (64, 1 << 20)):
            sizes = [need(B, G, V, dt) for B in range(1, 300)] + [need(B, G, V, dt) for B in (500, 1000, 1023, 1024, 1025, 4096)]
            assert sizes == sorted(sizes), (G, V, dt)


def test_verify_refusals():
    assert verify(B=0) == Bn.SV_OK
    assert verify(dt=3) == verify(G=65) == verify(V=(1 << 20) + 1) == Bn.SV_ERR_UNSUPPORTED
    assert verify(B=-1) == verify(G=0) == verify(V=0) == Bn.SV_ERR_ARG
    for k in ("p", "q", "draft", "u", "T", "tokens", "n", "alpha"):
        assert verify(**{k: None}) == Bn.SV_ERR_ARG, k
    assert verify(p=FAKE + 1) == verify(q=FAKE + 1) == verify(p=FAKE + 2, dt=Bn.SV_FP32) == Bn.SV_ERR_ARG
    for hints in (Bn.SV_HINT_NO_DENSE, Bn.SV_HINT_ALL_DENSE, Bn.SV_HINT_UNFILTERED, 16, -1):
        assert verify(hints=hints) == verify(hints=hints | Bn.SV_HINT_ALL_MIN_P) == Bn.SV_ERR_ARG, hints
    assert verify(ws=None) == verify(ws=FAKE + 128) == verify(wsb=need() - 1) == Bn.SV_ERR_WORKSPACE
    big = 1 << 60
    assert verify(B=1 << 17, G=64, V=1 << 20, wsb=big) == Bn.SV_ERR_UNSUPPORTED   # more threads than a launch


def test_sample_refusals():
    assert sample(R=0) == Bn.SV_OK
    assert sample(dt=2) == sample(V=(1 << 20) + 1) == Bn.SV_ERR_UNSUPPORTED
    assert sample(R=-1) == sample(V=0) == Bn.SV_ERR_ARG
    for k in ("z", "u", "T", "tokens"):
        assert sample(**{k: None}) == Bn.SV_ERR_ARG, k
    assert sample(z=FAKE + 1) == sample(z=FAKE + 2, dt=Bn.SV_FP32) == sample(hints=1) == Bn.SV_ERR_ARG
    assert sample(ws=None) == sample(ws=FAKE + 16) == sample(wsb=need(2, 0) - 1) == Bn.SV_ERR_WORKSPACE
    assert sample(R=1 << 30, V=1 << 20, wsb=1 << 62) == Bn.SV_ERR_UNSUPPORTED


def test_the_old_calls_take_no_min_p_hint():
    L = _ensure_built()
    n = Bn.spec_verify_workspace_bytes(2, 3, 64, Bn.SV_BF16)
    assert L.spec_verify_ex(FAKE, FAKE, Bn.SV_BF16, FAKE, None, FAKE, FAKE, None, None, None, Bn.SV_HINT_ALL_MIN_P, 2, 3, 64,
                            FAKE, FAKE, FAKE, None, FAKE, n, None) == Bn.SV_ERR_ARG
