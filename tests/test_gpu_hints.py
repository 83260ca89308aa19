"""Hints that no call of an object can use are refused by every call of it, and before a processor writes."""
import pytest
import torch

from speculative_sampling_verification_verify_amd import binding, logits as L

pytestmark = pytest.mark.gpu

R, V, G = 3, 500, 2


def tensors():
    f = torch.full((R,), 0.5, device="cuda")
    u = torch.full((R, G + 1), 0.5, device="cuda")
    return torch.randn((R, V), device="cuda"), torch.randn((R, G + 1, V), device="cuda"), torch.zeros((R, G), dtype=torch.int32, device="cuda"), u, f


def processor():
    return L.LogitProcessor(bias_ids=torch.zeros((R, 1), dtype=torch.int32, device="cuda"), bias_values=torch.ones((R, 1), device="cuda"))


@pytest.mark.parametrize("with_processor", [False, True])
@pytest.mark.parametrize("hints,min_p", [(1, True), (2, False), (4, True), (binding.SV_HINT_ALL_MIN_P, False),
                                         (binding.SV_HINT_ALL_MIN_P | 1, True), (16, True)])
def test_sampler(hints, min_p, with_processor):
    z, _, _, _, f = tensors()
    keep = z.clone()
    sam = binding.Sampler(R, V, binding.SV_FP32, hints=hints, min_p=min_p)
    more = dict(processor=processor()) if with_processor else {}
    for kw in ({}, dict(min_p=f)) if min_p else ({},):
        with pytest.raises(ValueError, match="hint"):
            sam(z, f, f, **kw, **more)
    assert torch.equal(z, keep)


@pytest.mark.parametrize("with_processor", [False, True])
def test_verifier(with_processor):
    _, p, d, u, f = tensors()
    keep, q = p.clone(), p[:, :G].contiguous()
    ver = binding.Verifier(R, G, V, binding.SV_FP32, hints=binding.SV_HINT_ALL_MIN_P)
    more = dict(processor=processor()) if with_processor else {}
    with pytest.raises((ValueError, binding.SpecVerifyError)):
        ver(p, q, d, u, f, **more)
    assert torch.equal(p, keep)


def test_the_hint_is_none_for_calls_without_min_p():
    z, p, d, u, f = tensors()
    sam = [binding.Sampler(R, V, binding.SV_FP32, hints=h, min_p=True) for h in (0, binding.SV_HINT_ALL_MIN_P)]
    a, b = [s(z, f, f).clone() for s in sam]
    assert torch.equal(a, b)
    a, b = [s(z, f, f, min_p=f).clone() for s in sam]
    assert torch.equal(a, b)
    ver = [binding.Verifier(R, G, V, binding.SV_FP32, hints=h, min_p=True) for h in (0, binding.SV_HINT_ALL_MIN_P)]
    for kw in ({}, dict(min_p=f)):
        a, b = [[t.clone() for t in v(p, p[:, :G].contiguous(), d, u, f, **kw)] for v in ver]
        assert all(torch.equal(x, y) for x, y in zip(a, b))
