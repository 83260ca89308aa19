"""What Verifier, Sampler and LogitProcessor do with calls that they refuse, with
buffers of their own and with streams given as handles."""
import numpy as np
import pytest
import torch

from speculative_sampling_verification_verify_amd import binding, logits as L
from logits_util import dev, make_head, pack_masks, zipf

pytestmark = pytest.mark.gpu

B, G, V, K = 3, 2, 300, 64


class Round:
    """Arguments of one round, and a processor whose penalties change its logits."""

    def __init__(self, dtype=torch.bfloat16):
        rng = np.random.default_rng(8)
        self.rng = rng
        self.history = L.History.new(B, V)
        L.spec_history_append(self.history, dev(zipf(rng, (B, 60), V)))
        self.proc = L.LogitProcessor(self.history, repetition=dev(np.full(B, 1.5, dtype=np.float32)))
        f = lambda *s: dev(rng.random(s).astype(np.float32))
        self.p = dev(rng.standard_normal((B, G + 1, V)), dtype)
        self.q = dev(rng.standard_normal((B, G, V)), dtype)
        self.x = dev(zipf(rng, (B, G), V))
        self.u, self.T = f(B, G + 1), torch.ones(B, device="cuda")
        self.u1 = f(B)
        self.gamma = torch.full((B,), G, dtype=torch.int32, device="cuda")


def test_a_refused_call_leaves_the_logits():
    """What the verify or the sampler refuses is refused before the processor
    has written: the corrected call then adjusts the logits once."""
    r = Round()
    ver, sam = binding.Verifier(B, G, V), binding.Sampler(B, V)
    before = r.p.clone()
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    bad = [dict(q_logits=r.q[:, :, :-1].contiguous()), dict(q_logits=r.q.float()), dict(uniforms=r.u1), dict(uniforms=None),
           dict(temperature=r.T.double()), dict(temperature=r.T[:2]), dict(temperature=None), dict(top_k=r.T), dict(top_p=r.gamma),
           dict(gamma_len=r.gamma[:1]), dict(gamma_len=r.gamma.long()), dict(draft_tokens=r.x.long()), dict(draft_tokens=None),
           dict(lenience=r.u), dict(temperature=r.T.cpu())]
    good = dict(q_logits=r.q, draft_tokens=r.x, uniforms=r.u, temperature=r.T)
    for kw in bad:
        with pytest.raises((ValueError, TypeError, binding.SpecVerifyError)):
            ver(r.p, **{**good, **kw}, processor=r.proc)
        torch.cuda.synchronize()
        assert torch.equal(r.p, before), kw
    big = binding.Verifier(B, G, V // 4)             # its workspace is for shorter rows
    if binding.spec_verify_workspace_bytes(B, G, V, 0) > big.workspace.numel():
        with pytest.raises((ValueError, binding.SpecVerifyError)):
            big(r.p, **good, processor=r.proc)
    hints = binding.Verifier(B, G, V)
    hints.hints = binding.SV_HINT_NO_DENSE | binding.SV_HINT_ALL_DENSE
    with pytest.raises((ValueError, binding.SpecVerifyError)):
        hints(r.p, **good, processor=r.proc)
    torch.cuda.synchronize()
    assert torch.equal(r.p, before)
    ver(r.p, **good, processor=r.proc)
    once = r.proc(before.clone(), r.x)
    assert torch.equal(r.p, once) and not torch.equal(once, before)

    z = dev(r.rng.standard_normal((B, V)), torch.bfloat16)
    before = z.clone()
    for kw in (dict(uniforms=r.u), dict(uniforms=None), dict(temperature=r.T.double()), dict(temperature=None), dict(top_k=r.T),
               dict(top_p=i32(B)), dict(top_p=r.u), dict(uniforms=r.u1.cpu())):
        with pytest.raises((ValueError, TypeError, binding.SpecVerifyError)):
            sam(z, **{**dict(uniforms=r.u1, temperature=r.T), **kw}, processor=r.proc)
        torch.cuda.synchronize()
        assert torch.equal(z, before), kw
    with pytest.raises((ValueError, binding.SpecVerifyError)):
        binding.Sampler(B, V + 1)(z, r.u1, r.T, processor=r.proc)
    with pytest.raises((ValueError, TypeError)):     # refused by the processor itself
        sam(z, r.u1, r.T, processor=r.proc, draft_tokens=r.x.long())
    torch.cuda.synchronize()
    assert torch.equal(z, before)
    sam(z, r.u1, r.T, processor=r.proc)
    assert torch.equal(z, r.proc(before.clone())) and not torch.equal(z, before)


def test_a_wrong_first_call_keeps_no_buffer():
    """Hidden states with a wrong number of rows, or a head of another
    vocabulary, in the first call: refused, and the next call is served."""
    r = Round()
    head = L.W4Head(*make_head(r.rng, V, K, 32))
    other = L.W4Head(*make_head(r.rng, V + 4, K, 32))
    h = lambda *s: dev(r.rng.standard_normal((*s, K)), torch.bfloat16)
    ver, sam = binding.Verifier(B, G, V), binding.Sampler(B, V)
    args = (r.q, r.x, r.u, r.T)
    for bad, by in ((h(B, G), head), (h(B + 1, G + 1), head), (h(B * (G + 1)), head), (h(B, G + 1), other),
                    (h(B, G + 1).cpu(), head)):
        with pytest.raises((ValueError, binding.SpecVerifyError)):
            ver.from_hidden(bad, by, *args)
    good = h(B, G + 1)
    ver.from_hidden(good, head, *args)
    assert torch.equal(ver.p_logits, head(good))
    for bad, by in ((h(B + 1), head), (h(B, 1), head), (h(B), other)):
        with pytest.raises((ValueError, binding.SpecVerifyError)):
            sam.from_hidden(bad, by, r.u1, r.T)
    good = h(B)
    sam.from_hidden(good, head, r.u1, r.T)
    assert torch.equal(sam.logits, head(good))


def test_a_grammar_is_never_dropped():
    """A processor with masks refuses a call that does not say which, before it
    writes anything; so do calls that pick masks where there are none."""
    r = Round()
    allowed = np.zeros((1, V), dtype=bool)
    allowed[0, 5] = True
    proc = L.LogitProcessor(r.history, masks=dev(pack_masks(allowed)))
    ver, sam = binding.Verifier(B, G, V), binding.Sampler(B, V)
    p, z = r.p.clone(), r.p[:, 0].contiguous()
    z0 = z.clone()
    for call in (lambda: proc(p, r.x), lambda: ver(p, r.q, r.x, r.u, r.T, processor=proc), lambda: proc(z),
                 lambda: sam(z, r.u1, r.T, processor=proc)):
        with pytest.raises(ValueError):
            call()
    at = torch.zeros((B, G + 1), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        r.proc(p, r.x, mask_rows=at)         # a processor without masks
    with pytest.raises(ValueError):
        ver(p, r.q, r.x, r.u, r.T, mask_rows=at)
    with pytest.raises(ValueError):
        sam(z, r.u1, r.T, mask_rows=at[:, 0].contiguous())
    torch.cuda.synchronize()
    assert torch.equal(p, r.p) and torch.equal(z, z0)
    assert (sam(z, r.u1, r.T, processor=proc, mask_rows=at[:, 0].contiguous()) == 5).all()
    proc(p, r.x, mask_rows=at - 1)           # -1: no mask
    assert torch.equal(p, r.p)


def test_append_without_a_history():
    with pytest.raises(ValueError, match="no history"):
        L.LogitProcessor(bias_ids=torch.zeros((1, 1), dtype=torch.int32), bias_values=torch.zeros((1, 1))).append(
            torch.zeros((1, 1), dtype=torch.int32))


def test_streams_given_as_handles():
    """Inside on_stream torch works on the stream that the handle names, the
    default stream (handle 0) included, whatever stream is current."""
    gpu, side, other = torch.device("cuda", 0), torch.cuda.Stream(), torch.cuda.Stream()
    for current in (torch.cuda.default_stream(), other):
        with torch.cuda.stream(current):
            for s, h in ((0, 0), (side.cuda_stream, side.cuda_stream), (side, side.cuda_stream), (None, current.cuda_stream),
                         (torch.cuda.default_stream(), 0)):
                with L.on_stream(s, gpu):
                    assert torch.cuda.current_stream().cuda_stream == h
            assert torch.cuda.current_stream() == current


def test_handles_name_no_device(monkeypatch):
    """The stream made of a handle is one of the tensors' device, which need not
    be the current one."""
    made = []
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: made.append((h, device)) or torch.cuda.Stream())
    with L.on_stream(77, torch.device("cuda", 0)):
        pass
    assert made == [(77, torch.device("cuda", 0))]


@pytest.mark.parametrize("handle", [False, True])
def test_rounds_on_the_default_stream(handle):
    """From a side stream, calls that name the default stream: workspaces and
    row limits are made where they are used."""
    r = Round()
    head = L.W4Head(*make_head(r.rng, V, K, 32))
    h = dev(r.rng.standard_normal((40, K)), torch.bfloat16)      # rows that need a workspace
    hb = dev(r.rng.standard_normal((B, G + 1, K)), torch.bfloat16)
    ver = binding.Verifier(B, G, V)
    gamma = torch.tensor([G, 1, G], dtype=torch.int32, device="cuda")
    want, full = head(h), head(hb)
    r.proc(full, r.x, rows=gamma + 1)
    stream = 0 if handle else torch.cuda.default_stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = [head(h, stream=stream) for _ in range(20)]
        ver.from_hidden(hb, head, r.q, r.x, r.u, r.T, gamma_len=gamma, processor=r.proc, stream=stream)
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
    assert torch.equal(ver.p_logits, full)
