"""spec_process_logits out of place where a workgroup takes its rows through the
LDS tile in several passes: enough sequences that a workgroup has many rows, and
rows whose 16-byte units lie otherwise from one to the next (V odd, or rows that
start between units), so that a place in the tile holds a unit of one row and
single elements of another.

In float32 the kernel follows the chain operation by operation, so fp32 rows
are compared for equality, and bf16 rows with that chain rounded once."""
import numpy as np
import pytest
import torch

from speculative_sampling_verification_verify_amd import logits as L
from logits_util import TYPES, dev, pack_masks, zipf

pytestmark = pytest.mark.gpu

# (B, J, V): many pieces of a row, one row a pass (8 passes); several short rows a pass; a few pieces
SHAPES = [(40, 8, 50257), (600, 5, 1003), (600, 9, 517), (130, 9, 9001)]


def chain(z, prompt, output, drafts, par, bias, allowed, rows, out):
    """The float32 chain on the touched values alone; z, out [B, J, V] float32."""
    B, J, V = z.shape
    f32 = np.float32
    for b in range(B):
        rho, pres, freq = (par[k][b] for k in ("repetition", "presence", "frequency"))
        add = {}
        for v, x in zip(bias[0][b].tolist(), bias[1][b]):
            if 0 <= v < V:
                add[v] = x if v not in add else add[v] + x
        ids = np.array(list(add), dtype=np.int64)
        vals = np.array(list(add.values()), dtype=f32)
        base = np.bincount(output[b], minlength=V)
        held = np.zeros(V, dtype=bool)
        held[prompt[b]] = True
        for j in range(min(max(rows[b], 0), J)):
            n = base.copy()
            np.add.at(n, drafts[b, :j], 1)
            v = np.nonzero(held | (n > 0))[0]
            x, c = z[b, j, v], n[v]
            x = np.where(x > 0, x / rho, x * rho)
            x = x - freq * c.astype(f32)
            x = x - np.where(c > 0, pres, f32(0))
            out[b, j] = z[b, j]
            out[b, j, v] = x
            out[b, j, ids] = out[b, j, ids] + vals
            if allowed is not None and allowed[1][b, j] >= 0:
                out[b, j, ~allowed[0][allowed[1][b, j]]] = -np.inf
    return out


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("at", [0, 1])
@pytest.mark.parametrize("masks", [False, True])
@pytest.mark.parametrize("B,J,V", SHAPES)
def test_several_passes(B, J, V, masks, at, dtype):
    rng = np.random.default_rng(V + 7 * at + masks)
    n = B * J * V
    room = torch.full((n + 16,), 9.0, dtype=TYPES[dtype], device="cuda")
    place = torch.full((n + 16,), 5.0, dtype=TYPES[dtype], device="cuda")
    x, out = room[at:at + n].view(B, J, V), place[at:at + n].view(B, J, V)
    gen = torch.Generator(device="cuda").manual_seed(V)
    x.copy_(3 * torch.randn((B, J, V), generator=gen, device="cuda"))
    prompt, output, drafts = zipf(rng, (B, 20), V), zipf(rng, (B, 30), V), zipf(rng, (B, J - 1), V)
    # what a row's last elements and its first hold has to be theirs: touch some of them
    drafts[:, 0], output[:, 0], prompt[:, 0] = V - 1, V - 2, 1
    f = lambda lo, hi: (lo + (hi - lo) * rng.random(B)).astype(np.float32)
    par = dict(repetition=f(0.7, 1.5), presence=f(-0.5, 1), frequency=f(-0.2, 0.7))
    bias = zipf(rng, (B, 6), V), (2 * rng.standard_normal((B, 6))).astype(np.float32)
    allowed = rows = None
    if masks:
        allowed = rng.random((4, V)) < np.array([0.02, 0.97, 0.5, 1.0])[:, None], rng.integers(-1, 4, (B, J)).astype(np.int32)
        rows = rng.integers(0, J + 1, B).astype(np.int32)
    hist = L.History.new(B, V)
    L.spec_history_append(hist, dev(prompt), prompt=True)
    L.spec_history_append(hist, dev(output))
    args = dict(history=hist, draft_tokens=dev(drafts), bias_ids=dev(bias[0]), bias_values=dev(bias[1]),
                **{k: dev(v) for k, v in par.items()})
    if masks:
        args.update(masks=dev(pack_masks(allowed[0])), mask_rows=dev(allowed[1]), rows=dev(rows))
    want = chain(x.float().cpu().numpy(), prompt, output, drafts, par, bias, allowed,
                 np.full(B, J) if rows is None else rows, out.float().cpu().numpy())
    want = torch.from_numpy(want).to(TYPES[dtype])
    for k in range(3):
        out.fill_(5.0)
        L.spec_process_logits(x, out=out, **args)
        got = out.cpu()
        bad = got != want
        assert not bad.any(), (k, int(bad.sum()), bad.nonzero()[:4].tolist())
    assert (place[:at] == 5).all() and (place[at + n:] == 5).all()
