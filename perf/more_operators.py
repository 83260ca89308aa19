"""What the 8-bit head and the min-p calls have to do, and how fast they do it.

* ``quantize``  8-bit floating point (e4m3) with a scale for each block of 128;
* ``f8``        logits from hidden states and a head of 8-bit weights with such scales;
* ``sample``    one token per row: temperature, min-p, top-k and top-p, from given uniforms;
* ``verify``    the verify step with the same processing of target and draft.

``run`` computes them in elementary torch operations, or, where ``own`` is true, with this
package's kernels on the same inputs.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}
TINY = 2.0 ** -126
# Most work of a drawn case.
PRODUCT = 2048 * 4096 * 152064
LOGITS = 256 * 15 * 152064


def listed():
    f8 = dict(op="f8", x="bf16", out="bf16")
    sa = dict(op="sample", dtype="bf16", T=0.8, min_p=0.05, top_k=0, top_p=1.0, off=0)
    ve = dict(op="verify", dtype="bf16", T=0.8, min_p=0.05, top_k=0, top_p=1.0, off=0, ragged=False)
    return [
        # The hidden state of one sequence.
        dict(op="quantize", name="quantize 1x2048", x="bf16", R=1, K=2048, rows=1),
        # A head at load time, in tiles of 128 x 128.
        dict(op="quantize", name="quantize head 128256x4096", x="bf16", R=128256, K=4096, rows=128),
        # One sequence's drafter step over a large vocabulary.
        dict(f8, name="f8 1x4096x152064", R=1, K=4096, N=152064),
        # fp32 states and logits over the tiny vocabulary, a last block of 16: all latency.
        dict(f8, name="f8 5x528x1000 fp32", R=5, K=528, N=1000, x="fp32", out="fp32"),
        # The target's rows of a verify: 64 sequences of 4 drafts and a bonus position.
        dict(f8, name="f8 320x4096x128255", R=320, K=4096, N=128255),
        # The target's rows of the largest verify.
        dict(f8, name="f8 2048x4096x152064", R=2048, K=4096, N=152064),
        # One sequence's drafter step.
        dict(sa, name="sample 1x32000", R=1, V=32000),
        # A drafter step of 256 sequences that use every filter.
        dict(sa, name="sample 256x152064 all", R=256, V=152064, T="mix", top_k=50, top_p=0.95),
        # Many short fp32 rows.
        dict(sa, name="sample 1000x1000 fp32", R=1000, V=1000, dtype="fp32", T=1.3, min_p=0.1),
        # One sequence's verify.
        dict(ve, name="verify 1x4x128256", B=1, G=4, V=128256),
        # The largest verify.
        dict(ve, name="verify 256x7x152064", B=256, G=7, V=152064, T=1.0),
        # Ragged drafts over an odd vocabulary; one sequence in four without min-p.
        dict(ve, name="verify 128x8x128255 mixed", B=128, G=8, V=128255, T="mix", top_p=0.9, off=4, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "f8", "f8", "sample", "sample", "verify", "verify"])
    if op == "quantize":
        rows, K = rng.choice([1, 128]), _log(rng, 100, 8192)
        R = _log(rng, 1, 4096) if rows == 1 else _log(rng, 1000, 128256)
        while R * K > 128256 * 4096:
            R = (R + 1) // 2
        return dict(op=op, x=rng.choice(["bf16", "bf16", "fp32"]), R=R, K=K, rows=rows)
    V = _log(rng, 1000, 152064)
    if op == "f8":
        K, R = 16 * max(1, _log(rng, 256, 8192) // 16), _log(rng, 1, 2048)
        while R * K * V > PRODUCT:
            R = (R + 1) // 2
        return dict(op=op, R=R, K=K, N=V, x=rng.choice(["bf16", "bf16", "fp32"]), out=rng.choice(["bf16", "fp32"]))
    c = dict(op=op, V=V, dtype=rng.choice(["bf16", "bf16", "fp32"]), T=rng.choice([0.6, 1.0, 1.5, "mix"]),
             min_p=rng.choice([0.02, 0.05, 0.1, 0.3]), top_k=rng.choice([0, 0, 5, 50]), top_p=rng.choice([1.0, 1.0, 0.8, 0.95]),
             off=rng.choice([0, 0, 0, 4]))
    if op == "sample":
        R = _log(rng, 1, 1000)
        while R * V > LOGITS // 8:
            R = (R + 1) // 2
        return dict(c, R=R)
    G, B = rng.randint(1, 8), _log(rng, 1, 256)
    while B * (2 * G + 1) * V * SIZE[c["dtype"]] > LOGITS:
        B = (B + 1) // 2
    return dict(c, B=B, G=G, ragged=rng.random() < 0.5)


# ---------------------------------------------------------------------------------------------------------------------
# Inputs.


def _hidden(gen, R, K, dtype):
    x = torch.randn((R, K), generator=gen, device=DEV)
    # a few channels of a hidden state are much larger than the rest
    loud = torch.rand((K,), generator=gen, device=DEV) < 0.01
    return torch.where(loud, 6 * x, x).to(TYPES[dtype])


def _prepare_f8(c, gen):
    N, K = c["N"], c["K"]
    w = torch.empty((N, K), dtype=F8, device=DEV)
    for lo in range(0, N, 16384):   # some head rows at a time
        part = torch.randn((min(N, lo + 16384) - lo, K), generator=gen, device=DEV)
        w[lo:lo + 16384] = (100 * part).clamp_(-448, 448).to(F8)
    s = 2e-4 * torch.exp(0.3 * torch.randn(((N + 127) // 128, (K + 127) // 128), generator=gen, device=DEV))
    return dict(hidden=_hidden(gen, c["R"], K, c["x"]), weights=w, scales=s,
                out=torch.empty((c["R"], N), dtype=TYPES[c["out"]], device=DEV))


def _logits(gen, rows, V, dtype):
    """Logits [rows, V] with a few likely tokens, as a model gives them."""
    z = torch.empty((rows, V), dtype=TYPES[dtype], device=DEV)
    for lo in range(0, rows, 256):
        n = min(rows, lo + 256) - lo
        part = torch.randn((n, V), generator=gen, device=DEV).mul_(3.0)
        part.sub_(torch.rand((n, V), generator=gen, device=DEV).mul_(V).add_(1).log_().mul_(1.1))
        z[lo:lo + n] = part
    return z


def _settings(c, gen, n):
    """temperature, min_p, top_k and top_p of n rows or sequences."""
    if c["T"] == "mix":
        T = torch.tensor([0.0, 0.6, 1.0, 1.3], device=DEV)[torch.randint(0, 4, (n,), generator=gen, device=DEV)]
    else:
        T = torch.full((n,), c["T"], device=DEV)
    min_p = torch.full((n,), c["min_p"], device=DEV)
    if c["off"]:
        min_p[::c["off"]] = 0.0
    return dict(temperature=T, min_p=min_p, k=c["top_k"],
                top_k=torch.full((n,), c["top_k"], dtype=torch.int32, device=DEV) if c["top_k"] else None,
                top_p=torch.full((n,), c["top_p"], device=DEV) if c["top_p"] < 1 else None)


def _call(c, cls, sizes):
    """The object that a user's program keeps for calls of one shape."""
    if not own:
        return None
    from speculative_sampling_verification_verify_amd import binding
    dtype = binding.SV_BF16 if c["dtype"] == "bf16" else binding.SV_FP32
    hints = 0 if c["off"] else binding.SV_HINT_ALL_MIN_P
    return getattr(binding, cls)(*sizes, dtype, hints=hints, min_p=True)


def _prepare_sample(c, gen):
    st = dict(logits=_logits(gen, c["R"], c["V"], c["dtype"]), uniforms=torch.rand((c["R"],), generator=gen, device=DEV))
    st.update(_settings(c, gen, c["R"]), call=_call(c, "Sampler", (c["R"], c["V"])))
    return st


def _prepare_verify(c, gen):
    B, G, V = c["B"], c["G"], c["V"]
    p = _logits(gen, B * (G + 1), V, c["dtype"]).view(B, G + 1, V)
    q = torch.empty((B, G, V), dtype=TYPES[c["dtype"]], device=DEV)
    drafts = torch.empty((B, G), dtype=torch.int32, device=DEV)
    st = _settings(c, gen, B)
    T, mp = st["temperature"][:, None], st["min_p"][:, None]
    for i in range(G):
        # a drafter close to the target, and what it sampled (by scores with Gumbel noise)
        z = p[:, i].float() + 0.5 * torch.randn((B, V), generator=gen, device=DEV)
        q[:, i] = z
        z = q[:, i].float()
        kept = z >= z.amax(1, keepdim=True) + T * mp.clamp(min=1e-9).log()
        noise = -torch.rand((B, V), generator=gen, device=DEV).clamp_(min=1e-12).log_().neg_().log_()
        drafts[:, i] = torch.where(kept, z + T * noise, -math.inf).argmax(1)
    st.update(p=p, q=q, drafts=drafts, uniforms=torch.rand((B, G + 1), generator=gen, device=DEV), gamma=None,
              call=_call(c, "Verifier", (B, G, V)))
    if c["ragged"]:
        st["gamma"] = (1 + torch.arange(B, device=DEV) % G).int()
    return st


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    if case["op"] == "quantize":
        st = dict(x=_hidden(gen, case["R"], case["K"], case["x"]), rows=case["rows"])
    else:
        st = {"f8": _prepare_f8, "sample": _prepare_sample, "verify": _prepare_verify}[case["op"]](case, gen)
    st["op"] = case["op"]
    return st


# ---------------------------------------------------------------------------------------------------------------------
# The operators in plain form.


def _plain_quantize(x, rows):
    R, K = x.shape
    xf = torch.zeros(((R + rows - 1) // rows * rows, (K + 127) // 128 * 128), device=x.device)
    xf[:R, :K] = x
    blocks = xf.view(xf.shape[0] // rows, rows, -1, 128)
    s = (blocks.abs().amax((1, 3)) / 448.0).clamp_(min=TINY)
    q = (blocks / s[:, None, :, None]).to(F8).view(xf.shape)
    return q[:R, :K].contiguous(), s


def _plain_f8(st):
    q, s = _plain_quantize(st["hidden"], 1)
    K, N = q.shape[1], st["out"].shape[1]
    x = q.float() * s.repeat_interleave(128, 1)[:, :K]
    for lo in range(0, N, 32768):   # some head rows at a time
        hi = min(N, lo + 32768)
        w = st["scales"][lo // 128:(hi + 127) // 128].repeat_interleave(128, 0)[:hi - lo].repeat_interleave(128, 1)[:, :K]
        st["out"][:, lo:hi] = x @ (st["weights"][lo:hi].float() * w).t()
    return st["out"]


def _plain_process(z, k, T, min_p, top_p):
    """The processed distributions of rows [n, V] of logits, in 64 bits: what decides lies next to a border."""
    z = z.double()
    first = torch.zeros_like(z).scatter_(1, z.argmax(1, keepdim=True), 1.0)
    top = z.amax(1, keepdim=True)
    Td = T.double()[:, None]
    s = torch.where((min_p[:, None] > 0) & (z < top + Td * min_p.double()[:, None].log()), -math.inf, z)
    if 0 < k < z.shape[1]:
        s = torch.where(s < s.topk(k, 1).values[:, -1:], -math.inf, s)
    e = torch.where(s == -math.inf, 0.0, torch.exp((s - top) / torch.where(Td > 0, Td, 1.0)))
    if top_p is not None:
        v, order = e.sort(1, descending=True)
        cum = v.cumsum(1)
        reach = (cum < top_p.double()[:, None] * cum[:, -1:]).sum(1, keepdim=True).clamp_(max=z.shape[1] - 1)
        e = torch.where(e < v.gather(1, reach), 0.0, e)
    return torch.where(Td > 0, e / e.sum(1, keepdim=True), first)


def _plain_draw(w, u):
    """min{v : C(v) > u Z}, and where rounding leaves none, the last weight above 0."""
    c = w.cumsum(1)
    at = (c <= u.double()[:, None] * c[:, -1:]).sum(1)
    V = w.shape[1]
    last = V - 1 - (w.flip(1) > 0).long().argmax(1)
    return torch.minimum(at, last)


def _plain_sample(st):
    out = torch.empty((st["logits"].shape[0],), dtype=torch.int32, device=DEV)
    prob = torch.empty((st["logits"].shape[0],), device=DEV)
    for lo in range(0, out.shape[0], 256):
        at = slice(lo, lo + 256)
        part = [None if st[k] is None else st[k][at] for k in ("temperature", "min_p", "top_p")]
        p = _plain_process(st["logits"][at], st["k"], *part)
        x = _plain_draw(p, st["uniforms"][at])
        out[at], prob[at] = x.int(), p.gather(1, x[:, None])[:, 0].float()
    return out, prob


def _plain_verify(st):
    p, q, x, u = st["p"], st["q"], st["drafts"].long(), st["uniforms"]
    B, G, V = q.shape
    gamma = torch.full((B,), G, device=DEV) if st["gamma"] is None else st["gamma"].long()
    settings = [st[k] for k in ("k", "temperature", "min_p", "top_p")]
    tokens = torch.full((B, G + 1), -1, dtype=torch.int32, device=DEV)
    alpha, pq = torch.zeros((B, G), device=DEV), torch.zeros((B, G, 2), device=DEV)
    n, open_ = torch.zeros((B,), dtype=torch.int32, device=DEV), torch.ones((B,), dtype=torch.bool, device=DEV)
    for i in range(G + 1):
        pi = _plain_process(p[:, i], *settings)
        drafted = gamma > i
        r, accept = pi, torch.zeros_like(open_)
        if i < G:
            qi = _plain_process(q[:, i], *settings)
            px, qx = pi.gather(1, x[:, i:i + 1])[:, 0], qi.gather(1, x[:, i:i + 1])[:, 0]
            alpha[:, i] = torch.where(drafted, torch.minimum(pi, qi).sum(1), 0.0)
            pq[:, i] = torch.where(drafted[:, None], torch.stack((px, qx), 1), 0.0)
            accept = drafted & (u[:, i].double() * qx < px)
            r = (pi - qi).clamp_(min=0)
            r = torch.where(drafted[:, None] & (r.sum(1, keepdim=True) > 0), r, pi)
        ends = open_ & ~accept & (gamma >= i)
        drawn = _plain_draw(r, u[:, G]).int()
        tokens[:, i] = torch.where(ends, drawn, torch.where(open_ & accept, x[:, min(i, G - 1)].int(), tokens[:, i]))
        open_ = open_ & accept
        n += open_.int()
    return tokens, n, alpha, pq


# ---------------------------------------------------------------------------------------------------------------------
# The same with this package's kernels.


def _own_quantize(st):
    from speculative_sampling_verification_verify_amd import logits as L
    return L.spec_quantize_f8(st["x"], st["rows"])


def _own_f8(st):
    from speculative_sampling_verification_verify_amd import logits as L
    return L.spec_logits_f8(st["hidden"], st["weights"], st["scales"], out=st["out"])


def _own_sample(st):
    tokens = st["call"](st["logits"], st["uniforms"], st["temperature"], st["top_k"], st["top_p"], min_p=st["min_p"])
    return tokens, st["call"].prob


def _own_verify(st):
    return st["call"](st["p"], st["q"], st["drafts"], st["uniforms"], st["temperature"], st["top_k"], st["top_p"],
                      st["gamma"], min_p=st["min_p"])


def run(state):
    op = state["op"]
    if own:
        return {"quantize": _own_quantize, "f8": _own_f8, "sample": _own_sample, "verify": _own_verify}[op](state)
    if op == "quantize":
        return _plain_quantize(state["x"], state["rows"])
    return {"f8": _plain_f8, "sample": _plain_sample, "verify": _plain_verify}[op](state)


# ---------------------------------------------------------------------------------------------------------------------
# What a pass cannot do without, and its result in 64 bits.


def work(case):
    c = case
    if c["op"] == "quantize":
        R, K = c["R"], c["K"]
        blocks = (R + c["rows"] - 1) // c["rows"] * ((K + 127) // 128)
        return {"bytes": R * K * (SIZE[c["x"]] + 1) + 4 * blocks, "flops": 3 * R * K}
    if c["op"] == "f8":
        R, K, N = c["R"], c["K"], c["N"]
        return {"bytes": N * K + 4 * ((N + 127) // 128) * ((K + 127) // 128) + R * K * SIZE[c["x"]] + R * N * SIZE[c["out"]],
                "flops": 2 * R * K * N}
    if c["op"] == "sample":
        return {"bytes": c["R"] * (c["V"] * SIZE[c["dtype"]] + 24), "flops": 2 * c["R"] * c["V"]}
    rows = sum(2 * (1 + b % c["G"]) + 1 for b in range(c["B"])) if c["ragged"] else c["B"] * (2 * c["G"] + 1)
    return {"bytes": rows * c["V"] * SIZE[c["dtype"]] + 24 * c["B"] * (c["G"] + 1), "flops": 2 * rows * c["V"]}


def _exact_quantize(st):
    """The scales alone: which of two codes a value on their border takes is a matter of 32 bits."""
    x, rows = st["x"], st["rows"]
    s = torch.empty(((x.shape[0] + rows - 1) // rows, (x.shape[1] + 127) // 128), dtype=torch.float64, device=x.device)
    for j in range(s.shape[1]):
        biggest = x[:, 128 * j:128 * j + 128].abs().amax(1).double()
        pad = torch.zeros((s.shape[0] * rows,), dtype=torch.float64, device=x.device)
        pad[:len(biggest)] = biggest
        s[:, j] = pad.view(-1, rows).amax(1) / 448
    return None, s.clamp_(min=TINY)


def _exact_f8(st):
    x, w, sw = st["hidden"], st["weights"], st["scales"].double()
    R, K = x.shape
    N = w.shape[0]
    out = torch.zeros((R, N), dtype=torch.float64, device=x.device)
    for j in range(sw.shape[1]):
        xb = x[:, 128 * j:128 * j + 128].float()
        # the 8-bit codes are part of the definition: formed in 32 bits
        s = torch.maximum(xb.abs().amax(1) / 448.0, torch.tensor(TINY, device=x.device))
        q = (xb / s[:, None]).to(F8).double()
        for lo in range(0, N, 16384):
            dot = q @ w[lo:lo + 16384, 128 * j:128 * j + 128].double().t().contiguous()
            dot *= sw[lo // 128:lo // 128 + 128, j].repeat_interleave(128)[:dot.shape[1]]
            out[:, lo:lo + 16384] += s.double()[:, None] * dot
    return out


def _exact_row(z, T, min_p, top_k, top_p):
    """(ids ascending, their probabilities) of one row."""
    z = z.double()
    if T == 0:
        return np.array([int(z.argmax())]), np.array([1.0])
    top = float(z.max())
    ids = (z >= top + T * math.log(min_p)).nonzero()[:, 0] if min_p > 0 else torch.arange(len(z), device=z.device)
    v, ids = z[ids].cpu().numpy(), ids.cpu().numpy()
    keep = np.ones(len(v), dtype=bool)
    if 0 < top_k < len(v):
        keep = v >= np.sort(v)[-top_k]
    e = np.where(keep, np.exp((v - top) / T), 0.0)
    if top_p < 1:
        down = np.argsort(-v, kind="stable")
        at = min(int(np.searchsorted(np.cumsum(e[down]), top_p * e.sum())), len(v) - 1)
        e = np.where(v >= v[down[at]], e, 0.0)
    ids, e = ids[e > 0], e[e > 0]
    return ids, e / e.sum()


def _settings_of(st, b):
    """One row's settings, as numbers."""
    return (float(st["temperature"][b]), float(st["min_p"][b]), st["k"], 1.0 if st["top_p"] is None else float(st["top_p"][b]))


def _exact_sample(st):
    """The probability of the token that the uniform picks."""
    R = st["logits"].shape[0]
    u, prob = st["uniforms"].double().tolist(), np.zeros(R)
    for r in range(R):
        _, p = _exact_row(st["logits"][r], *_settings_of(st, r))
        c = np.cumsum(p)
        prob[r] = p[min(int(np.searchsorted(c, u[r] * c[-1], side="right")), len(p) - 1)]
    return None, prob


def _exact_verify(st):
    """The overlaps and the probabilities of the drafts."""
    B, G, V = st["q"].shape
    gamma = [G] * B if st["gamma"] is None else st["gamma"].tolist()
    drafts = st["drafts"].tolist()
    alpha, pq = np.zeros((B, G)), np.zeros((B, G, 2))
    for b in range(B):
        of = _settings_of(st, b)
        for i in range(gamma[b]):
            (pi, pv), (qi, qv) = _exact_row(st["p"][b, i], *of), _exact_row(st["q"][b, i], *of)
            _, a, c = np.intersect1d(pi, qi, assume_unique=True, return_indices=True)
            alpha[b, i] = np.minimum(pv[a], qv[c]).sum()
            pq[b, i] = pv[pi == drafts[b][i]].sum(), qv[qi == drafts[b][i]].sum()
    return None, None, alpha, pq


def exact(case, seed):
    return {"quantize": _exact_quantize, "f8": _exact_f8, "sample": _exact_sample,
            "verify": _exact_verify}[case["op"]](prepare(case, seed))
