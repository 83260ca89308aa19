"""What the operators around the verify step have to do, and how fast they do it.

Three operators stand between a model and the verify / sampling calls:

* ``w4``       logits from hidden states and a head of 4-bit weights with group scales;
* ``process``  penalties for repeated tokens, biases and grammar masks on those logits;
* ``history``  the state of the penalties: which tokens a sequence holds, and how often.

``run`` computes them in elementary torch operations, or, where ``own`` is true, with this
package's kernels on the same inputs.
"""
import math

import torch

own = False

DEV = "cuda"
INT_MIN = -(1 << 31)
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}


def listed():
    w4 = dict(op="w4", x="bf16", scale="bf16", out="bf16", zeros=False)
    pr = dict(op="process", dtype="bf16", first=0, bias=0, masks=0, ragged=False, inplace=False, penalties=True)
    return [
        # One sequence's drafter step: a small model's head, one row.
        dict(w4, name="w4 1x2048x32000 g64", R=1, K=2048, N=32000, group=64),
        # One sequence's bonus position of a large vocabulary, zero points per group.
        dict(w4, name="w4 1x4096x152064 g128 z", R=1, K=4096, N=152064, group=128, zeros=True),
        # fp32 hidden states and logits over the tiny test vocabulary: all latency.
        dict(w4, name="w4 5x512x1000 g32 fp32", R=5, K=512, N=1000, group=32, x="fp32", scale="fp32", out="fp32", zeros=True),
        # A drafter step of 32 sequences; an odd vocabulary.
        dict(w4, name="w4 32x4096x128255 g128", R=32, K=4096, N=128255, group=128),
        # The target's rows of a verify: 64 sequences of 4 drafts and a bonus position.
        dict(w4, name="w4 320x4096x128256 g128 z", R=320, K=4096, N=128256, group=128, zeros=True),
        # One sequence's drafter step: its repetition, presence and frequency penalties.
        dict(pr, name="process 1x1x32000", B=1, J=1, V=32000, hist=300, first=3),
        # The target's rows of the largest verify, with penalties that follow the drafts.
        dict(pr, name="process 256x8x152064", B=256, J=8, V=152064, hist=2000),
        # Constrained decoding: ragged drafts, a grammar mask per position, biases and penalties.
        dict(pr, name="process 128x9x128256 masks", B=128, J=9, V=128256, hist=1200, bias=300, masks=64, ragged=True),
        # Many short fp32 rows.
        dict(pr, name="process 1000x5x1000 fp32", B=1000, J=5, V=1000, hist=150, bias=8, dtype="fp32"),
        # Grammar masks alone, in place, over an odd vocabulary.
        dict(pr, name="mask in place 64x5x128255", B=64, J=5, V=128255, hist=0, masks=32, inplace=True, penalties=False),
        # Eight sequences enter: their slots are cleared and take prompts of 4096 tokens.
        dict(op="history", name="history prompts 8x4096", S=256, B=8, T=4096, V=152064, prompt=True, old=3000),
        # Every slot starts again from one verify's output tokens (with their padding).
        dict(op="history", name="history outputs 256x8", S=256, B=256, T=8, V=128256, prompt=False, old=500),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["w4", "w4", "process", "process", "history"])
    V = _log(rng, 1000, 152064)
    if op == "w4":
        group = rng.choice([32, 64, 128])
        K = group * max(1, _log(rng, 256, 8192) // group)
        R = _log(rng, 1, 320)
        while R * K * V > 320 * 4096 * 128256:
            R = (R + 1) // 2
        return dict(op=op, R=R, K=K, N=V, group=group, x=rng.choice(["bf16", "bf16", "fp32"]),
                    scale=rng.choice(["bf16", "fp32"]), out=rng.choice(["bf16", "fp32"]), zeros=rng.random() < 0.5)
    if op == "process":
        J, B = rng.randint(1, 9), _log(rng, 1, 256)
        while B * J * V > 256 * 8 * 152064 // 2:
            B = (B + 1) // 2
        pen = rng.random() < 0.8
        inplace = not pen and rng.random() < 0.5
        return dict(op=op, dtype=rng.choice(["bf16", "fp32"]), B=B, J=J, V=V, hist=_log(rng, 1, 4000) if pen else 0,
                    first=rng.randint(0, 3), bias=0 if inplace else rng.choice([0, 1, 17, 300]), masks=rng.choice([0, 1, 16] if pen else [1, 16]),
                    ragged=rng.random() < 0.5, inplace=inplace, penalties=pen)
    B = _log(rng, 1, 256)
    return dict(op=op, S=B + rng.randint(0, 9), B=B, T=_log(rng, 1, max(8, 32768 // B)), V=V, prompt=rng.random() < 0.5,
                old=_log(rng, 1, 3000))


# ---------------------------------------------------------------------------------------------------------------------
# Inputs.


def _tokens(gen, shape, V):
    """Token ids, frequent ones at low ids as tokenizers order them."""
    u = torch.rand(shape, generator=gen, device=DEV)
    return (u * u * u * V).long().clamp_(max=V - 1)


def _history(gen, S, V, n):
    """counts, ids and num of S sequences that hold n tokens each, about a third of them from the prompt."""
    counts = torch.zeros((S, V), dtype=torch.int32, device=DEV)
    if n:
        t = _tokens(gen, (S, n), V)
        k = n // 3
        counts.scatter_add_(1, t[:, k:], torch.ones_like(t[:, k:], dtype=torch.int32))
        seen = torch.zeros((S, V), dtype=torch.bool, device=DEV).scatter_(1, t[:, :k], True)
        counts = torch.where(seen, counts | INT_MIN, counts)
    held = counts != 0
    ids = torch.full((S, V), -1, dtype=torch.int32, device=DEV)
    row, col = held.nonzero(as_tuple=True)
    ids[row, (held.cumsum(1) - 1)[row, col]] = col.int()
    return dict(counts=counts, ids=ids, num=held.sum(1).int())


def _prepare_w4(c, gen):
    R, K, N, G = c["R"], c["K"], c["N"], c["K"] // c["group"]
    x = torch.randn((R, K), generator=gen, device=DEV)
    # a few channels of a hidden state are much larger than the rest
    loud = torch.rand((K,), generator=gen, device=DEV) < 0.01
    x = torch.where(loud, 6 * x, x)
    q = torch.randn((N, K), generator=gen, device=DEV, dtype=torch.float16).mul_(2.6).add_(7.5)
    q = q.round_().clamp_(0, 15).byte()
    s = 0.012 * torch.exp(0.3 * torch.randn((N, G), generator=gen, device=DEV))
    st = dict(hidden=x.to(TYPES[c["x"]]), weights=q[:, 0::2] | (q[:, 1::2] << 4), scales=s.to(TYPES[c["scale"]]), zeros=None)
    if c["zeros"]:
        st["zeros"] = torch.randint(6, 11, (N, G), generator=gen, device=DEV, dtype=torch.uint8)
    st["out"] = torch.empty((R, N), dtype=TYPES[c["out"]], device=DEV)
    return st


def _prepare_process(c, gen):
    B, J, V, n = c["B"], c["J"], c["V"], c["first"] + c["J"] - 1
    st = dict(logits=(3 * torch.randn((B, J, V), generator=gen, device=DEV)).to(TYPES[c["dtype"]]), first=c["first"])
    st["out"] = st["logits"] if c["inplace"] else torch.zeros_like(st["logits"])
    st["drafts"] = _tokens(gen, (B, n), V).int() if n and c["penalties"] else None
    st.update(_history(gen, B, V, c["hist"]) if c["penalties"] else dict(counts=None, ids=None, num=None))
    st["slots"] = torch.randperm(B, generator=gen, device=DEV).int() if c["penalties"] else None
    for name, lo, hi in (("repetition", 1.0, 1.3), ("presence", -0.5, 1.0), ("frequency", 0.0, 0.6)):
        st[name] = lo + (hi - lo) * torch.rand((B,), generator=gen, device=DEV) if c["penalties"] else None
    st["bias_ids"] = st["bias_values"] = None
    if c["bias"]:
        nb = min(c["bias"], V)
        # no id twice, and lists that end early
        ids = torch.randint(0, V, (B, 1), generator=gen, device=DEV) + torch.arange(nb, device=DEV) * (V // nb)
        st["bias_ids"] = (ids % V).int()
        st["bias_ids"][:, nb - nb // 4:] = -1
        st["bias_values"] = 4 * torch.randn((B, nb), generator=gen, device=DEV)
    st["masks"] = st["mask_rows"] = None
    if c["masks"]:
        W = (V + 31) // 32
        dense = torch.tensor([0.002, 0.05, 0.97, 0.4], device=DEV)[torch.arange(c["masks"], device=DEV) % 4]
        bits = torch.rand((c["masks"], W, 32), generator=gen, device=DEV) < dense[:, None, None]
        st["masks"] = (bits.long() << torch.arange(32, device=DEV)).sum(2).to(torch.int32)
        st["mask_rows"] = torch.randint(-1, c["masks"], (B, J), generator=gen, device=DEV, dtype=torch.int32)
    st["rows"] = (1 + torch.arange(B, device=DEV) % J).int() if c["ragged"] else None
    return st


def _prepare_history(c, gen):
    st = _history(gen, c["S"], c["V"], c["old"])
    st["slots"] = torch.randperm(c["S"], generator=gen, device=DEV)[:c["B"]].int()
    t = _tokens(gen, (c["B"], c["T"]), c["V"]).int()
    # tokens end early and are padded with -1
    length = torch.randint(1, c["T"] + 1, (c["B"], 1), generator=gen, device=DEV)
    st["tokens"] = torch.where(torch.arange(c["T"], device=DEV) < length, t, -1)
    st["prompt"] = c["prompt"]
    return st


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    st = {"w4": _prepare_w4, "process": _prepare_process, "history": _prepare_history}[case["op"]](case, gen)
    st["op"] = case["op"]
    return st


# ---------------------------------------------------------------------------------------------------------------------
# The operators in plain form.


def _plain_w4(st):
    w, s, x = st["weights"], st["scales"].float(), st["hidden"].float()
    N, G = s.shape
    q = torch.stack((w & 15, w >> 4), 2).view(N, G, -1).float()
    z = 8.0 if st["zeros"] is None else st["zeros"].float()[:, :, None]
    st["out"].copy_(x @ ((q - z) * s[:, :, None]).view(N, -1).t())
    return st["out"]


def _plain_process(st):
    B, J, V = st["logits"].shape
    z = st["logits"].float()
    if st["counts"] is not None:
        word = st["counts"][st["slots"].long()][:, None, :].expand(B, J, V)
        count = word & 0x7FFFFFFF
        if st["drafts"] is not None:
            n = st["drafts"].shape[1]
            sees = torch.arange(n, device=z.device) < st["first"] + torch.arange(J, device=z.device)[:, None]
            drafts = st["drafts"].long()[:, None, :].expand(B, J, n)
            count = count.contiguous().scatter_add_(2, drafts, sees.int().expand(B, J, n).contiguous())
        col = {k: st[k][:, None, None] for k in ("repetition", "presence", "frequency")}
        z = torch.where((word < 0) | (count > 0), torch.where(z > 0, z / col["repetition"], z * col["repetition"]), z)
        z = z - col["frequency"] * count.float() - torch.where(count > 0, col["presence"], 0.0)
    if st["bias_ids"] is not None:
        ids = st["bias_ids"].long()
        add = torch.where(ids >= 0, st["bias_values"], 0.0)
        z = z.scatter_add(2, ids.clamp(min=0)[:, None, :].expand(B, J, -1), add[:, None, :].expand(B, J, -1))
    if st["masks"] is not None:
        bit = torch.arange(V, device=z.device)
        allowed = (st["masks"][:, bit // 32] >> (bit % 32)) & 1 == 1
        rows = st["mask_rows"].long()
        z = torch.where(allowed[rows.clamp(min=0)] | (rows < 0)[:, :, None], z, -math.inf)
    if st["rows"] is not None:
        z = torch.where((torch.arange(J, device=z.device) < st["rows"][:, None])[:, :, None], z, st["out"].float())
    st["out"].copy_(z)
    return st["out"]


def _plain_history(st):
    t, slots, V = st["tokens"].long(), st["slots"].long(), st["counts"].shape[1]
    n = torch.zeros((t.shape[0], V + 1), dtype=torch.int32, device=t.device)
    n.scatter_add_(1, torch.where(t < 0, V, t), torch.ones_like(t, dtype=torch.int32))
    n = n[:, :V]
    st["counts"][slots] = torch.where(n > 0, INT_MIN, 0).int() if st["prompt"] else n
    st["num"][slots] = (n > 0).sum(1).int()
    return st["counts"], st["num"]


# ---------------------------------------------------------------------------------------------------------------------
# The same with this package's kernels.


def _own_w4(st):
    from speculative_sampling_verification_verify_amd import logits as L
    return L.spec_logits_w4(st["hidden"], st["weights"], st["scales"], st["zeros"], out=st["out"])


def _own_process(st):
    from speculative_sampling_verification_verify_amd import logits as L
    history = None if st["counts"] is None else L.History(st["counts"], st["ids"], st["num"])
    return L.spec_process_logits(st["logits"], out=st["out"], history=history, slots=st["slots"],
                                 draft_tokens=st["drafts"], first=st["first"], repetition=st["repetition"],
                                 presence=st["presence"], frequency=st["frequency"], bias_ids=st["bias_ids"],
                                 bias_values=st["bias_values"], masks=st["masks"], mask_rows=st["mask_rows"],
                                 rows=st["rows"])


def _own_history(st):
    from speculative_sampling_verification_verify_amd import logits as L
    history = L.History(st["counts"], st["ids"], st["num"])
    L.spec_history_reset(history, st["slots"])
    L.spec_history_append(history, st["tokens"], st["slots"], prompt=st["prompt"])
    return st["counts"], st["num"]


def run(state):
    if own:
        return {"w4": _own_w4, "process": _own_process, "history": _own_history}[state["op"]](state)
    else:
        return {"w4": _plain_w4, "process": _plain_process, "history": _plain_history}[state["op"]](state)


# ---------------------------------------------------------------------------------------------------------------------
# What a pass cannot do without, and its result in 64 bits.


def work(case):
    c = case
    if c["op"] == "w4":
        R, K, N, G = c["R"], c["K"], c["N"], c["K"] // c["group"]
        head = N * K // 2 + N * G * (SIZE[c["scale"]] + (1 if c["zeros"] else 0))
        return {"bytes": head + R * K * SIZE[c["x"]] + R * N * SIZE[c["out"]], "flops": 2 * R * K * N}
    if c["op"] == "process":
        B, J, V = c["B"], c["J"], c["V"]
        rows = sum(1 + b % J for b in range(B)) if c["ragged"] else B * J
        masks = c["masks"] * ((V + 31) // 32) * 4
        if c["inplace"]:   # only what the masks forbid is written
            dense = [(0.002, 0.05, 0.97, 0.4)[m % 4] for m in range(c["masks"])]
            return {"bytes": masks + rows * V * SIZE[c["dtype"]] * sum(1 - d for d in dense) / (len(dense) + 1), "flops": rows * V}
        lists = B * (8 * min(c["hist"], V) + 8 * c["bias"] + 4 * (c["first"] + J - 1))
        return {"bytes": 2 * rows * V * SIZE[c["dtype"]] + masks + lists, "flops": 5 * rows * V}
    # a token is read once, and its count is read and written; what the slot held is read and cleared
    return {"bytes": c["B"] * (12 * c["T"] + 8 * min(c["old"], c["V"])), "flops": c["B"] * c["T"]}


def _exact_w4(st):
    x, w, s = st["hidden"].double(), st["weights"], st["scales"].double()
    N, G = s.shape
    out = torch.empty((x.shape[0], N), dtype=torch.float64, device=x.device)
    half = w.shape[1] // G
    for lo in range(0, N, 16384):   # some head rows at a time
        hi = min(N, lo + 16384)
        part = torch.zeros((x.shape[0], hi - lo), dtype=torch.float64, device=x.device)
        for g in range(G):
            b = w[lo:hi, g * half:(g + 1) * half].int()
            xe, xo = x[:, 2 * g * half:2 * (g + 1) * half:2], x[:, 2 * g * half + 1:2 * (g + 1) * half:2]
            zero = 8.0 if st["zeros"] is None else st["zeros"][lo:hi, g].double()
            dot = xe.contiguous() @ (b % 16).double().t().contiguous()
            dot = dot + xo.contiguous() @ (b // 16).double().t().contiguous()
            part += s[lo:hi, g] * (dot - (xe.sum(1) + xo.sum(1))[:, None] * zero)
        out[:, lo:hi] = part
    return out


def _exact_process(st):
    out = st["out"].double().clone()
    B, J, V = out.shape
    rows = [J] * B if st["rows"] is None else st["rows"].tolist()
    slots = None if st["slots"] is None else st["slots"].tolist()
    which = None if st["mask_rows"] is None else st["mask_rows"].tolist()
    table = None
    if st["masks"] is not None:
        table = torch.stack([(st["masks"] >> i) & 1 for i in range(32)], 2).flatten(1)[:, :V].bool()
    par = {k: None if st[k] is None else st[k].double().tolist() for k in ("repetition", "presence", "frequency")}
    for b in range(B):
        n = rows[b]
        z = st["logits"][b, :n].double()
        if slots is not None:
            word = st["counts"][slots[b]].long()
            count = (word % (1 << 31)).double().repeat(n, 1)
            if st["drafts"] is not None:
                t = st["drafts"][b].long()
                for j in range(n):
                    count[j].index_add_(0, t[:st["first"] + j], torch.ones_like(t[:st["first"] + j], dtype=torch.float64))
            rho, pres, freq = par["repetition"][b], par["presence"][b], par["frequency"][b]
            held = (word < 0) | (count >= 1)
            z = torch.where(held & (z > 0), z / rho, torch.where(held, z * rho, z)) - (count >= 1) * pres - count * freq
        if st["bias_ids"] is not None:
            ok = st["bias_ids"][b] >= 0
            extra = torch.zeros(V, dtype=torch.float64, device=z.device)
            z = z + extra.index_add_(0, st["bias_ids"][b][ok].long(), st["bias_values"][b][ok].double())
        if table is not None:
            for j in range(n):
                if which[b][j] >= 0:
                    z[j] = z[j].masked_fill(~table[which[b][j]], -math.inf)
        out[b, :n] = z
    return out


def exact(case, seed):
    if case["op"] == "history":   # whole numbers
        return None
    return {"w4": _exact_w4, "process": _exact_process}[case["op"]](prepare(case, seed))
