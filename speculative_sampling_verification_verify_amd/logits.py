"""ctypes binding of libspeclogits.so (the C ABI in include/spec_logits.h): the
operators between a model and the verify / sampling calls of ``binding``.

Argument marshalling only, as in ``binding``: the functions keep the C names.
``History`` holds the three arrays of a token history, ``W4Head`` a 4-bit and
``F8Head`` an 8-bit head, and ``LogitProcessor`` what a batch of sequences asks
of its logits; the last three are also taken by ``binding.Verifier`` and ``binding.Sampler``.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import NamedTuple, Optional

import torch

from .binding import SV_BF16, SV_OK, _check, _dtype_code

_HERE = os.path.dirname(os.path.abspath(__file__))
# The in-tree build; SL_LIBRARY names another build of the same source (the
# host-sanitized one the ABI tests also run against).
LIB_PATH = os.environ.get("SL_LIBRARY") or os.path.join(_HERE, "libspeclogits.so")

SL_MAX_K = 65536
SL_MAX_ROWS = 1 << 20
SL_MAX_DRAFT = 64
SL_MAX_BIAS = 1024
SL_MAX_MASKS = 1 << 20

SL_F8 = 2
SL_BF16_F8 = 4
SL_F8_BLOCK = 128

EXPORTED = ("spec_logits_w4", "spec_logits_w4_workspace_bytes", "spec_quantize_f8", "spec_logits_f8",
            "spec_logits_f8_workspace_bytes", "spec_history_append", "spec_history_reset", "spec_process_logits",
            "spec_logits_strerror")

_lib = None


class SpecLogitsError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where} failed with {code}: {spec_logits_strerror(code)}")
        self.code = code


def lib() -> ctypes.CDLL:
    """Load the HIP library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing; build it with __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.spec_logits_w4_workspace_bytes.argtypes = [i, i, i, i]
        L.spec_logits_w4_workspace_bytes.restype = sz
        L.spec_logits_w4.argtypes = [vp, i, vp, vp, i, vp, i, i, i, i, vp, i, vp, sz, vp]
        L.spec_logits_w4.restype = i
        L.spec_quantize_f8.argtypes = [vp, i, i, i, i, vp, vp, vp]
        L.spec_quantize_f8.restype = i
        L.spec_logits_f8_workspace_bytes.argtypes = [i, i, i]
        L.spec_logits_f8_workspace_bytes.restype = sz
        L.spec_logits_f8.argtypes = [vp, i, vp, vp, vp, i, i, i, vp, i, vp, sz, vp]
        L.spec_logits_f8.restype = i
        L.spec_history_append.argtypes = [vp, vp, vp, i, i, vp, vp, i, i, i, vp]
        L.spec_history_append.restype = i
        L.spec_history_reset.argtypes = [vp, vp, vp, i, i, vp, i, vp]
        L.spec_history_reset.restype = i
        L.spec_process_logits.argtypes = [vp, vp, i, vp, vp, vp, i, vp, vp, i, i, vp, vp, vp, vp, vp, i, vp, i, vp, vp,
                                          i, i, i, vp]
        L.spec_process_logits.restype = i
        L.spec_logits_strerror.argtypes = [i]
        L.spec_logits_strerror.restype = ctypes.c_char_p
        _lib = L
    return _lib


def spec_logits_strerror(code: int) -> str:
    return lib().spec_logits_strerror(code).decode()


def _gpu(t: torch.Tensor, name: str) -> torch.device:
    dev = t.device
    if dev.type != "cuda":
        raise ValueError(f"{name} must live in GPU memory")
    return dev


def _arg(t: Optional[torch.Tensor], name: str, dtype, shape, dev) -> Optional[int]:
    """The checked tensor's address (None for None); `shape` is a tuple.  These
    checks are a good part of a small call's time, hence the one expression."""
    if t is None:
        return None
    if not (t.dtype is dtype and t.shape == shape and t.device == dev and t.is_contiguous()):
        _check(t, name, dtype, shape, dev)
    return t.data_ptr()


# torch.cuda.current_stream makes a Stream object; the handle is all that is needed.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(fn, where: str, dev: torch.device, stream, *args) -> None:
    """Enqueue on `stream` (None: the current stream of the tensors' device,
    which need not be the current device)."""
    if stream is None:
        h = _raw_stream(dev.index)
    else:
        h = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if torch.cuda.device_count() == 1 or dev.index == torch.cuda.current_device():
        rc = fn(*args, h or None)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, h or None)
    if rc != SV_OK:
        raise SpecLogitsError(rc, where)


def on_stream(stream, dev: Optional[torch.device] = None):
    """A context in which torch allocates and computes on `stream` (a torch
    stream, a handle of one of `dev`, or None: the current one).  Handle 0 is the
    default stream, which ExternalStream does not give; a handle names no device
    (dev None: the current one), and memory must come from the stream that uses
    it."""
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        h = int(stream)
        stream = torch.cuda.ExternalStream(h, device=dev) if h else torch.cuda.default_stream(dev)
    return torch.cuda.stream(stream)


# ---------------------------------------------------------------------------
# Logits from a 4-bit head.
# ---------------------------------------------------------------------------
def spec_logits_w4(hidden: torch.Tensor, weights: torch.Tensor, scales: torch.Tensor,
                   zeros: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   out_dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """out[..., n] = sum_k (w[n, k] - zeros[n, k // group]) * scales[n, k // group] * hidden[..., k].

    hidden [..., K] bf16 or fp32; weights [N, K / 2] uint8 (even k in the low
    four bits); scales [N, K / group] bf16 or fp32; zeros [N, K / group] uint8
    or None (8).  `out` [..., N] or a new tensor of out_dtype (hidden's).  The
    workspace of many rows is torch's, allocated on the stream for the call."""
    if hidden.dim() < 1 or weights.dim() != 2 or scales.dim() != 2:
        raise ValueError("hidden must be [..., K], weights [N, K / 2] and scales [N, K / group]")
    dev = _gpu(hidden, "hidden")
    lead, K = hidden.shape[:-1], hidden.shape[-1]
    N, G = scales.shape
    R = lead.numel()
    xt, st = _dtype_code(hidden), _dtype_code(scales)
    x = _arg(hidden, "hidden", hidden.dtype, hidden.shape, dev)
    w = _arg(weights, "weights", torch.uint8, (N, K // 2), dev)
    s = _arg(scales, "scales", scales.dtype, (N, G), dev)
    z = _arg(zeros, "zeros", torch.uint8, (N, G), dev)
    if K == 0 or G == 0 or N == 0 or K % G:
        raise ValueError(f"scales: {G} groups do not divide K = {K}")
    if out is None:
        with on_stream(stream, dev):
            out = torch.empty((*lead, N), dtype=out_dtype or hidden.dtype, device=dev)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"out: expected {out_dtype}, got {out.dtype}")
    o = _arg(out, "out", out.dtype, (*lead, N), dev)
    need = lib().spec_logits_w4_workspace_bytes(xt, K // G, R, K)
    ws = None
    if need:
        with on_stream(stream, dev):
            ws = torch.empty(need, dtype=torch.uint8, device=dev)
    _call(_lib.spec_logits_w4, "spec_logits_w4", dev, stream, x, xt, w, s, st, z, K // G, R, K, N, o, _dtype_code(out),
          None if ws is None else ws.data_ptr(), need)
    return out


class W4Head:
    """A head of 4-bit weights: called with hidden states, gives their logits."""

    def __init__(self, weights: torch.Tensor, scales: torch.Tensor, zeros: Optional[torch.Tensor] = None):
        self.weights, self.scales, self.zeros = weights, scales, zeros
        self.N, self.K = weights.shape[0], 2 * weights.shape[1]

    def __call__(self, hidden, out=None, out_dtype=None, stream=None):
        return spec_logits_w4(hidden, self.weights, self.scales, self.zeros, out, out_dtype, stream)


# ---------------------------------------------------------------------------
# 8-bit floating point with a scale for each block of 128.
# ---------------------------------------------------------------------------
_F8 = torch.float8_e4m3fn


def _codes(t: torch.Tensor, name: str, shape, dev) -> int:
    """The address of a tensor of e4m3 codes (float8_e4m3fn, or uint8 bit patterns)."""
    return _arg(t, name, torch.uint8 if t.dtype is torch.uint8 else _F8, shape, dev)


def _blocks(n: int) -> int:
    return (n + SL_F8_BLOCK - 1) // SL_F8_BLOCK


def spec_quantize_f8(x: torch.Tensor, rows: int = 1, codes: Optional[torch.Tensor] = None,
                     scales: Optional[torch.Tensor] = None, stream=None):
    """x [..., K] bf16 or fp32 as e4m3 codes [..., K] with one scale for each 128
    values of a row (rows = 1: scales [..., ceil(K / 128)]) or for each tile of
    128 x 128 (rows = 128, x [R, K]: scales [ceil(R / 128), ceil(K / 128)]).
    Returns (codes, scales), new tensors where they are not given."""
    if x.dim() < 1 or (rows != 1 and x.dim() != 2):
        raise ValueError("x must be [..., K], or [R, K] where rows share a scale")
    if rows not in (1, SL_F8_BLOCK):
        raise ValueError(f"rows: 1 or {SL_F8_BLOCK}, got {rows}")
    dev = _gpu(x, "x")
    lead, K = x.shape[:-1], x.shape[-1]
    R = lead.numel()
    p = _arg(x, "x", x.dtype, x.shape, dev)
    xt = _dtype_code(x)
    shape = (*lead, _blocks(K)) if rows == 1 else (_blocks(R), _blocks(K))
    if codes is None or scales is None:
        with on_stream(stream, dev):
            if codes is None:
                codes = torch.empty(x.shape, dtype=_F8, device=dev)
            if scales is None:
                scales = torch.empty(shape, dtype=torch.float32, device=dev)
    _call(lib().spec_quantize_f8, "spec_quantize_f8", dev, stream, p, xt, rows, R, K,
          _codes(codes, "codes", x.shape, dev), _arg(scales, "scales", torch.float32, shape, dev))
    return codes, scales


def spec_logits_f8(hidden: torch.Tensor, weights: torch.Tensor, scales: torch.Tensor,
                   hidden_scales: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   out_dtype: Optional[torch.dtype] = None, stream=None, f8_products: bool = False) -> torch.Tensor:
    """out[..., n] = sum over blocks b of 128 k of hs[..., b] * scales[n // 128, b] *
    sum_{k in b} h[..., k] * weights[n, k].

    weights [N, K] e4m3 codes (float8_e4m3fn, or uint8 bit patterns) with scales
    [ceil(N / 128), ceil(K / 128)] float32.  hidden [..., K] bf16 or fp32, quantised
    in the call as by spec_quantize_f8; or codes, with their hidden_scales [...,
    ceil(K / 128)].  `out` [..., N] or a new tensor of out_dtype (hidden's; bf16
    for codes).  The workspace of many rows is torch's, allocated on the stream
    for the call.

    Sums are held in float32.  With f8_products, an output in bf16 of more than 64
    rows takes the matrix cores' 8-bit products, in half the time: of 8 consecutive
    k they drop what is small beside the largest product (include/spec_logits.h)."""
    if hidden.dim() < 1 or weights.dim() != 2:
        raise ValueError("hidden must be [..., K] and weights [N, K]")
    dev = _gpu(hidden, "hidden")
    lead, K = hidden.shape[:-1], hidden.shape[-1]
    N, R = weights.shape[0], lead.numel()
    if hidden_scales is None:
        xt = _dtype_code(hidden)
        x, xs = _arg(hidden, "hidden", hidden.dtype, hidden.shape, dev), None
    else:
        xt, x = SL_F8, _codes(hidden, "hidden", hidden.shape, dev)
        xs = _arg(hidden_scales, "hidden_scales", torch.float32, (*lead, _blocks(K)), dev)
    w = _codes(weights, "weights", (N, K), dev)
    s = _arg(scales, "scales", torch.float32, (_blocks(N), _blocks(K)), dev)
    if out is None:
        with on_stream(stream, dev):
            out = torch.empty((*lead, N), dtype=out_dtype or (torch.bfloat16 if xt == SL_F8 else hidden.dtype), device=dev)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"out: expected {out_dtype}, got {out.dtype}")
    o, ot = _arg(out, "out", out.dtype, (*lead, N), dev), _dtype_code(out)
    if f8_products:
        if ot != SV_BF16:
            raise ValueError("f8_products: only an output in bf16 can be formed by 8-bit products")
        ot = SL_BF16_F8
    need = lib().spec_logits_f8_workspace_bytes(ot, R, K)
    ws = None
    if need:
        with on_stream(stream, dev):
            ws = torch.empty(need, dtype=torch.uint8, device=dev)
    _call(_lib.spec_logits_f8, "spec_logits_f8", dev, stream, x, xt, xs, w, s, R, K, N, o, ot,
          None if ws is None else ws.data_ptr(), need)
    return out


class F8Head:
    """A head of 8-bit floating-point weights: called with hidden states, gives their
    logits (f8_products: as in spec_logits_f8, for logits in bf16)."""

    def __init__(self, weights: torch.Tensor, scales: torch.Tensor, f8_products: bool = False):
        self.N, self.K = self._sizes(weights)
        _check(scales, "scales", scales.dtype, (_blocks(self.N), _blocks(self.K)), scales.device)
        self.weights, self.scales, self.f8_products = weights, scales, f8_products

    @staticmethod
    def _sizes(weights):
        if weights.dim() != 2:
            raise ValueError("weights must be [N, K]")
        N, K = weights.shape
        if K % 16 or not 0 < K <= SL_MAX_K:
            raise ValueError(f"a head's K is a multiple of 16 of at most {SL_MAX_K}, got {K}")
        return N, K

    @classmethod
    def quantize(cls, weights: torch.Tensor, stream=None, f8_products: bool = False) -> "F8Head":
        """The head of bf16 or fp32 weights [N, K], quantised."""
        cls._sizes(weights)
        return cls(*spec_quantize_f8(weights, SL_F8_BLOCK, stream=stream), f8_products)

    def __call__(self, hidden, out=None, out_dtype=None, stream=None):
        return spec_logits_f8(hidden, self.weights, self.scales, None, out, out_dtype, stream, self.f8_products)


# ---------------------------------------------------------------------------
# The token history.
# ---------------------------------------------------------------------------
class History(NamedTuple):
    """Token history of S slots over a vocabulary of V (see spec_logits.h):
    counts [S, V], ids [S, V] and num [S], int32."""
    counts: torch.Tensor
    ids: torch.Tensor
    num: torch.Tensor

    @classmethod
    def new(cls, S: int, V: int, device="cuda") -> "History":
        z = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=device)
        return cls(z(S, V), z(S, V), z(S))


def _history_args(history: History):
    """(counts, ids, num, S, V) as the C entry points take them, and the device."""
    counts, ids, num = history
    if counts.dim() != 2:
        raise ValueError("history.counts must be [S, V]")
    dev = _gpu(counts, "history.counts")
    shape = counts.shape
    S, V = shape
    return (_arg(counts, "history.counts", torch.int32, shape, dev), _arg(ids, "history.ids", torch.int32, shape, dev),
            _arg(num, "history.num", torch.int32, (S,), dev), S, V), dev


def spec_history_append(history: History, tokens: torch.Tensor, slots: Optional[torch.Tensor] = None,
                        prompt: bool = False, stream=None) -> None:
    """Add tokens [B, T] (int32; ids outside the vocabulary, such as the -1 that
    pads a verify's out_tokens, are skipped) to the history of slots [B]
    (None: 0..B-1), as output tokens or as prompt tokens."""
    h, dev = _history_args(history)
    if tokens.dim() != 2:
        raise ValueError("tokens must be [B, T]")
    B, T = tokens.shape
    t = _arg(tokens, "tokens", torch.int32, (B, T), dev)
    s = _arg(slots, "slots", torch.int32, (B,), dev)
    if T == 0:
        return
    _call(lib().spec_history_append, "spec_history_append", dev, stream, *h, s, t, B, T, 1 if prompt else 0)


def spec_history_reset(history: History, slots: Optional[torch.Tensor] = None, stream=None) -> None:
    """Empty the given slots [B] (int32), or with None every slot."""
    h, dev = _history_args(history)
    B = h[3] if slots is None else slots.numel()
    _call(lib().spec_history_reset, "spec_history_reset", dev, stream, *h, _arg(slots, "slots", torch.int32, (B,), dev), B)


# ---------------------------------------------------------------------------
# Penalties, biases and masks.
# ---------------------------------------------------------------------------
def spec_process_logits(logits: torch.Tensor, out: Optional[torch.Tensor] = None,
                        history: Optional[History] = None, slots: Optional[torch.Tensor] = None,
                        draft_tokens: Optional[torch.Tensor] = None, first: int = 0,
                        repetition: Optional[torch.Tensor] = None, presence: Optional[torch.Tensor] = None,
                        frequency: Optional[torch.Tensor] = None, bias_ids: Optional[torch.Tensor] = None,
                        bias_values: Optional[torch.Tensor] = None, masks: Optional[torch.Tensor] = None,
                        mask_rows: Optional[torch.Tensor] = None, rows: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """Penalties for repeated tokens, biases and grammar masks on logits
    [B, J, V] or [B, V], in place or into `out` (see spec_logits.h).

    Row (b, j) sees the history of slots[b] (None: slot b) and the first
    `first + j` of draft_tokens[b] (rows may be strided).  repetition, presence,
    frequency [B] float32; bias_ids [B, NB] int32 with bias_values [B, NB]
    float32; masks [M, ceil(V / 32)] int32 bits with mask_rows [B, J] int32 (-1:
    no mask); rows [B] int32: rows j >= rows[b] are left alone."""
    shape = logits.shape
    if len(shape) not in (2, 3):
        raise ValueError("logits must be [B, J, V] or [B, V]")
    dev = _gpu(logits, "logits")
    B, V = shape[0], shape[-1]
    J = shape[1] if len(shape) == 3 else 1
    dt = _dtype_code(logits)
    z = _arg(logits, "logits", logits.dtype, shape, dev)
    if out is None:
        out = logits
    o = _arg(out, "out", logits.dtype, shape, dev)
    h = (None, None, None, 0)
    if history is not None:
        h, hdev = _history_args(history)
        if h[4] != V or hdev != dev:
            raise ValueError(f"history is for V = {h[4]} on {hdev}, the logits have V = {V} on {dev}")
        h = h[:4] if h[3] else (None, None, None, 0)
    elif slots is not None:
        raise ValueError("slots without a history")
    s = _arg(slots, "slots", torch.int32, (B,), dev)
    d, stride = None, 0
    if draft_tokens is not None:
        n = first + J - 1
        if draft_tokens.dim() != 2 or draft_tokens.shape[0] != B or draft_tokens.shape[1] < n:
            raise ValueError(f"draft_tokens: expected [{B}, >= {n}], got {tuple(draft_tokens.shape)}")
        if draft_tokens.dtype != torch.int32:
            raise TypeError(f"draft_tokens: expected torch.int32, got {draft_tokens.dtype}")
        if draft_tokens.device != dev:
            raise ValueError(f"draft_tokens is on {draft_tokens.device}, expected {dev}")
        row, col = draft_tokens.stride()
        if col != 1 and draft_tokens.shape[1] > 1:
            raise ValueError("draft_tokens must be contiguous along its rows")
        if n > 0:
            d, stride = draft_tokens.data_ptr(), row if B > 1 else n
    f32, i32, per = torch.float32, torch.int32, (B,)
    rep, pres, freq = _arg(repetition, "repetition", f32, per, dev), _arg(presence, "presence", f32, per, dev), \
        _arg(frequency, "frequency", f32, per, dev)
    if (bias_ids is None) != (bias_values is None) or (masks is None) != (mask_rows is None):
        raise ValueError("bias_ids and bias_values, and masks and mask_rows, go together")
    NB, bi, bv = 0, None, None
    if bias_ids is not None:
        NB = bias_ids.shape[-1]
        bi, bv = _arg(bias_ids, "bias_ids", i32, (B, NB), dev), _arg(bias_values, "bias_values", f32, (B, NB), dev)
        if NB == 0:
            bi = bv = None
    M, mt, mr = 0, None, None
    if masks is not None:
        M = masks.shape[0]
        mt = _arg(masks, "masks", i32, (M, (V + 31) // 32), dev)
        mr = _arg(mask_rows, "mask_rows", i32, (B, J) if len(shape) == 3 or mask_rows.dim() == 2 else per, dev)
        if M == 0:
            raise ValueError("masks is empty")
    _call(lib().spec_process_logits, "spec_process_logits", dev, stream, z, o, dt, *h, s if h[3] else None, d, stride,
          int(first), rep, pres, freq, bi, bv, NB, mt, M, mr, _arg(rows, "rows", i32, per, dev), B, J, V)
    return out


class LogitProcessor:
    """What B sequences ask of their logits: their history and slots, their
    penalties and biases, and the table of grammar masks.  Called with logits,
    adjusts them in place (or into `out`).  With masks, every call says by
    mask_rows which of them a row takes (-1: none)."""

    def __init__(self, history: Optional[History] = None, slots: Optional[torch.Tensor] = None,
                 repetition: Optional[torch.Tensor] = None, presence: Optional[torch.Tensor] = None,
                 frequency: Optional[torch.Tensor] = None, bias_ids: Optional[torch.Tensor] = None,
                 bias_values: Optional[torch.Tensor] = None, masks: Optional[torch.Tensor] = None):
        self.history, self.slots = history, slots
        self.repetition, self.presence, self.frequency = repetition, presence, frequency
        self.bias_ids, self.bias_values, self.masks = bias_ids, bias_values, masks

    def __call__(self, logits, draft_tokens=None, first=0, mask_rows=None, rows=None, out=None, stream=None):
        return spec_process_logits(logits, out, self.history, self.slots, draft_tokens, first, self.repetition,
                                   self.presence, self.frequency, self.bias_ids, self.bias_values,
                                   self.masks, mask_rows, rows, stream)

    def append(self, tokens, stream=None):
        """Add a verify's out_tokens [B, T] (or a prompt's, with history calls of
        one's own) to the sequences' history."""
        if self.history is None:
            raise ValueError("the processor has no history")
        spec_history_append(self.history, tokens, self.slots, stream=stream)
