"""Plain implementations of the logits operators, on the CPU, in float64:
the product with a 4-bit head, the token history, and penalties, biases and
masks.  Written from the formulas, value by value where that is affordable;
``process_rows_f32`` is the same chain in float32 with each operation rounded
by itself, which the kernel follows bit for bit."""
from __future__ import annotations

import numpy as np


def unpack_w4(weights: np.ndarray) -> np.ndarray:
    """[N, K/2] bytes -> [N, K] values 0..15 (even k in the low four bits)."""
    w = np.asarray(weights, dtype=np.uint8)
    out = np.empty((w.shape[0], 2 * w.shape[1]), dtype=np.int64)
    out[:, 0::2] = w & 15
    out[:, 1::2] = w >> 4
    return out


def w4_product(hidden, weights, scales, zeros=None) -> np.ndarray:
    """sum_g s[n, g] * sum_{k in g} (w[n, k] - z[n, g]) * x[r, k], [R, N] float64."""
    q = unpack_w4(weights).astype(np.float64)
    s = np.asarray(scales, dtype=np.float64)
    N, G = s.shape
    K = q.shape[1]
    z = np.full((N, G), 8.0) if zeros is None else (np.asarray(zeros, dtype=np.int64) & 15).astype(np.float64)
    w = ((q.reshape(N, G, K // G) - z[:, :, None]) * s[:, :, None]).reshape(N, K)
    return np.asarray(hidden, dtype=np.float64) @ w.T


def w4_error_bound(hidden, weights, scales, zeros=None, parts: int = 1) -> np.ndarray:
    """How far float32 sums may be from w4_product.  The terms w x of every part
    and z x are summed apart within at most 128 k and then over those entries of
    K.  A term passes at most a rounding for each product of its entry, or the 24
    of its entry's sum of x, then two for each entry (the scaled sum is added, the
    zero points are taken out) and two of its own (the factors s z and z X); a
    column that up to 16 wavefronts share takes 15 additions more.  Every rounding
    is at most 2^-24 of a partial sum, which is at most the sum of the absolute
    terms."""
    q = unpack_w4(weights).astype(np.float64)
    s = np.abs(np.asarray(scales, dtype=np.float64))
    N, G = s.shape
    K = q.shape[1]
    z = np.full((N, G), 8.0) if zeros is None else (np.asarray(zeros, dtype=np.int64) & 15).astype(np.float64)
    w = ((q.reshape(N, G, K // G) + z[:, :, None]) * s[:, :, None]).reshape(N, K)
    entry = min(K // G, 128)
    return 2.0 ** -24 * (max(parts * entry, 24) + 2 * (-(-K // entry)) + 17) * (np.abs(np.asarray(hidden, dtype=np.float64)) @ w.T)


class TokenHistory:
    """counts, in_prompt and the set of held tokens of S slots, as dictionaries."""

    def __init__(self, S: int, V: int):
        self.S, self.V = S, V
        self.out = [dict() for _ in range(S)]
        self.prompt = [set() for _ in range(S)]

    def append(self, tokens, slots=None, prompt=False):
        for b, row in enumerate(np.asarray(tokens)):
            s = b if slots is None else int(slots[b])
            if not 0 <= s < self.S:
                continue
            for v in row.tolist():
                if 0 <= v < self.V:
                    if prompt:
                        self.prompt[s].add(v)
                    else:
                        self.out[s][v] = self.out[s].get(v, 0) + 1

    def reset(self, slots=None):
        for s in range(self.S) if slots is None else [int(x) for x in slots]:
            if 0 <= s < self.S:
                self.out[s], self.prompt[s] = {}, set()

    def counts(self) -> np.ndarray:
        c = np.zeros((self.S, self.V), dtype=np.uint32)
        for s in range(self.S):
            for v, n in self.out[s].items():
                c[s, v] = n
            for v in self.prompt[s]:
                c[s, v] |= np.uint32(0x80000000)
        return c

    def num(self) -> np.ndarray:
        return np.array([len(set(self.out[s]) | self.prompt[s]) for s in range(self.S)])


def _rows_of(rows, b, J):
    return J if rows is None else int(min(max(int(rows[b]), 0), J))


def _process(z_in, out, real, history, slots, drafts, first, repetition, presence, frequency, bias_ids, bias_values,
             masks, mask_rows, rows):
    """The chain in the arithmetic of `real` (np.float64 or np.float32);
    returns the rows and, beside them, the sum of the absolute values that went
    into each (for error bounds)."""
    B, J, V = z_in.shape
    size = np.zeros((B, J, V))
    for b in range(B):
        s = None if history is None else (b if slots is None else int(slots[b]))
        held = s is not None and 0 <= s < history.S
        rho = real(1.0 if repetition is None else repetition[b])
        pres = real(0.0 if presence is None else presence[b])
        freq = real(0.0 if frequency is None else frequency[b])
        for j in range(_rows_of(rows, b, J)):
            z = z_in[b, j].astype(real).copy()
            m = int(mask_rows[b][j]) if mask_rows is not None else -1
            if not (rho > 0 and np.isfinite(rho)) or not np.isfinite(pres) or not np.isfinite(freq) or m < -1 \
                    or (masks is not None and m >= len(masks)):
                out[b, j] = np.nan
                continue
            count = dict(history.out[s]) if held else {}
            prompt = history.prompt[s] if held else set()
            if drafts is not None:
                for v in np.asarray(drafts[b])[:first + j].tolist():
                    if 0 <= v < V:
                        count[v] = count.get(v, 0) + 1
            size[b, j] = np.abs(z)
            with np.errstate(over="ignore", invalid="ignore"):
                for v in set(count) | set(prompt):
                    c = count.get(v, 0)
                    z1 = z[v] / rho if z[v] > 0 else z[v] * rho
                    f = freq * real(c)
                    size[b, j, v] = abs(z1) + abs(f) + (abs(pres) if c else 0.0)
                    z[v] = (z1 - f) - (pres if c else real(0.0))
                if bias_ids is not None:
                    add = {}
                    for v, x in zip(np.asarray(bias_ids[b]).tolist(), np.asarray(bias_values[b])):
                        if 0 <= v < V:
                            add[v] = real(x) if v not in add else add[v] + real(x)
                            size[b, j, v] += abs(float(x))
                    for v, x in add.items():
                        z[v] = z[v] + x
            if m >= 0:
                word = np.asarray(masks)[m].astype(np.int64) & 0xFFFFFFFF
                ok = (word[np.arange(V) // 32] >> (np.arange(V) % 32)) & 1
                z[ok == 0] = -np.inf
            out[b, j] = z
    return out, size


def process_rows(logits, out=None, history=None, slots=None, drafts=None, first=0, repetition=None, presence=None,
                 frequency=None, bias_ids=None, bias_values=None, masks=None, mask_rows=None, rows=None):
    """Penalties, biases and masks in float64; `out` (default: the logits) holds
    what unused rows keep.  Returns (rows, sum of absolute terms)."""
    z = np.asarray(logits, dtype=np.float64)
    o = (z if out is None else np.asarray(out, dtype=np.float64)).copy()
    return _process(z, o, np.float64, history, slots, drafts, first, repetition, presence, frequency, bias_ids,
                    bias_values, masks, mask_rows, rows)


def process_rows_f32(logits, out=None, **kw):
    """The same in float32, each operation rounded by itself."""
    z = np.asarray(logits, dtype=np.float32)
    o = (z if out is None else np.asarray(out, dtype=np.float32)).copy()
    args = dict(history=None, slots=None, drafts=None, first=0, repetition=None, presence=None, frequency=None,
                bias_ids=None, bias_values=None, masks=None, mask_rows=None, rows=None)
    args.update(kw)
    return _process(z, o, np.float32, *args.values())[0]
