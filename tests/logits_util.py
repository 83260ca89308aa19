"""Inputs and comparisons shared by the tests of the logits operators."""
import numpy as np
import torch

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
# Half a step, relative to the value.
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -126, "fp32": 2.0 ** -126}


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def host(t):
    """A tensor's exact values, as float64 or int64."""
    t = t.detach().cpu()
    return (t.double() if t.is_floating_point() else t.long()).numpy()


def make_head(rng, N, K, group, scale="bf16", zeros=True, power=False):
    """Random weights, scales (powers of two with `power`) and zeros, on the GPU."""
    w = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    if power:
        s = 2.0 ** rng.integers(-3, 2, (N, K // group))
    else:
        s = 0.02 * np.exp(0.4 * rng.standard_normal((N, K // group)))
    z = rng.integers(0, 16, (N, K // group), dtype=np.uint8) if zeros else None
    return dev(w), dev(s, TYPES[scale]), None if z is None else dev(z)


def head_arrays(w, s, z):
    return w.cpu().numpy(), host(s), None if z is None else z.cpu().numpy()


def zipf(rng, shape, V):
    return np.minimum((rng.random(shape) ** 3 * V).astype(np.int64), V - 1).astype(np.int32)


def pack_masks(allowed):
    """[M, V] booleans -> [M, ceil(V/32)] int32."""
    M, V = allowed.shape
    W = (V + 31) // 32
    bits = np.zeros((M, W * 32), dtype=np.uint64)
    bits[:, :V] = allowed
    words = (bits.reshape(M, W, 32) << np.arange(32, dtype=np.uint64)).sum(2)
    return words.astype(np.uint32).view(np.int32)
