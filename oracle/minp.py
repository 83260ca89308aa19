"""CPU oracle for min-p (test infrastructure only): of a row, the values whose
probability is at least min_p times the largest one's stay, z >= zmax +
T ln(min_p); what is left goes through the processing, sampling and verify of
``oracle.verify``."""
import math

import numpy as np

from . import verify as V


def cut(z, T, min_p):
    """The row with what min-p drops at -inf (T = 0 and min_p <= 0: as it is)."""
    if not T > 0 or not min_p > 0 or not V.row_is_valid(z):
        return z
    return np.where(z < z.max() + float(T) * math.log(float(min_p)), -np.inf, z)


def valid(min_p):
    return float(min_p) <= 1.0   # not NaN


def sample(logits, u, T, top_k, top_p, min_p):
    """Tokens, their probabilities and decision margins."""
    R = len(logits)
    tok, prob, margin = np.full(R, -1, np.int32), np.full(R, np.nan), np.full(R, np.inf)
    for r in range(R):
        z = V.decode_row(logits[r])
        if not valid(min_p[r]):
            continue
        z = cut(z, float(T[r]), min_p[r])
        tok[r], margin[r] = V.sample_row(z, float(u[r]), T[r], int(top_k[r]), float(top_p[r]))
        if tok[r] >= 0:
            prob[r] = V.process(z, float(T[r]), int(top_k[r]), float(top_p[r])).prob[tok[r]]
    return tok, prob, margin


def verify(p, q, draft, u, T, top_k, top_p, min_p, gamma, lenience=None):
    """A list of oracle.verify.SeqResult."""
    out = []
    B, G = draft.shape
    for b in range(B):
        if not valid(min_p[b]):
            out.append(V.invalid_result(G))
            continue
        of = lambda rows: np.stack([cut(V.decode_row(z), float(T[b]), min_p[b]) for z in rows])
        out.append(V.verify_sequence(of(p[b]), of(q[b]), draft[b], u[b], float(T[b]), int(top_k[b]), float(top_p[b]),
                                     int(gamma[b]), 1.0 if lenience is None else float(lenience[b])))
    return out
