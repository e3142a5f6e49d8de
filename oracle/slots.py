"""One adapter per request, in fp64 (oracle -- test infrastructure only).

A server runs the tokens of many requests over one frozen base, each request
with an adapter of its own ("QLoRA", skillbyai, Merging the adapter for
serving: an unmerged adapter can be swapped over one base; llm-compass,
方法与公式, the displayed formula, per token):
    h[m] = W x[m] + scale_a B_a (A_a x[m]),   a = ids[m]
and only W x[m] where a names no adapter of the table.
"""

from __future__ import annotations

import numpy as np


def token_slots(lengths, slots, n_tokens: int) -> np.ndarray:
    """int32 [n_tokens]: requests one after another, -1 behind the last."""
    out = np.full(n_tokens, -1, dtype=np.int32)
    at = 0
    for n, s in zip(np.asarray(lengths).tolist(), np.asarray(slots).tolist()):
        n = max(0, n)
        out[at:at + n] = s
        at += n
        if at >= n_tokens:
            break
    return out


def linear_fwd_slots(x, W, A, B, scale, ids):
    """(h, size) in fp64: the layer, and the sum of the absolute values of the
    low-rank terms of each output (a bound's scale, not a result)."""
    x, W, A, B = (np.asarray(t, dtype=np.float64) for t in (x, W, A, B))
    scale, ids = np.asarray(scale, dtype=np.float64), np.asarray(ids)
    h = x @ W.T
    size = np.zeros_like(h)
    for m, a in enumerate(ids.tolist()):
        if 0 <= a < A.shape[0]:
            u = scale[a] * (A[a] @ x[m])
            h[m] += B[a] @ u
            size[m] = np.abs(B[a]) @ np.abs(u)
    return h, size
