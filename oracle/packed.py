"""Plain float64 forms of the operators on matrices of 4-bit weights with group scales: the
values of a packed matrix, the product with it and the gradient of its rows, and a whole
mixture-of-experts layer for a few tokens. Nothing is shared with the HIP path."""
from __future__ import annotations

import numpy as np

from . import formats as F


def codes(q: np.ndarray) -> np.ndarray:
    """u8 [..., K/2] -> the 4-bit codes [..., K], low nibble first."""
    return np.stack([q & 15, q >> 4], axis=-1).reshape(*q.shape[:-1], -1)


def values(w: dict) -> np.ndarray:
    """The matrix a packed dict stands for: fmt "nvfp4", "mxfp4" or "int4"; q, s (bytes, or the
    scales' values for int4), z or None, g (nvfp4), group (int4)."""
    c = codes(w["q"])
    if w["fmt"] == "int4":
        zero = 8.0 if w["z"] is None else np.repeat((w["z"] & 15).astype(np.float64), w["group"], -1)
        return (c - zero) * np.repeat(w["s"].astype(np.float64), w["group"], -1)
    v = F.e2m1_value(c).astype(np.float64)
    if w["fmt"] == "mxfp4":
        return v * np.repeat(F.e8m0_value(w["s"]).astype(np.float64), 32, -1)
    g = np.asarray(w["g"], np.float64).reshape(-1, *[1] * (c.ndim - 1)) if c.ndim == 3 else float(w["g"][0])
    return v * np.repeat(F.e4m3_value(w["s"]).astype(np.float64), 16, -1) * g


def linear(x, W, base=None):
    y = x.astype(np.float64) @ W.T
    return y if base is None else y + base


def linear_backward(dy, W, dbase=None):
    dx = dy.astype(np.float64) @ W
    return dx if dbase is None else dx + dbase


def mlp(x, w13, w2):
    half = w13.shape[0] // 2
    a, b = w13[:half] @ x, w13[half:] @ x
    return w2 @ (a / (1.0 + np.exp(-a)) * b)


def tokens(x, router, w13, w2, k, base=None, shared=None) -> dict:
    """y, ids and weights of a layer: router [E, H], w13 [E, 2I, H], w2 [E, H, I], shared (w13, w2,
    gate or None) or None."""
    x = x.astype(np.float64)
    logits = x @ router.astype(np.float64).T
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :k]
    y = np.zeros((x.shape[0], w2.shape[1]))
    if base is not None:
        y += base
    p = np.zeros(ids.shape)
    for t in range(x.shape[0]):
        top = logits[t, ids[t]]
        e = np.exp(top - top[0])
        p[t] = e / e.sum()
        for j in range(k):
            y[t] += p[t, j] * mlp(x[t], w13[ids[t, j]], w2[ids[t, j]])
        if shared is not None:
            s13, s2, gate = shared
            g = 1.0 if gate is None else 1.0 / (1.0 + np.exp(-(x[t] @ gate.astype(np.float64))))
            y[t] += g * mlp(x[t], s13, s2)
    return {"y": y, "ids": ids, "w": p}
