"""Plain float64 forms of the operators around the experts: the permutation of
tokens into expert order and back, the routing weights' gradient, and low-rank
adapters, each with its gradient. Loops and whole-array products only; nothing
is shared with the HIP path."""
from __future__ import annotations

import numpy as np


def permute_index(ids: np.ndarray, E: int) -> dict:
    """Stable sort of the slots t * k + j by expert; ids outside [0, E) are dropped."""
    flat = np.asarray(ids).reshape(-1)
    order = [s for e in range(E) for s in np.flatnonzero(flat == e)]
    off = np.zeros(E + 1, np.int32)
    for e in range(E):
        off[e + 1] = off[e] + np.count_nonzero(flat == e)
    slot_row = np.full(flat.size, -1, np.int32)
    slot_row[order] = np.arange(len(order))
    sorted_slots = np.full(flat.size, -1, np.int32)
    sorted_slots[:len(order)] = order
    return {"sorted": sorted_slots, "slot_row": slot_row.reshape(np.shape(ids)), "off": off}


def permute(x: np.ndarray, index: dict, rows: np.ndarray) -> np.ndarray:
    """rows with every held row replaced by its token's row."""
    out = np.array(rows)
    k = index["slot_row"].shape[1]
    n = index["off"][-1]
    out[:n] = x[index["sorted"][:n] // k]
    return out


def unpermute(rows: np.ndarray, slot_row: np.ndarray, w: np.ndarray | None) -> np.ndarray:
    """Weighted sum of each token's rows (w None: plain sum, the permutation's gradient)."""
    M, k = slot_row.shape
    y = np.zeros((M, rows.shape[1]))
    for t in range(M):
        for j in range(k):
            r = slot_row[t, j]
            if 0 <= r < M * k:
                y[t] += rows[r].astype(np.float64) * (1.0 if w is None else float(w[t, j]))
    return y


def unpermute_backward(dy, rows, slot_row, w, drows) -> tuple:
    """(drows, dw); rows that no slot names keep what `drows` holds."""
    M, k = slot_row.shape
    dr, dw = np.array(drows, dtype=np.float64), np.zeros((M, k))
    for t in range(M):
        for j in range(k):
            r = slot_row[t, j]
            if 0 <= r < M * k:
                dr[r] = float(w[t, j]) * dy[t].astype(np.float64)
                dw[t, j] = np.dot(dy[t].astype(np.float64), rows[r].astype(np.float64))
    return dr, dw


def route_backward(ids, w, dw, E: int) -> np.ndarray:
    """Gradient of softmax over the selected logits, at the selected logits."""
    M, k = ids.shape
    w, dw = w.astype(np.float64), dw.astype(np.float64)
    out = np.zeros((M, E))
    for t in range(M):
        mean = float(np.dot(w[t], dw[t]))
        for j in range(k):
            if 0 <= ids[t, j] < E:
                out[t, ids[t, j]] += w[t, j] * (dw[t, j] - mean)
    return out


def lora(x, ids, A, B, scale, base) -> tuple:
    """(y, z) of y = base + scale[g] * B[g] (A[g] x) row by row."""
    M, r = x.shape[0], A.shape[1]
    y, z = np.array(base, dtype=np.float64), np.zeros((M, r))
    for g in range(A.shape[0]):
        t = np.flatnonzero(ids == g)
        z[t] = x[t].astype(np.float64) @ A[g].astype(np.float64).T
        y[t] += float(scale[g]) * (z[t] @ B[g].astype(np.float64).T)
    return y, z


def lora_backward(dy, x, z, ids, A, B, scale, dbase) -> tuple:
    """(dx, dA, dB)."""
    dx = np.array(dbase, dtype=np.float64)
    dA, dB = np.zeros(A.shape), np.zeros(B.shape)
    for g in range(A.shape[0]):
        t = np.flatnonzero(ids == g)
        dyt = dy[t].astype(np.float64)
        dz = float(scale[g]) * (dyt @ B[g].astype(np.float64))
        dx[t] += dz @ A[g].astype(np.float64)
        dA[g] = dz.T @ x[t].astype(np.float64)
        dB[g] = float(scale[g]) * (dyt.T @ z[t].astype(np.float64))
    return dx, dA, dB
