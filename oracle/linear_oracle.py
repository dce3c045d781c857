"""Plain float64 oracle of the calls for experts of one's own (test
infrastructure only): row grouping, linear maps by group with their epilogue
and gradients, 8-bit checkpoints and the combine.

Written from the formulas in include/moe.h, one group or one token at a time;
it shares nothing with the HIP library.  Scales and codes of a checkpoint are
the one place where float32 decides a value: they are computed in float32,
operation by operation, as the definition says.
"""

from __future__ import annotations

import numpy as np
from scipy.special import erfc

from .moe_oracle import e4m3_decode

__all__ = ["group_rows", "activation", "activation_backward", "grouped_linear",
           "grouped_linear_backward", "checkpoint_pack", "checkpoint_unpack", "combine_rows",
           "combine_rows_backward", "BLOCK"]

BLOCK = 64


def group_rows(idx, n_experts: int, capacity: int = 0):
    """offsets [N + 1], row_token (one entry per row), slot_row [T, k]."""
    idx = np.asarray(idx)
    T, k = idx.shape
    kept = [[] for _ in range(n_experts)]
    for t in range(T):
        for s in range(k):
            e = int(idx[t, s])
            if 0 <= e < n_experts and (capacity == 0 or len(kept[e]) < capacity):
                kept[e].append((t, s))
    offsets = np.zeros(n_experts + 1, dtype=np.int32)
    slot_row = np.full((T, k), -1, dtype=np.int32)
    row_token = []
    for e in range(n_experts):
        for t, s in kept[e]:
            slot_row[t, s] = len(row_token)
            row_token.append(t)
        offsets[e + 1] = len(row_token)
    return offsets, np.array(row_token, dtype=np.int32), slot_row


def _sigmoid(z):
    out = np.empty_like(z)
    pos = z >= 0
    out[pos] = 1 / (1 + np.exp(-z[pos]))
    t = np.exp(z[~pos])
    out[~pos] = t / (1 + t)
    return out


def activation(act: str, z):
    if act == "none":
        return z.copy()
    if act == "relu":
        return np.where(z > 0, z, 0.0)
    if act == "gelu":
        return z * 0.5 * erfc(-z / np.sqrt(2))
    if act == "silu":
        return z * _sigmoid(z)
    assert act == "swiglu"
    a, b = np.split(z, 2, axis=1)
    return a * _sigmoid(a) * b


def activation_backward(act: str, z, dy):
    """dz from dy = dL/d act(z)."""
    if act == "none":
        return dy.copy()
    if act == "relu":
        return np.where(z > 0, dy, 0.0)
    if act == "gelu":
        return dy * (0.5 * erfc(-z / np.sqrt(2)) + z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi))
    if act == "silu":
        p = _sigmoid(z)
        return dy * (p + z * p * (1 - p))
    assert act == "swiglu"
    a, b = np.split(z, 2, axis=1)
    p = _sigmoid(a)
    return np.concatenate([dy * b * (p + a * p * (1 - p)), dy * a * p], axis=1)


def _groups(offsets):
    return [(e, int(offsets[e]), int(offsets[e + 1])) for e in range(len(offsets) - 1)
            if offsets[e + 1] > offsets[e]]


def _source(x, row_index, a, b):
    return x[row_index[a:b]] if row_index is not None else x[a:b]


def grouped_linear(x, offsets, w, act="none", row_index=None, bias=None, residual=None,
                   rows=None):
    """(y, z) of rows 0 .. offsets[-1]; rows past it are NaN."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    rows = int(offsets[-1]) if rows is None else rows
    zd = w.shape[1]
    z = np.full((rows, zd), np.nan)
    for e, a, b in _groups(offsets):
        z[a:b] = _source(x, row_index, a, b) @ w[e].T
        if bias is not None:
            z[a:b] += np.asarray(bias[e], np.float64)
    y = activation(act, z)
    if residual is not None:
        y = y + np.asarray(residual, np.float64)
    return y, z


def grouped_linear_backward(x, offsets, w, dy, z, act="none", row_index=None):
    """(dx, dw, dbias, dz) with the pre-activations z the activation is
    differentiated at (None for act "none")."""
    x, w, dy = (np.asarray(v, np.float64) for v in (x, w, dy))
    dz = np.full((dy.shape[0], w.shape[1]), np.nan)
    dx = np.full((dy.shape[0], w.shape[2]), np.nan)
    dw, db = np.zeros(w.shape), np.zeros(w.shape[:2])
    for e, a, b in _groups(offsets):
        dz[a:b] = activation_backward(act, None if z is None else z[a:b], dy[a:b])
        dx[a:b] = dz[a:b] @ w[e]
        dw[e] = dz[a:b].T @ _source(x, row_index, a, b)
        db[e] = dz[a:b].sum(0)
    return dx, dw, db, dz


_VALUES = e4m3_decode(np.arange(127, dtype=np.uint8))  # the non-negative ones, ascending


def _encode(v):
    """float32 values, |v| <= 448 -> nearest E4M3 codes, ties to the even code."""
    a = np.abs(v.astype(np.float64))
    hi = np.clip(np.searchsorted(_VALUES, a), 1, 126)
    lo = hi - 1
    dl, dh = a - _VALUES[lo], _VALUES[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code | np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)


def checkpoint_pack(x):
    """(codes uint8, scale float32) of x [rows, cols] (float32 values)."""
    x = np.asarray(x, np.float32)
    v = x.reshape(x.shape[0], x.shape[1] // BLOCK, BLOCK)
    fin = np.isfinite(v)
    m = np.maximum(np.max(np.where(fin, np.abs(v), 0), axis=2), np.float32(1e-30))
    inv = np.float32(448) / m
    s = np.where(fin, v, 0) * inv[:, :, None]
    codes = np.where(fin, _encode(np.clip(s, -448, 448)), 0x7F)
    return codes.reshape(x.shape).astype(np.uint8), (m / np.float32(448)).astype(np.float32)


def checkpoint_unpack(codes, scale):
    v = e4m3_decode(codes).reshape(codes.shape[0], codes.shape[1] // BLOCK, BLOCK)
    return (v * np.asarray(scale, np.float64)[:, :, None]).reshape(codes.shape)


def combine_rows(rows, slot_row, gate=None):
    rows = np.asarray(rows, np.float64)
    T, k = slot_row.shape
    y = np.zeros((T, rows.shape[1]))
    for t in range(T):
        for s in range(k):
            r = slot_row[t, s]
            if 0 <= r < rows.shape[0]:
                y[t] += rows[r] * (1.0 if gate is None else float(gate[t, s]))
    return y


def combine_rows_backward(rows, slot_row, gate, dy):
    rows, dy = np.asarray(rows, np.float64), np.asarray(dy, np.float64)
    T, k = slot_row.shape
    drows, dgate = np.full(rows.shape, np.nan), np.zeros((T, k))
    for t in range(T):
        for s in range(k):
            r = slot_row[t, s]
            if 0 <= r < rows.shape[0]:
                drows[r] = dy[t] * (1.0 if gate is None else float(gate[t, s]))
                dgate[t, s] = dy[t] @ rows[r]
    return drows, dgate
