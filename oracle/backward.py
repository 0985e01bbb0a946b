"""Gradients of the combine and of the dispatch.

Test infrastructure only (see the package docstring).

y[t] = sum_k w[t,k] * rows[slot[t,k]] is linear in the rows and in the weights, so with a gradient dy of y
d_rows[slot[t,k]] = w[t,k] * dy[t] and d_w[t,k] = <dy[t], rows[slot[t,k]]>; the dispatch rows[slot[t,k]] = x[t]
has dx[t] = sum_k d_rows[slot[t,k]]. Readings taken: the row gradient is one fp32 product rounded to bf16; the
dispatch gradient is an fp32 sum in ascending k from +0.0, rounded once; d_w is given in float64, for a
comparison with a tolerance. Entries with slot -1 take no part (d_w = 0).
"""

import numpy as np

from .formats import bf16_bits_to_f32, f32_to_bf16_bits


def combine_backward(dy_bits, rows, slot_idx, topk_weights, d_rows_bits):
    """(d_rows bits, d_w float64 [S, K], sum of the terms' magnitudes [S, K]). rows: float values [R, H];
    d_rows_bits uint16 [R, H] is what the rows held before (rows that no entry names keep it)."""
    dy = bf16_bits_to_f32(np.asarray(dy_bits, dtype=np.uint16))
    rows = np.asarray(rows)
    slot_idx = np.asarray(slot_idx)
    w = np.asarray(topk_weights, dtype=np.float32)
    out = np.array(d_rows_bits, dtype=np.uint16, copy=True)
    d_w, magnitude = np.zeros(slot_idx.shape), np.zeros(slot_idx.shape)
    for k in range(slot_idx.shape[1]):
        live = np.nonzero((slot_idx[:, k] >= 0) & (slot_idx[:, k] < rows.shape[0]))[0]
        s = slot_idx[live, k]
        out[s] = f32_to_bf16_bits(np.multiply(w[live, k, None], dy[live], dtype=np.float32))
        terms = dy[live].astype(np.float64) * rows[s].astype(np.float64)
        d_w[live, k] = terms.sum(axis=1)
        magnitude[live, k] = np.abs(terms).sum(axis=1)
    return out, d_w, magnitude


def dispatch_backward(d_rows_bits, slot_idx):
    """dx bits uint16 [S, H] from d_rows uint16 [R, H]."""
    rows = bf16_bits_to_f32(np.asarray(d_rows_bits, dtype=np.uint16))
    slot_idx = np.asarray(slot_idx)
    acc = np.zeros((slot_idx.shape[0], rows.shape[1]), dtype=np.float32)
    for k in range(slot_idx.shape[1]):
        live = np.nonzero((slot_idx[:, k] >= 0) & (slot_idx[:, k] < rows.shape[0]))[0]
        acc[live] = np.add(acc[live], rows[slot_idx[live, k]], dtype=np.float32)
    return f32_to_bf16_bits(acc)
