"""Plain definitions of the 8-bit layer around the dispatch: rows in 8 bits, the experts' INT8 product, the RMS norm
with the residual's addition and its gradients, and the router's balance loss and its gradient.

Test infrastructure only (see the package docstring). The experts' product is the grouped GEMM over the rows that
ShareToOutput lays out ("HCCL Window 模式 (Non-SHMEM) 代码深度剖析", section 3.9); the pages state neither a
norm nor a loss, so those are their formulas. Readings taken:

* rows in 8 bits: the dispatch's own arithmetic (``dispatch.py``) on rows of finite values; a row that holds a NaN or an
  infinity has scale NaN and zero codes;
* the norm takes the sum as it is held (bf16), its mean and root in 64 bits, rounds 1 / rms to fp32 once and then each of
  the two products; what it quantises is that fp32 value;
* gradients and the balance loss are returned in 64 bits, unrounded.
"""

import math

import numpy as np

from .dispatch import QUANT_FP8_E4M3_DYN
from .formats import bf16_bits_to_f32, e4m3fn_decode, e4m3fn_encode, f32_to_bf16_bits

SOFTMAX, SIGMOID = 0, 1


def row_quantize_f32(y, quant):
    """(codes uint8 [R, H], scales float32 [R]) of fp32 rows."""
    y = np.ascontiguousarray(y, dtype=np.float32)
    top = np.float32(448.0 if quant == QUANT_FP8_E4M3_DYN else 127.0)
    codes = np.zeros(y.shape, dtype=np.uint8)
    scales = np.zeros(y.shape[0], dtype=np.float32)
    for r, row in enumerate(y):
        if not np.all(np.isfinite(row)):
            scales[r] = np.nan
            continue
        scales[r] = np.float32(np.abs(row).max()) / top
        if scales[r] == 0:
            continue
        q = row / scales[r]
        codes[r] = e4m3fn_encode(q) if quant == QUANT_FP8_E4M3_DYN else np.clip(np.rint(q), -127, 127).astype(np.int8).view(np.uint8)
    return codes, scales


def row_quantize(x_bits, quant):
    return row_quantize_f32(bf16_bits_to_f32(x_bits), quant)


def row_values(codes, scales, quant):
    """The fp32 products code * scale, before they are rounded to bf16."""
    v = e4m3fn_decode(codes).astype(np.float32) if quant == QUANT_FP8_E4M3_DYN else codes.view(np.int8).astype(np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        return v * np.asarray(scales, dtype=np.float32)[:, None]


def int8_sums(a_codes, base, w_codes):
    """int64 [R, O] sums of each group's rows, and the group of every row (-1 outside all of them). A base below an
    earlier one counts as that one; all are held to [0, R]."""
    R, G, O = a_codes.shape[0], w_codes.shape[0], w_codes.shape[1]
    c, group = np.zeros((R, O), dtype=np.int64), np.full(R, -1)
    reached = 0
    for g in range(G):
        lo = max(min(max(int(base[g]), 0), R), reached)
        hi = max(min(max(int(base[g + 1]), 0), R), lo)
        reached = hi
        if hi > lo:
            # products below 2^14 and sums below 2^28 are exact in float64, where the matrix product is fast
            c[lo:hi] = (a_codes[lo:hi].astype(np.float64) @ w_codes[g].astype(np.float64).T).astype(np.int64)
            group[lo:hi] = g
    return c, group


def int8_product(a_codes, a_scales, base, w_codes, w_scales):
    """fp32 [R, O] values v, each step rounded (zero outside the groups), and the group of every row."""
    c, group = int8_sums(a_codes, base, w_codes)
    with np.errstate(over="ignore", invalid="ignore"):
        v = c.astype(np.float32) * np.asarray(a_scales, dtype=np.float32)[:, None]
        v = v * np.asarray(w_scales, dtype=np.float32)[np.maximum(group, 0)]
    v[group < 0] = 0
    return v, group


def rms_norm(x_bits, residual_bits, weight, eps):
    """(sum as bf16 bits, y float32): weight float32 [H]."""
    s = x_bits
    if residual_bits is not None:
        s = f32_to_bf16_bits(bf16_bits_to_f32(x_bits) + bf16_bits_to_f32(residual_bits))
    h = bf16_bits_to_f32(s)
    H = h.shape[1]
    with np.errstate(over="ignore", invalid="ignore"):
        r = np.array([1.0 / math.sqrt(math.fsum(float(v) * float(v) for v in row) / H + float(np.float32(eps)))
                      if np.all(np.isfinite(row)) else (np.nan if np.any(np.isnan(row)) else 0.0) for row in h]).astype(np.float32)
        return s, (h * r[:, None]) * np.asarray(weight, dtype=np.float32)


def rms_norm_backward(dy_bits, sum_bits, weight, eps, d_sum_bits=None):
    """(dx float64 [S, H], d_weight float64 [H])."""
    dy, h, w = (np.asarray(v, dtype=np.float64) for v in (bf16_bits_to_f32(dy_bits), bf16_bits_to_f32(sum_bits), weight))
    r = 1.0 / np.sqrt((h * h).mean(axis=1, keepdims=True) + float(np.float32(eps)))
    n, g = h * r, dy * w
    dx = r * (g - n * (g * n).mean(axis=1, keepdims=True))
    if d_sum_bits is not None:
        dx = dx + bf16_bits_to_f32(d_sum_bits).astype(np.float64)
    return dx, (dy * n).sum(axis=0)


def balance(logits, topk_idx, coef, score):
    """(loss, counts int64 [E], tokens, d_logits float64 [S, E] for d_loss = 1) of float logits."""
    l = np.asarray(logits, dtype=np.float64)
    S, E = l.shape
    valid = (topk_idx >= 0) & (topk_idx < E)
    counts = np.bincount(topk_idx[valid], minlength=E)
    s = np.zeros((S, E))
    turn = np.ones((S, E))
    tokens = 0
    for t in range(S):
        if not valid[t].any():
            continue
        tokens += 1
        top = l[t].max()
        if top == -np.inf:
            continue
        if score == SIGMOID:
            with np.errstate(over="ignore"):
                # sigmoid(l) = exp(min(l, 0)) / (1 + exp(-|l|)), taken against the largest logit
                e = np.exp(np.minimum(l[t], 0) - min(top, 0.0)) / (1 + np.exp(-np.abs(l[t])))
                turn[t] = np.where(l[t] > 0, np.exp(-np.abs(l[t])), 1.0) / (1 + np.exp(-np.abs(l[t])))
        else:
            e = np.exp(l[t] - top)
        s[t] = e / e.sum()
    if tokens == 0:
        return 0.0, counts, 0, np.zeros((S, E))
    each = float(np.float32(coef)) * E / (float(counts.sum()) * tokens)
    d = each * s * (counts - (s * counts).sum(axis=1, keepdims=True)) * turn
    return each * float((s * counts).sum()), counts, tokens, d
