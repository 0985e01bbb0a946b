"""Microscaled (MX) rows: blocks of 32 values with one E8M0 scale byte, E2M1 or E4M3 codes, and the experts'
product of such rows.

Test infrastructure only (see the package docstring).

The element and scale formats are those of the OCP Microscaling specification, version 1.0. Everything is
computed in float64, where bf16 values, their power-of-two multiples and the code tables are exact; a code is
found as the nearest table entry with a tie going to the even code, which is round to nearest even.

Readings taken: for E2M1 the scale exponent is floor(log2(amax)) - 2 (the specification's) and values past 6
become 6; for E4M3 it is the smallest e with amax <= 448 * 2^e, so that nothing saturates; e is held to
[-127, 127]; an all-zero block has byte 0 and zero codes with the values' signs; a block with a NaN or an
infinity has byte 255 and all its codes are zero.
"""

import numpy as np

from .formats import bf16_bits_to_f32, e4m3fn_decode

E2M1, E4M3 = 1, 2
BLOCK = 32

_E2M1_MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _magnitudes(form):
    if form == E2M1:
        return _E2M1_MAGNITUDES
    return np.asarray(e4m3fn_decode(np.arange(0x7F, dtype=np.uint8)), dtype=np.float64)  # 0x7F is NaN


def _nearest_code(a, form):
    """Index of the table entry nearest to each a >= 0, ties to the even index, past the end the last."""
    table = _magnitudes(form)
    middle = (table[1:] + table[:-1]) / 2  # exact in float64
    below = np.searchsorted(middle, a, side="left")  # entries whose upper middle lies below a
    tie = (below < len(middle)) & (middle[np.minimum(below, len(middle) - 1)] == a)
    return np.where(tie & (below % 2 == 1), below + 1, below)


def mx_quantize(rows_bits, form):
    """bf16 rows (uint16 [R, H], H % 32 == 0) -> (codes uint8 [R, H / 2 or H], scales uint8 [R, H / 32])."""
    rows_bits = np.asarray(rows_bits, dtype=np.uint16)
    R, H = rows_bits.shape
    x = bf16_bits_to_f32(rows_bits).astype(np.float64).reshape(R, H // BLOCK, BLOCK)
    bad = ~np.isfinite(x).all(axis=2)
    mag = np.where(bad[..., None], 0.0, np.abs(x))
    amax = mag.max(axis=2)
    _, power = np.frexp(amax)  # amax in [2^(power-1), 2^power)
    if form == E2M1:
        e = power - 1 - 2
    else:
        e = power - 1 - 8
        e = np.where(amax > 448.0 * np.exp2(e.astype(np.float64)), e + 1, e)
    e = np.clip(np.where(amax > 0, e, -127), -127, 127)
    code = _nearest_code(mag / np.exp2(e.astype(np.float64))[..., None], form).astype(np.uint8)
    sign_bit = 0x08 if form == E2M1 else 0x80
    code = np.where(bad[..., None], 0, code | (np.signbit(x) * sign_bit)).astype(np.uint8).reshape(R, H)
    scales = np.where(bad, 255, e + 127).astype(np.uint8)
    if form == E2M1:
        code = code[:, 0::2] | (code[:, 1::2] << 4)
    return np.ascontiguousarray(code), scales


def mx_values(codes, scales, form):
    """float64 values of MX rows [..., H] (NaN for blocks with byte 255)."""
    codes, scales = np.asarray(codes, dtype=np.uint8), np.asarray(scales, dtype=np.uint8)
    if form == E2M1:
        pair = np.stack([codes & 15, codes >> 4], axis=-1).reshape(*codes.shape[:-1], -1)
        v = np.where(pair & 8, -1.0, 1.0) * _E2M1_MAGNITUDES[pair & 7]
    else:
        v = np.asarray(e4m3fn_decode(codes), dtype=np.float64)
    scale = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    v = v.reshape(*scales.shape, BLOCK) * scale[..., None]
    return v.reshape(*scales.shape[:-1], -1)


def mx_product(a, w, group_base, gated=False):
    """float64 [R, O or O/2] of rows a [R, H] with weights w [G, O, H] (values, see mx_values); NaN rows of
    the result where no group has the row. gated: silu(first half) * second half."""
    a, w = np.asarray(a, dtype=np.float64), np.asarray(w, dtype=np.float64)
    G, O = w.shape[:2]
    out = np.full((a.shape[0], O), np.nan)
    for g in range(G):
        lo, hi = int(group_base[g]), int(group_base[g + 1])
        out[lo:hi] = a[lo:hi] @ w[g].T
    if not gated:
        return out
    gate, up = out[:, : O // 2], out[:, O // 2 :]
    with np.errstate(over="ignore"):
        return gate / (1.0 + np.exp(-gate)) * up
