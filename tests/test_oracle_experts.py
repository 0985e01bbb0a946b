"""The oracle of the gradients and of the MX rows against things other than itself: blocks worked by hand,
torch's E4M3 cast, the formats' own bounds, and difference quotients of the combine."""

import numpy as np
import pytest
import torch

import oracle
from workloads import f32_to_bf16_input, random_tiny_routing

E2M1, E4M3 = 1, 2


def bits(values):
    return f32_to_bf16_input(np.asarray(values, dtype=np.float32))


def block(values, form):
    row = np.zeros((1, 32), dtype=np.float32)
    row[0, : len(values)] = values
    codes, scales = oracle.mx_quantize(bits(row), form)
    return codes[0], int(scales[0, 0])


def test_e2m1_block_by_hand():
    # amax 7 = 1.75 * 2^2: exponent 2 - 2 = 0, byte 127; 7 saturates at 6 (code 7). Ties go to even codes:
    # 0.25 -> 0, 0.75 -> 1 (code 2), 1.25 -> 1 (code 2), 1.75 -> 2 (code 4), 2.5 -> 2, 3.5 -> 4 (code 6), 5 -> 4
    codes, byte = block([7, -0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -6, 0.375, -0.0], E2M1)
    assert byte == 127
    want = [7, 8, 2, 2, 4, 4, 6, 6, 15, 1, 8, 0]
    got = [int(c) for pair in codes[:6] for c in (pair & 15, pair >> 4)]
    assert got == want
    assert np.all(codes[6:] == 0)


def test_e4m3_block_by_hand():
    # amax 448 fits the scale 1 (byte 127); 450 (not above 448 * 2^1) takes 2 (byte 128)
    codes, byte = block([448.0, 1.0, -0.5], E4M3)
    assert byte == 127 and [int(c) for c in codes[:4]] == [0x7E, 0x38, 0xB0, 0]
    codes, byte = block([450.0, 2.0], E4M3)  # 225 lies nearer to 224 (0x76) than to 240
    assert byte == 128 and [int(c) for c in codes[:2]] == [0x76, 0x38]


@pytest.mark.parametrize("form", [E2M1, E4M3])
def test_zero_and_non_finite_blocks(form):
    row = np.zeros((1, 128), dtype=np.float32)
    row[0, 3] = -0.0
    row[0, 32:64] = np.nan
    row[0, 64:96] = 1.0
    row[0, 70] = -np.inf
    row[0, 96] = 1e-40  # a bf16 subnormal: the exponent stops at -127
    codes, scales = oracle.mx_quantize(bits(row), form)
    assert scales[0].tolist()[:3] == [0, 255, 255] and scales[0, 3] == 0
    v = oracle.mx_values(codes, scales, form)[0]
    assert np.all(v[:32] == 0) and np.signbit(v[3]) and not np.signbit(v[4])
    assert np.all(np.isnan(v[32:96])) and np.all(np.isfinite(v[96:]))


def test_e4m3_codes_match_torch_cast():
    rng = np.random.default_rng(5)
    x = bits(rng.standard_normal((64, 96)) * np.exp2(rng.integers(-30, 30, (64, 1))))
    codes, scales = oracle.mx_quantize(x, E4M3)
    v = torch.from_numpy(oracle.bf16_bits_to_f32(x)).view(64, 3, 32)
    q = torch.ldexp(v, -(torch.from_numpy(scales.astype(np.int32)) - 127).unsqueeze(-1))
    want = q.to(torch.float8_e4m3fn).view(torch.uint8).numpy().reshape(64, 96)
    assert np.array_equal(codes, want)


@pytest.mark.parametrize("form", [E2M1, E4M3])
def test_error_bounds(form):
    rng = np.random.default_rng(6)
    x = bits(rng.standard_normal((200, 64)) * np.exp2(rng.integers(-100, 100, (200, 1))))
    codes, scales = oracle.mx_quantize(x, form)
    v, ref = oracle.mx_values(codes, scales, form), oracle.bf16_bits_to_f32(x).astype(np.float64)
    scale = np.repeat(np.exp2(scales.astype(np.float64) - 127), 32, axis=1)
    if form == E4M3:  # half a step: 2^-4 relative, or half the smallest subnormal 2^-9
        assert np.all(np.abs(v - ref) <= np.maximum(np.abs(ref) * 2.0**-4, scale * 2.0**-10))
        assert np.all(np.abs(ref).reshape(200, 2, 32).max(axis=2) <= 448 * scale[:, ::32])
    else:  # at most 0.5 * scale below 4, then half of the step 2 up to 6, and the cut from just below 8 to 6
        assert np.all(np.abs(v - ref) <= np.where(np.abs(ref) < 4 * scale, 0.5 * scale, 2 * scale))


def test_product_against_loops():
    rng = np.random.default_rng(7)
    a = oracle.mx_values(*oracle.mx_quantize(bits(rng.standard_normal((5, 64))), E2M1), E2M1)
    w = np.stack([oracle.mx_values(*oracle.mx_quantize(bits(rng.standard_normal((4, 64))), E2M1), E2M1) for _ in range(3)])
    base = [0, 2, 2, 4]
    out = oracle.mx_product(a, w, base)
    for r, g in ((0, 0), (1, 0), (2, 2), (3, 2)):
        for o in range(4):
            assert out[r, o] == pytest.approx(sum(a[r, h] * w[g, o, h] for h in range(64)), rel=1e-12, abs=1e-12)
    assert np.all(np.isnan(out[4]))
    gated = oracle.mx_product(a, w, base, gated=True)
    assert gated[0, 1] == pytest.approx(out[0, 1] / (1 + np.exp(-out[0, 1])) * out[0, 3], rel=1e-12)


def combined(rows, slot, w):
    """The combine in float64."""
    y = np.zeros((slot.shape[0], rows.shape[1]))
    for t in range(slot.shape[0]):
        for k in range(slot.shape[1]):
            if slot[t, k] >= 0:
                y[t] += w[t, k] * rows[slot[t, k]]
    return y


def test_gradients_are_difference_quotients():
    """L = <dy, combine(rows, w)> is linear in each argument, so a step of one is exact up to rounding."""
    rng = np.random.default_rng(8)
    S, K, E, H = 5, 3, 6, 16
    idx = random_tiny_routing(rng, S, K, E, p_mask=0.2)
    slot = oracle.layout(idx, E, 2, 2)["slot_idx"]
    dy = bits(rng.standard_normal((S, H)))
    rows = oracle.bf16_bits_to_f32(bits(rng.standard_normal((S * K, H)))).astype(np.float64)
    w = rng.random((S, K)).astype(np.float32)
    g = oracle.bf16_bits_to_f32(dy).astype(np.float64)
    d_rows, d_w, _ = oracle.combine_backward(dy, rows, slot, w, np.zeros((S * K, H), np.uint16))
    d_rows = oracle.bf16_bits_to_f32(d_rows).astype(np.float64)
    loss = lambda r, ww: float((g * combined(r, slot, ww)).sum())  # noqa: E731
    h = 0.5
    for t in range(S):
        for k in range(K):
            up, down = w.astype(np.float64), w.astype(np.float64)
            up[t, k] += h
            down[t, k] -= h
            assert d_w[t, k] == pytest.approx((loss(rows, up) - loss(rows, down)) / (2 * h), abs=1e-9)
    for r in range(S * K):
        for c in (0, 7, H - 1):
            up, down = rows.copy(), rows.copy()
            up[r, c] += h
            down[r, c] -= h
            assert d_rows[r, c] == pytest.approx((loss(up, w) - loss(down, w)) / (2 * h), rel=2.0**-8, abs=1e-9)
    # the dispatch: L = <d, dispatch(x)>, dx the sum of the rows' gradients
    d = bits(rng.standard_normal((S * K, H)))
    dx = oracle.bf16_bits_to_f32(oracle.dispatch_backward(d, slot)).astype(np.float64)
    df = oracle.bf16_bits_to_f32(d).astype(np.float64)
    for t in range(S):
        want = sum((df[s] for s in slot[t] if s >= 0), np.zeros(H))
        assert np.all(np.abs(dx[t] - want) <= np.abs(want) * 2.0**-8 + 1e-6)
