"""The oracle of the rows in 8 bits, the INT8 product, the RMS norm and the balance loss against things other than
itself: values worked by hand, the dispatch's own quantiser, torch's integer products, and difference quotients in
64 bits (central, step 2^-10: off by the third derivative times 2^-20 / 6 and by 2^-53 * 2^10 of the values)."""

import math

import numpy as np
import pytest
import torch

import oracle
from workloads import f32_to_bf16_input

E4M3, INT8 = 1, 2


def bits(values):
    return f32_to_bf16_input(np.asarray(values, dtype=np.float32))


def test_rows_by_hand():
    # amax 254: scale 2; 3 / 2 = 1.5 -> 2 (even), 5 / 2 = 2.5 -> 2, -1 / 2 = -0.5 -> 0
    codes, scales = oracle.row_quantize(bits([[254, 3, 5, -1, -254, 0]]), INT8)
    assert scales[0] == 2 and codes.view(np.int8)[0].tolist() == [127, 2, 2, 0, -127, 0]
    # amax 448: scale 1; 17 lies between 16 and 18 -> 16 (even mantissa)
    codes, scales = oracle.row_quantize(bits([[448, 17, -0.5, 0]]), E4M3)
    assert scales[0] == 1 and codes[0].tolist() == [0x7E, 0x58, 0xB0, 0]
    assert oracle.row_values(codes, scales, E4M3)[0].tolist() == [448, 16, -0.5, 0]


@pytest.mark.parametrize("quant", [E4M3, INT8])
def test_rows_are_the_dispatchs(quant):
    rng = np.random.default_rng(1)
    x = bits(rng.standard_normal((40, 256)) * np.exp2(rng.integers(-100, 100, (40, 1))))
    x[7] = 0
    want = (oracle.quantize_e4m3_dynamic if quant == E4M3 else oracle.quantize_int8_dynamic)(x)
    codes, scales = oracle.row_quantize(x, quant)
    assert np.array_equal(codes, want[0].view(np.uint8)) and np.array_equal(scales, want[1])


def test_rows_not_finite():
    x = bits([[1, 2, np.nan, 4], [1, -np.inf, 3, 4], [1, 2, 3, 4]])
    codes, scales = oracle.row_quantize(x, INT8)
    assert np.isnan(scales[:2]).all() and np.isfinite(scales[2]) and not codes[:2].any()
    assert np.isnan(oracle.row_values(codes, scales, INT8)[:2]).all()


def test_int8_sums_are_torchs():
    rng = np.random.default_rng(2)
    a, w = rng.integers(-128, 128, (9, 48)).astype(np.int8), rng.integers(-128, 128, (3, 7, 48)).astype(np.int8)
    c, group = oracle.int8_sums(a, [2, 4, 4, 8], w)
    assert group.tolist() == [-1, -1, 0, 0, 2, 2, 2, 2, -1]
    for r in range(9):
        want = torch.zeros(7, dtype=torch.int64)
        if group[r] >= 0:
            want = (torch.from_numpy(w[group[r]]).long() * torch.from_numpy(a[r]).long()).sum(dim=1)
        assert c[r].tolist() == want.tolist()
    # a base below an earlier one counts as that one, and all are held to the rows
    assert oracle.int8_sums(a, [5, 3, 6, 99], w)[1].tolist() == [-1] * 5 + [1] + [2] * 3
    v, _ = oracle.int8_product(a, np.full(9, 0.5), [0, 9, 9, 9], w, np.full((3, 7), 0.25))
    assert np.array_equal(v, oracle.int8_sums(a, [0, 9, 9, 9], w)[0].astype(np.float32) / 8)


def test_norm_by_hand():
    # 3 and 4 from 1 + 2 and 1 + 3: mean square 12.5, eps 3.5: 1 / rms = 1 / 4
    s, y = oracle.rms_norm(bits([[1, 1]]), bits([[2, 3]]), np.array([1, 2], dtype=np.float32), 3.5)
    assert oracle.bf16_bits_to_f32(s)[0].tolist() == [3, 4] and y[0].tolist() == [0.75, 2.0]
    s, y = oracle.rms_norm(bits([[0, 0, 0, 0]]), None, np.ones(4, dtype=np.float32), 1e-6)
    assert not y.any()
    # values whose squares leave fp32's range, of either end
    for v in (1e30, 1e-30):
        y = oracle.rms_norm(bits([[v, -v]]), None, np.ones(2, dtype=np.float32), 1e-45)[1]
        if v > 1:
            assert y[0].tolist() == [1, -1]
        else:
            assert abs(y[0, 0] - float(oracle.bf16_bits_to_f32(bits([v]))[0]) / math.sqrt(1e-45)) < 1e-7


def test_norm_gradient_is_the_difference():
    rng = np.random.default_rng(3)
    S, H, eps = 3, 32, 0.01
    s, dy, d_sum = (oracle.bf16_bits_to_f32(bits(rng.standard_normal((S, H)))).astype(np.float64) for _ in range(3))
    w = rng.standard_normal(H).astype(np.float32).astype(np.float64)

    def f(h, w):
        return float((h / np.sqrt((h * h).mean(axis=1, keepdims=True) + float(np.float32(eps))) * w * dy).sum() + (h * d_sum).sum())

    dx, dw = oracle.rms_norm_backward(bits(dy), bits(s), w, eps, bits(d_sum))
    for _ in range(5):
        v, u = rng.standard_normal((S, H)), rng.standard_normal(H)
        step = 2.0**-10
        quotient = (f(s + step * v, w + step * u) - f(s - step * v, w - step * u)) / (2 * step)
        assert abs(quotient - (dx * v).sum() - (dw * u).sum()) < 1e-3 * (np.abs(dx * v).sum() + np.abs(dw * u).sum())


@pytest.mark.parametrize("score", [0, 1])
def test_balance_gradient_is_the_difference(score):
    rng = np.random.default_rng(4 + score)
    S, E, K = 12, 9, 3
    l = rng.standard_normal((S, E)) * 2
    l[2, 1:] = -np.inf
    l[5] = -np.inf
    l[7] = np.nan
    idx = rng.integers(-1, E + 2, (S, K)).astype(np.int32)
    idx[0], idx[1], idx[7] = (4, 4, 4), (0, -1, 3), (-1, E, -5)
    loss, counts, tokens, d = oracle.balance(l, idx, 0.01, score)
    assert tokens == sum(bool(((r >= 0) & (r < E)).any()) for r in idx) and counts.sum() == ((idx >= 0) & (idx < E)).sum()
    assert not d[7].any() and not d[5].any() and not d[2, 1:].any() and loss > 0
    free = np.isfinite(l)
    for _ in range(5):
        v = np.where(free, rng.standard_normal((S, E)), 0)
        step = 2.0**-10
        quotient = (oracle.balance(l + step * v, idx, 0.01, score)[0] - oracle.balance(l - step * v, idx, 0.01, score)[0]) / (2 * step)
        assert abs(quotient - (d * v).sum()) < 1e-4 * np.abs(d * v).sum()


def test_balance_by_hand():
    # two tokens, both to expert 0 of 2, equal logits: s = 1/2, n = (2, 0), N = T = 2: loss = c * 2 / 4 * 2 * 1
    idx = np.array([[0], [0]], dtype=np.int32)
    loss, counts, tokens, d = oracle.balance(np.zeros((2, 2)), idx, 1.0, 0)
    assert loss == 1.0 and counts.tolist() == [2, 0] and tokens == 2
    assert np.allclose(d, [[0.25, -0.25]] * 2)  # 1/2 * s * (n - 1)
    assert oracle.balance(np.zeros((2, 2)), -np.ones((2, 1), dtype=np.int32), 1.0, 0)[0] == 0.0
    # logits far below zero keep their scores
    assert abs(oracle.balance(np.array([[-500.0, -501.0]]), idx[:1], 1.0, 1)[0] - 2 * math.e / (math.e + 1)) < 1e-12
