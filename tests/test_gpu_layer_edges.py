"""GPU tests of the 8-bit layer's calls at their edges: the balance loss over several GPUs' tokens and at the ends of its
factors' ranges, more rows than one call of the library converts, and products of many rows.

Tolerances, derived before the first run, are written at each test; u = 2^-24 is fp32's rounding. The oracle is numpy in
64 bits.
"""

import numpy as np
import pytest
import torch

import oracle
from test_gpu_layer import (DEV, E4M3, GATED, INT8, PLAIN, U, balance_case, bf16_bits, bf16_dev, bits, int8_rows, moe, near, note, poison,
                            poisoned, routing, same_bits, same_rows8, to_dev, values)  # noqa: F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- the balance loss


@pytest.mark.parametrize("score", [0, 1])
def test_gradient_of_the_loss_over_several_gpus(moe, score):  # noqa: F811
    """A batch in three uneven parts, of which one is half padding, as three GPUs have them: with the sums of their counts and of
    their numbers of tokens each part gets its rows of the whole batch's gradient. Tolerance: d_logits = c s (g - dot), (64 + far)
    u c s (|g| + sum s |g|), with far below 20 for normal values and the bracket at most twice the largest |g|."""
    rng = np.random.default_rng(20 + score)
    S, E, K, coef = 700, 48, 4, 0.3
    l = rng.standard_normal((S, E)).astype(np.float32)
    idx = routing(rng, S, E, K, "")
    idx[rng.random((S, K)) < 0.1] = -1
    idx[100:160] = -1
    counts, tokens, want = oracle.balance(l, idx, coef, score)[1:]
    parts = [slice(0, 20), slice(20, 160), slice(160, S)]
    logits, tables = [to_dev(l[p]) for p in parts], [to_dev(idx[p]) for p in parts]
    own = [moe.moe_balance_loss(a, t, coef, score) for a, t in zip(logits, tables)]
    all_counts = sum(b.num_tokens_per_expert for b in own)
    all_tokens = sum(b.num_tokens for b in own)
    assert np.array_equal(all_counts.cpu().numpy(), counts) and int(all_tokens) == tokens
    one = torch.ones(1, device=DEV)
    got = [values(moe.moe_balance_loss_backward(one, a, t, all_counts, all_tokens, coef, score)) for a, t in zip(logits, tables)]
    largest = np.abs(counts - counts.sum() // E).max()
    near(np.concatenate(got), want, 84 * U * coef * E / (counts.sum() * tokens) * 2 * largest, "d_logits")


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_gradient_of_counts_that_pass_32_bits_together(moe, kind):  # noqa: F811
    """Counts of many GPUs, each in int32, 2^33 in all. Tolerance: (64 + far) u c s (|g| + sum s |g|), with far below 20 for normal
    values and |g| at most the largest count, and half a step of bf16."""
    rng = np.random.default_rng(22)
    S, E = 9, 6
    l = rng.standard_normal((S, E)).astype(np.float32)
    dev = to_dev(l).to(kind)
    l = dev.float().cpu().numpy().astype(np.float64)
    counts = np.array([2**31 - 1, 2**31 - 1, 2**31 - 5, 2**31 - 1, 17, 0], dtype=np.int32)
    tokens = 2**31 - 1
    idx = to_dev(rng.integers(0, E, (S, 2)).astype(np.int32))
    got = moe.moe_balance_loss_backward(torch.ones(1, device=DEV), dev, idx, to_dev(counts), to_dev(np.array([tokens], dtype=np.int32)), 1.0)
    n = counts.astype(np.float64)
    s = np.exp(l - l.max(axis=1, keepdims=True))
    s /= s.sum(axis=1, keepdims=True)
    each = E / (n.sum() * tokens)
    want = each * s * (n - (s * n).sum(axis=1, keepdims=True))
    tol = 84 * U * each * s * 2 * n.max() + (2.0**-8 * np.abs(want) if kind is torch.bfloat16 else 0)
    near(got.float().cpu().numpy(), want, tol, "d_logits")


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("coef,d_loss", [(3e38, 1e-36), (1e-36, 1e30), (1e-44, 3e38), (1.0, 1e-37)])
def test_gradient_of_factors_at_both_ends_of_the_range(moe, score, coef, d_loss):  # noqa: F811
    """coef * E / (N T) may leave fp32's range where the gradient does not. Tolerance: (64 + far) u c s (|g| + sum s |g|) with
    c = d_loss coef E / (N T), far below 20 for normal values, and half of the smallest subnormal for each rounding: the factor of
    a count, the 12 products of the row's sum, and two more products."""
    rng = np.random.default_rng(23)
    S, E, K = 5, 12, 2
    l = rng.standard_normal((S, E)).astype(np.float32)
    idx = np.full((S, K), -1, dtype=np.int32)
    idx[2] = 3, 7
    counts, tokens, unit = oracle.balance(l, idx, 1.0, score)[1:]
    factor = float(np.float32(coef)) * float(np.float32(d_loss))
    want = unit * factor
    dev, table = to_dev(l), to_dev(idx)
    b = moe.moe_balance_loss(dev, table, coef, score)
    got = moe.moe_balance_loss_backward(torch.tensor([d_loss], device=DEV), dev, table, b.num_tokens_per_expert, b.num_tokens, coef, score)
    largest = np.abs(counts - counts.sum() // E).max()
    note("factors", coef, d_loss, np.abs(want).max())
    near(values(got), want, 84 * U * factor * E / (counts.sum() * tokens) * 2 * largest + 15 * 2.0**-150, "d_logits")


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("score", [0, 1])
def test_scores_far_below_the_largest(moe, score, kind):  # noqa: F811
    """Tokens whose largest logit lies anywhere from -200 to 40 and whose others lie up to 85 below it: each keeps its score and its
    gradient, to balance_case's bounds."""
    rng = np.random.default_rng(25)
    S, E = 150, 40
    l = (np.linspace(-200, 40, S)[:, None] - rng.uniform(0, 85, (S, E))).astype(np.float32)
    balance_case(moe, l, routing(rng, S, E, 4, ""), score, kind, coef=1.0)


# ---------------------------------------------------------------- rows in 8 bits


MOST = 1 << 20  # rows that one call of the library converts


@pytest.mark.parametrize("quant", [E4M3, INT8])
@pytest.mark.parametrize("given", [False, True])
def test_more_rows_than_one_call_converts(moe, quant, given):  # noqa: F811
    """2^20 + 300 rows at a stride, as all experts' weights may be, with counts on both sides of the parts' border; on the
    current stream and on one that the call is given. Bit for bit."""
    rng = np.random.default_rng(24 + quant)
    R, H = MOST + 300, 32
    x = bits(rng.standard_normal((R, H)))
    wide = poison((R, H + 8), torch.bfloat16)
    wide[:, :H] = bf16_dev(x)
    at = np.concatenate((np.arange(40), np.arange(MOST - 40, R)))
    codes, scales = oracle.row_quantize(x[at], quant)
    back = bits(oracle.row_values(codes, scales, quant))
    index = to_dev(at)
    stream = torch.cuda.Stream() if given else None
    for n in (None, -3, 5, MOST, MOST + 1, R - 1, R + 9):
        used = R if n is None else min(max(n, 0), R)
        count = None if n is None else torch.tensor([n], dtype=torch.int32, device=DEV)
        out = moe.ScaledRows(poison((R, H), torch.uint8), poison(R, torch.float32))
        values_out = poison((R, H + 8), torch.bfloat16)
        torch.cuda.synchronize()  # the buffers are whole before another stream uses them
        note("rows in parts", quant, given, n)
        moe.moe_row_quantize(wide[:, :H], quant, num_rows=count, out=out, stream=stream)
        moe.moe_row_dequantize(out, quant, num_rows=count, out=values_out[:, :H], stream=stream)
        torch.cuda.synchronize()
        some = at < used
        same_rows8(moe.ScaledRows(out.codes[index][: some.sum()], out.scales[index][: some.sum()]), codes[some], scales[some])
        same_bits(bf16_bits(values_out[:, :H][index])[some], back[some])
        assert poisoned(out.codes[used:]) and poisoned(out.scales[used:]) and poisoned(values_out[used:]) and poisoned(values_out[:, H:])


def test_parts_of_rows_refuse_what_one_call_refuses(moe):  # noqa: F811
    """Outputs over inputs and over one another, where only parts that do not run together touch."""
    R, H = MOST + 300, 32
    buf = torch.zeros(2 * R * H + 64, dtype=torch.uint8, device=DEV)
    rows = buf[: 2 * R * H].view(torch.bfloat16).view(R, H)
    scales = torch.zeros(R, device=DEV)
    last = buf[2 * R * H - R * H : 2 * R * H].view(R, H)  # over the later rows
    with pytest.raises(ValueError, match="overlap"):
        moe.moe_row_quantize(rows, INT8, out=(last, scales))
    with pytest.raises(ValueError, match="overlap"):
        moe.moe_row_dequantize((last, scales), INT8, out=rows)
    codes = torch.zeros((R, H), dtype=torch.uint8, device=DEV)
    over = codes.view(-1)[-4 * R :].view(torch.float32)  # scales over the later codes
    with pytest.raises(ValueError, match="overlap"):
        moe.moe_row_quantize(rows, INT8, out=(codes, over))
    with pytest.raises(ValueError):
        moe.moe_row_quantize(rows, 0, out=(codes, scales))


# ---------------------------------------------------------------- the product


@pytest.mark.parametrize("R,G,H,O,epilogue", [(65536, 8, 256, 128, GATED), (50000, 1, 272, 100, PLAIN), (65536, 8, 256, 384, PLAIN),
                                              (50000, 3, 1552, 260, PLAIN), (70000, 2, 144, 640, GATED), (1 << 20, 1, 64, 64, PLAIN)])
def test_products_of_many_rows_and_few_outputs(moe, R, G, H, O, epilogue):  # noqa: F811
    """Rows around the groups' borders and at the ends, bit for bit; gated ones to silu's 2^-14 and half a step of bf16."""
    rng = np.random.default_rng(R + O)
    base = np.concatenate(([0], np.sort(rng.integers(0, R + 1, G - 1)), [R])).astype(np.int32)
    a, scales = int8_rows(rng, R, H)
    w = rng.integers(-128, 128, (G, O, H)).astype(np.int8)
    w_scales = (np.exp2(rng.uniform(-5, 0, (G, O))) / (np.sqrt(H) * 4)).astype(np.float32)
    note("many rows", R, G, H, O, epilogue)
    got = moe.moe_scaled_product(moe.ScaledRows(to_dev(a), to_dev(scales)), moe.ScaledRows(to_dev(w), to_dev(w_scales)), to_dev(base), epilogue)
    at = np.unique(np.clip(np.concatenate([np.arange(b - 300, b + 300) for b in base]), 0, R - 1))
    v, group = oracle.int8_product(a[at], scales[at], np.searchsorted(at, base), w, w_scales)
    assert (group == np.searchsorted(base, at, side="right") - 1).all()
    some = got[to_dev(at)]
    if epilogue == PLAIN:
        same_bits(bf16_bits(some), bits(v))
    else:
        gate, up = v[:, : O // 2].astype(np.float64), v[:, O // 2 :].astype(np.float64)
        want = gate / (1 + np.exp(-gate)) * up
        near(values(some), want, (2.0**-8 + 2.0**-13) * np.abs(want) + 2.0**-133, "gated")
