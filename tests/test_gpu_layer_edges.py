"""GPU tests of the 8-bit layer's calls at their edges: the balance loss over several GPUs' tokens and at the ends of its
factors' ranges.

Tolerances, derived before the first run, are written at each test; u = 2^-24 is fp32's rounding. The oracle is numpy in
64 bits.
"""

import numpy as np
import pytest
import torch

import oracle
from test_gpu_layer import DEV, U, moe, near, note, routing, to_dev, values  # noqa: F401

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
