"""GPU tests of the 8-bit layer's calls at their edges: the balance loss over several GPUs' tokens and at the ends of its
factors' ranges, more rows than one call of the library converts, products of many rows, gradients of the norm
whose mean cancels, and the links of a whole step.

Tolerances, derived before the first run, are written at each test; u = 2^-24 is fp32's rounding. The oracle is numpy in
64 bits.
"""

import numpy as np
import pytest
import torch

import oracle
from test_gpu_layer import (DEV, E4M3, GATED, INT8, PLAIN, Step, U, balance_case, bf16_bits, bf16_dev, bits, equal, int8_rows, moe, near, note,
                            poison, poisoned, routing, same_bits, same_rows8, to_dev, values)  # noqa: F401

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


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("coef,d_loss", [(3e38, 3.0), (1e-33, -1e-3), (1e20, 1e20)])
def test_gradient_of_small_scores_and_large_factors(moe, score, coef, d_loss):  # noqa: F811
    """The factor alone, times a count, is outside fp32's range, and the gradients of an expert that all but has the token and of
    the others, with scores of 1e-9, are not. Tolerance: (64 + far) u c s (|g| + sum s |g|), far 20, and 15 halves of the smallest
    subnormal, as above."""
    S, E, K = 5, 12, 2
    rng = np.random.default_rng(26)
    l = (rng.standard_normal((S, E)) - 20).astype(np.float32)
    l[:, 3] = 1
    idx = np.full((S, K), -1, dtype=np.int32)
    idx[2] = 3, 7
    unit = oracle.balance(l, idx, 1.0, score)[3]
    factor = float(np.float32(coef)) * float(np.float32(d_loss))
    u = l[2].astype(np.float64) if score == 0 else -np.logaddexp(0, -l[2].astype(np.float64))
    s = np.exp(u - u.max()) / np.exp(u - u.max()).sum()
    g = np.isin(np.arange(E), (3, 7))
    tol = np.zeros((S, E))
    tol[2] = 88 * U * abs(factor) * E / 2 * s * (g + (s * g).sum()) + 15 * 2.0**-150
    dev, table = to_dev(l), to_dev(idx)
    b = moe.moe_balance_loss(dev, table, coef, score)
    got = values(moe.moe_balance_loss_backward(torch.tensor([d_loss], device=DEV), dev, table, b.num_tokens_per_expert, b.num_tokens, coef, score))
    near(got, unit * factor, tol, "d_logits")


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("score", [0, 1])
def test_scores_far_below_the_largest(moe, score, kind):  # noqa: F811
    """Tokens whose largest logit lies anywhere from -200 to 40 and whose others lie up to 85 below it: each keeps its score and its
    gradient, to balance_case's bounds."""
    rng = np.random.default_rng(25)
    S, E = 150, 40
    l = (np.linspace(-200, 40, S)[:, None] - rng.uniform(0, 85, (S, E))).astype(np.float32)
    balance_case(moe, l, routing(rng, S, E, 4, ""), score, kind, coef=1.0)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("S,E", [(64, 512), (65, 512), (128, 257), (128, 256), (129, 256)])
def test_around_the_most_tokens_of_one_workgroup(moe, S, E, score):  # noqa: F811
    rng = np.random.default_rng(S + E)
    balance_case(moe, rng.standard_normal((S, E)).astype(np.float32), routing(rng, S, E, 6, "padded"), score, "fp32")


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


# ---------------------------------------------------------------- the norm's gradient


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("S,H", [(40, 64), (40, 528), (20, 1040)])
def test_norm_gradient_where_the_mean_cancels(moe, S, H, kind):  # noqa: F811
    """Rows whose mean of g * n all but cancels, by the last weight, so that it is what the products' roundings would make of it; where
    dy is 0 the gradient is that mean alone. The reference is in 80 bits. Tolerance: as for other rows, 2^-21 of the terms and
    half a step; the mean's own sum, of H products in 64 bits, is off by (H + 8) 2^-53 of their magnitudes."""
    rng = np.random.default_rng(H)
    h, dy = (oracle.bf16_bits_to_f32(bits(rng.standard_normal((S, H)))).astype(np.longdouble) for _ in range(2))
    w = (1 + 0.3 * rng.standard_normal(H)).astype(np.float32)
    if kind == "bf16":
        w = oracle.bf16_bits_to_f32(bits(w))
    dy[:, ::5] = 0
    h[:, -1] = dy[:, -1] = 1
    h[1:], dy[1:] = h[0], dy[0]  # one weight for all rows: they differ in sign and in powers of two
    h *= np.exp2(rng.integers(-9, 9, (S, 1)))
    dy *= np.exp2(rng.integers(-9, 9, (S, 1))) * rng.choice([-1, 1], (S, 1))
    near_zero = -(h[0, :-1] * dy[0, :-1] * w[:-1].astype(np.longdouble)).sum() / (h[0, -1] * dy[0, -1])
    w[-1] = oracle.bf16_bits_to_f32(bits([near_zero]))[0] if kind == "bf16" else np.float32(near_zero)
    g = dy * w.astype(np.longdouble)
    r = 1 / np.sqrt((h * h).mean(axis=1, keepdims=True) + float(np.float32(1e-5)))
    n = h * r
    m = (g * n).mean(axis=1, keepdims=True)
    want = r * (g - n * m)
    off = (H + 8) * 2.0**-53 * np.abs(g * n).mean(axis=1, keepdims=True)
    tol = 2.0**-21 * (np.abs(r * g) + np.abs(r * n * m)) + np.abs(r * n) * off + 2.0**-8 * np.abs(want) + 2.0**-133
    weight = bf16_dev(bits(w)) if kind == "bf16" else to_dev(w)
    as_rows = lambda v: bf16_dev(bits(v.astype(np.float64)))  # noqa: E731
    assert np.array_equal(values(as_rows(h)), h.astype(np.float32)) and np.array_equal(values(as_rows(dy)), dy.astype(np.float32))
    dx, _ = moe.moe_rms_norm_backward(as_rows(dy), as_rows(h), weight, 1e-5)
    near(values(dx), want.astype(np.float64), tol.astype(np.float64), "dx")


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


# ---------------------------------------------------------------- together


def silu_bound(v):
    """Gate times up of the product's values v [R, 2 I], and its bound: silu to 2^-14, then half a step of bf16."""
    half = v.shape[1] // 2
    gate, up = v[:, :half].astype(np.float64), v[:, half:].astype(np.float64)
    want = gate / (1 + np.exp(-gate)) * up
    return want, (2.0**-8 + 2.0**-13) * np.abs(want) + 2.0**-133


def host8(rows8):
    return rows8[0].cpu().numpy().view(np.int8), rows8[1].cpu().numpy()


def test_every_link_of_a_step(moe):  # noqa: F811
    """A layer's forward and backward pass, each call's result against the oracle's of what that call was given on the GPU: bit for
    bit but for the activation (silu_bound), the balance loss (as in balance_case), the weights' gradient of the combine (128
    additions' roundings) and the norm's gradients (2^-21 of their terms and half a step; (S / 256 + 85) u for d_weight)."""
    step = Step(moe, 7)
    S, H, E, K = step.S, step.H, step.E, step.K
    coef = 0.01
    normed = moe.moe_rms_norm(step.x, step.norm_weight, residual=step.residual, quant=INT8, out=torch.empty_like(step.x))
    logits = normed.out.float() @ step.router
    lay = moe.moe_layout(step.topk_idx, E, 1, 1)
    loss = moe.moe_balance_loss(logits, step.topk_idx, coef)
    moe.moe_dispatch(normed.out, lay.slot_idx, step.window, INT8)
    rows = lay.expert_slot_base[E:]
    un = moe.moe_unpack(step.window, rows, S, K, H, INT8)
    mid = moe.moe_scaled_product(moe.ScaledRows(un.expand_x, un.expand_scales), step.up, lay.expert_slot_base, GATED)
    mid8 = moe.moe_row_quantize(mid, INT8, num_rows=rows)
    expert_out = moe.moe_scaled_product(mid8, step.down, lay.expert_slot_base)
    y = moe.moe_combine(expert_out, lay.slot_idx, step.topk_weights)
    shared_mid = moe.moe_scaled_product(normed.rows8, step.shared_up, step.all_rows, GATED)
    shared_mid8 = moe.moe_row_quantize(shared_mid, INT8)
    shared = moe.moe_scaled_product(shared_mid8, step.shared_down, step.all_rows)
    d_rows, d_weights = moe.moe_combine_backward(step.dy, expert_out, lay.slot_idx, step.topk_weights)
    d_out = moe.moe_dispatch_backward(d_rows, lay.slot_idx)
    d_logits = moe.moe_balance_loss_backward(torch.ones(1, device=DEV), logits, step.topk_idx, loss.num_tokens_per_expert, loss.num_tokens, coef)
    dx, d_norm = moe.moe_rms_norm_backward(d_out, normed.sum, step.norm_weight, d_sum=step.dy)

    idx, weights, slots = step.topk_idx.cpu().numpy(), step.topk_weights.cpu().numpy(), lay.slot_idx.cpu().numpy()
    w = step.norm_weight.cpu().numpy()
    total, yn = oracle.rms_norm(bf16_bits(step.x), bf16_bits(step.residual), w, 1e-6)
    same_bits(bf16_bits(normed.sum), total, "sum")
    same_bits(bf16_bits(normed.out), bits(yn), "normed")
    same_rows8(normed.rows8, *oracle.row_quantize_f32(yn, INT8), "normed in 8 bits")
    want = oracle.layout(idx, E, 1, 1)
    assert np.array_equal(slots, want["slot_idx"])
    base, used = want["expert_slot_base"], int(want["expert_slot_base"][E])
    token = np.empty(used, dtype=np.int64)
    token[slots.ravel()] = np.arange(slots.size) // K
    codes, scales = oracle.row_quantize(bf16_bits(normed.out), INT8)
    same_rows8(moe.ScaledRows(un.expand_x[:used], un.expand_scales[:used]), codes[token], scales[token], "unpacked")
    for first, at, up, second, down, out, edges in ((moe.ScaledRows(un.expand_x, un.expand_scales), mid, step.up, mid8, step.down, expert_out, base),
                                                    (normed.rows8, shared_mid, step.shared_up, shared_mid8, step.shared_down, shared, [0, S])):
        near(values(at), *silu_bound(oracle.int8_product(*host8(first), edges, *host8(up))[0]), "activation")
        same_rows8(second, *oracle.row_quantize(bf16_bits(at), INT8), "activation in 8 bits")
        same_bits(bf16_bits(out), bits(oracle.int8_product(*host8(second), edges, *host8(down))[0]), "second product")
    same_bits(bf16_bits(y), oracle.combine(bf16_bits(expert_out), slots, weights), "y")

    want_rows, want_w, magnitude = oracle.combine_backward(bf16_bits(step.dy), values(expert_out), slots, weights, bf16_bits(d_rows))
    same_bits(bf16_bits(d_rows), want_rows, "d_rows")
    near(values(d_weights), want_w, 128 * U * magnitude + 1e-37, "d_weights")
    same_bits(bf16_bits(d_out), oracle.dispatch_backward(want_rows, slots), "d_out")
    l = values(logits)
    want, counts, tokens, want_d = oracle.balance(l, idx, coef, 0)
    near(values(loss.loss), [want], 412 * U * want, "loss")
    assert np.array_equal(loss.num_tokens_per_expert.cpu().numpy(), counts) and int(loss.num_tokens) == tokens == S
    far = l.max(axis=1, keepdims=True).astype(np.float64) - l
    s = np.exp(-far) / np.exp(-far).sum(axis=1, keepdims=True)
    g = np.abs(counts - counts.sum() // E)
    near(values(d_logits), want_d, coef * E / (counts.sum() * tokens) * U * (64 + far) * s * (g + (s * g).sum(axis=1, keepdims=True)), "d_logits")
    want_dx, want_dw = oracle.rms_norm_backward(bf16_bits(d_out), total, w, 1e-6, bf16_bits(step.dy))
    h, do = oracle.bf16_bits_to_f32(total).astype(np.float64), values(d_out).astype(np.float64)
    r = 1 / np.sqrt((h * h).mean(axis=1, keepdims=True) + 1e-6)
    terms = np.abs(r * do * w) + np.abs(h * r * r * (do * w * h * r).mean(axis=1, keepdims=True)) + np.abs(values(step.dy))
    near(values(dx), want_dx, 2.0**-21 * terms + 2.0**-8 * np.abs(want_dx) + 2.0**-133, "dx")
    near(values(d_norm), want_dw, (S / 256 + 85) * U * np.abs(do * h * r).sum(axis=0), "d_norm")


def test_steps_on_streams_that_wait_for_their_inputs(moe):  # noqa: F811
    """Steps on streams of their own, each behind the one that made its inputs: eagerly, then both at once as graphs."""
    steps = [Step(moe, 8), Step(moe, 9)]
    want = [s() for s in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    graphs = []
    for s, stream, w in zip(steps, streams, want):
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            got = s()
        torch.cuda.synchronize()
        assert equal(got, w)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            outs = s()
        graphs.append((g, outs))
    for _ in range(3):
        for s in steps:
            s.x.copy_(torch.randn(s.S, s.H, device=DEV).to(torch.bfloat16))
        want = [s() for s in steps]
        torch.cuda.synchronize()
        for (g, _), stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                g.replay()
        torch.cuda.synchronize()
        assert all(equal(outs, w) for (_, outs), w in zip(graphs, want))


def test_calls_that_are_given_their_stream(moe):  # noqa: F811
    """Each call on a stream that waits for its inputs, which outlive it; results as on the current stream."""
    step = Step(moe, 10)
    logits = torch.randn((step.S, step.E), device=DEV)
    one = torch.ones(1, device=DEV)

    def calls(stream):
        n = moe.moe_rms_norm(step.x, step.norm_weight, residual=step.residual, quant=INT8, stream=stream)
        v = moe.moe_row_dequantize(n.rows8, INT8, stream=stream)
        q = moe.moe_row_quantize(v, E4M3, stream=stream)
        mid = moe.moe_scaled_product(n.rows8, step.shared_up, step.all_rows, GATED, stream=stream)
        dx, dw = moe.moe_rms_norm_backward(step.dy, n.sum, step.norm_weight, d_sum=v, stream=stream)
        b = moe.moe_balance_loss(logits, step.topk_idx, 1.0, stream=stream)
        d = moe.moe_balance_loss_backward(one, logits, step.topk_idx, b.num_tokens_per_expert, b.num_tokens, 1.0, stream=stream)
        return [n.sum, n.rows8.codes, n.rows8.scales, v, q.codes, q.scales, mid, dx, dw, *b, d]

    want = calls(None)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    for given in (stream, stream.cuda_stream):
        got = calls(given)
        torch.cuda.synchronize()
        assert equal(got, want)
