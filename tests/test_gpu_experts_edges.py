"""GPU tests of the calls around the experts at their edges: values at the ends of the formats' ranges, gates far
below zero, bases that descend, weights of more rows than a layout has, and calls given a stream.

Tolerances, derived before the first run, are written at each test; the oracle is numpy in 64 bits.
"""

import numpy as np
import pytest
import torch

import oracle
from test_gpu_experts import (DEV, E2M1, E4M3, bf16_bits, bf16_dev, bits, moe, mx_random, note, poison, same_bits,
                              spread_rows, table, to_dev, weight_error_bound)  # noqa: F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- bases that descend


def disjoint(base, R):
    """The rows [lo, hi) of each group where a base below an earlier one counts as that one."""
    b, reached, out = np.clip(base, 0, R), 0, []
    for g in range(len(base) - 1):
        lo, reached = max(b[g], reached), max(b[g], b[g + 1], reached)
        out.append((lo, reached))
    return out


DESCENDING = [  # R, G, O, H: the waves that share H; four pairs of 32 x 64 and of 64 x 64; two pairs of 64 x 128
    (40, 6, 24, 160), (500, 8, 100, 544), (640, 32, 700, 544), (1600, 32, 300, 544), (3000, 40, 900, 544), (900, 130, 8, 64),
]


@pytest.mark.parametrize("R,G,O,H", DESCENDING)
def test_descending_bases_give_disjoint_groups(moe, R, G, O, H):  # noqa: F811
    """Each row of the groups' disjoint reading has the product with its own group's weights, whichever kernel
    runs, and no other row is touched. Exact sums: bit for bit."""
    rng = np.random.default_rng(R + O)
    note("descending bases", R, G, O, H)
    a, w = mx_random(rng, (R, H), -1, 1), mx_random(rng, (G, O, H), -1, 1)
    av, wv = oracle.mx_values(*a, E2M1), oracle.mx_values(*w, E2M1)
    ascending = np.linspace(0, R - 3, G + 1).astype(np.int32)
    swapped, back, random = ascending.copy(), ascending.copy(), rng.integers(-5, R + 5, G + 1).astype(np.int32)
    swapped[1], swapped[2] = swapped[2], swapped[1]
    back[G // 2] = 0
    for base in (ascending, swapped, back, random, random[::-1].copy(), ascending[::-1].copy()):
        want, inside = np.zeros((R, O)), np.zeros(R, dtype=bool)
        for g, (lo, hi) in enumerate(disjoint(base, R)):
            want[lo:hi] = av[lo:hi] @ wv[g].T
            inside[lo:hi] = True
        out = poison((R, O), torch.bfloat16)
        moe.moe_mx_product(moe.MxRows(*map(to_dev, a)), moe.MxRows(*map(to_dev, w)), to_dev(base), out=out)
        got = bf16_bits(out)
        same_bits(got[inside], bits(want[inside].astype(np.float32)), "rows of the groups")
        assert np.all(got[~inside] == 0xABAB)


# ---------------------------------------------------------------- the ends of the formats' ranges


@pytest.mark.parametrize("S,K,H", [(5, 2, 64), (40, 5, 2080), (9, 16, 8224)])
def test_checkpoint_gradient_of_the_largest_values(moe, S, K, H):  # noqa: F811
    """Rows that hold bf16's lowest and highest finite values: E4M3 holds them as 2^128, which fp32 does not, but
    their products with dy, zeros among it, are finite, and so is the gradient. The bound of the gradient's tests."""
    rng = np.random.default_rng(H)
    slot = table(rng, S, K, 2 * K, 0.1)
    R = S * K
    rows, w = spread_rows(rng, R, H), rng.random((S, K), dtype=np.float32)
    dy = bits(rng.standard_normal((S, H)) * 2.0**-40)
    rows[:, 7], rows[:, 40], rows[::2, 50] = 0xFF7F, 0x7F7F, 0x7F70
    dy[:, 7] = 0
    codes, scales = oracle.mx_quantize(rows, E4M3)
    values = oracle.mx_values(codes, scales, E4M3)
    assert np.abs(values).max() == 2.0**128
    y, kept = moe.moe_combine_checkpoint(bf16_dev(rows), to_dev(slot), to_dev(w))
    got = moe.moe_combine_backward_mx(bf16_dev(dy), kept, to_dev(slot), to_dev(w), d_expert_out=poison((R, H), torch.bfloat16))
    want, want_w, magnitude = oracle.combine_backward(dy, values, slot, w, np.full((R, H), 0xABAB))
    same_bits(bf16_bits(got[0]), want, "d_rows")
    assert np.isfinite(want_w).all()
    assert np.all(np.abs(got[1].cpu().numpy() - want_w) <= weight_error_bound(magnitude))


@pytest.mark.parametrize("R,O,H", [(20, 40, 256), (300, 300, 544), (900, 3000, 1056)])
def test_product_of_scales_far_apart(moe, R, O, H):  # noqa: F811
    """Scales near both ends of E8M0 whose products are near 1: exact sums as with scales near 1, bit for bit."""
    rng = np.random.default_rng(R)
    (a, _), (w, _) = mx_random(rng, (R, H), 0, 0), mx_random(rng, (2, O, H), 0, 0)
    far = rng.integers(-125, 126, H // 32)
    a_scales = (127 + far + rng.integers(-1, 2, (R, H // 32))).astype(np.uint8)
    w_scales = (127 - far + rng.integers(-1, 2, (2, O, H // 32))).astype(np.uint8)
    base = np.array([0, R // 3, R], dtype=np.int32)
    got = moe.moe_mx_product(moe.MxRows(to_dev(a), to_dev(a_scales)), moe.MxRows(to_dev(w), to_dev(w_scales)), to_dev(base))
    want = oracle.mx_product(oracle.mx_values(a, a_scales, E2M1), oracle.mx_values(w, w_scales, E2M1), base)
    same_bits(bf16_bits(got), bits(want.astype(np.float32)), "scales far apart")


# ---------------------------------------------------------------- gates far below zero, and not finite ones


def gated(c):
    """silu(gate) * up of exact sums [R, O], as the definition has it, in 64 bits."""
    gate, up = c[:, : c.shape[1] // 2], c[:, c.shape[1] // 2 :]
    with np.errstate(over="ignore", invalid="ignore"):
        return gate / (1 + np.exp(-gate)) * up


GATED = [(20, 2, 48, 128), (300, 3, 300, 160), (640, 32, 700, 128), (900, 8, 5000, 128), (4000, 4, 5200, 128)]


@pytest.mark.parametrize("R,G,O,H", GATED)
@pytest.mark.parametrize("up_scale", [-60, 0, 60])
def test_gates_far_below_zero(moe, R, G, O, H, up_scale):  # noqa: F811
    """Gates down to -400 with large, ordinary and tiny up projections. Sums are exact (one scale for the gates and
    one for the up rows, multiples of 1/4 below 36 * 160 times the scale). exp(v / 2), |v| <= 174, has an argument
    off by two roundings of at most 87 * 1.45, so 2 * 126 * ln 2 * 2^-24 < 2^-16 relative, twice that in its square
    with a few ulps: 2^-14; then half a bf16 step 2^-8 or half of bf16's smallest subnormal, 2^-134. Below
    -174 silu's magnitude is under 175 * exp(-174) and 0 may stand for it."""
    rng = np.random.default_rng(R + O)
    note("gates far below zero", R, G, O, H, up_scale)
    a, w = mx_random(rng, (R, H), 0, 0), mx_random(rng, (G, O, H), 0, 0)
    w[1][:, O // 2 :] = 127 + up_scale
    base = np.linspace(0, R, G + 1).astype(np.int32)
    out = moe.moe_mx_product(moe.MxRows(*map(to_dev, a)), moe.MxRows(*map(to_dev, w)), to_dev(base), moe.MOE_MX_GATED)
    c = oracle.mx_product(oracle.mx_values(*a, E2M1), oracle.mx_values(*w, E2M1), base)
    gate, up = c[:, : O // 2], c[:, O // 2 :]
    assert gate.min() < -180 and ((gate < -90) & (gate > -174)).any()
    want, got = gated(c), oracle.bf16_bits_to_f32(bf16_bits(out)).astype(np.float64)
    low = np.where(gate < -174, 175 * np.exp(-174.0) * np.abs(up), 0)
    assert np.all(np.abs(got - want) <= np.abs(want) * (2.0**-8 + 2.0**-14) + 2.0**-134 + low)


@pytest.mark.parametrize("R,G,O", [(40, 2, 64), (300, 2, 600), (640, 32, 700), (900, 8, 5000), (4000, 4, 5200)])
def test_gated_product_of_what_is_not_finite(moe, R, G, O):  # noqa: F811
    """One value a row, so that a sum is one product: gates and up projections of zero, ordinary, huge, infinite
    (past fp32's range) and NaN values in every pairing, against the definition applied to the sums as fp32 has
    them. Zeros keep their sign; tolerance as for finite gates."""
    rng = np.random.default_rng(R)
    H = 64
    a, w = mx_random(rng, (R, H), 0, 0), mx_random(rng, (G, O, H), 0, 0)
    a[0][:] = 0
    column = rng.integers(0, H, R)
    a[0][np.arange(R), column // 2] = np.where(column % 2 == 0, 0x02, 0x20)  # 1.0
    ends = np.array([127, 254, 255], dtype=np.uint8)
    a[1][:] = ends[np.minimum(rng.integers(0, 8, (R, 1)) // 3, 2)]
    w[1][:] = ends[np.minimum(rng.integers(0, 40, (G, O, 1)) // 19, 2)]
    base = np.linspace(0, R, G + 1).astype(np.int32)
    note("not finite", R, G, O)
    out = moe.moe_mx_product(moe.MxRows(*map(to_dev, a)), moe.MxRows(*map(to_dev, w)), to_dev(base), moe.MOE_MX_GATED)
    with np.errstate(over="ignore", invalid="ignore"):
        sums = oracle.mx_product(oracle.mx_values(*a, E2M1), oracle.mx_values(*w, E2M1), base).astype(np.float32).astype(np.float64)
        want = gated(sums).astype(np.float32).astype(np.float64)
        got = oracle.bf16_bits_to_f32(bf16_bits(out)).astype(np.float64)
        assert np.isnan(want).any() and np.isinf(want).any() and np.isfinite(want).any()
        assert np.array_equal(np.isnan(got), np.isnan(want))
        rest = ~np.isnan(want)
        same = got[rest] == want[rest]
        close = np.abs(got[rest] - want[rest]) <= np.abs(want[rest]) * (2.0**-8 + 2.0**-14) + 2.0**-134
        assert np.all(same | (close & np.isfinite(want[rest])))
        zero = rest & (want == 0) & (got == 0)
        assert np.array_equal(np.signbit(got[zero]), np.signbit(want[zero]))


# ---------------------------------------------------------------- matrices of more rows than a layout has


@pytest.mark.parametrize("form", [E2M1, E4M3])
def test_more_rows_than_a_layout(moe, form):  # noqa: F811
    """17 matrices of 65536 rows, more than 2^20: there and back, with a device count and without, and the E2M1 ones
    as the weights of a product."""
    rng = np.random.default_rng(40)
    G, O, H = 17, 65536, 32
    w = bits(rng.standard_normal((G * O, H)))
    codes, scales = oracle.mx_quantize(w, form)
    dev = bf16_dev(w)
    q = moe.moe_mx_quantize(dev, form)
    assert np.array_equal(q.codes.cpu().numpy(), codes) and np.array_equal(q.scales.cpu().numpy(), scales)
    values = bits(oracle.mx_values(codes, scales, form).astype(np.float32))
    assert np.array_equal(bf16_bits(moe.moe_mx_dequantize(q, form)), values)
    for count in (-(2**31), 0, 1000, 2**20, 2**20 + 9, G * O, 2**31 - 1):
        n, num = min(max(count, 0), G * O), torch.tensor([count], dtype=torch.int32, device=DEV)
        out = moe.MxRows(poison(codes.shape, torch.uint8), poison(scales.shape, torch.uint8))
        moe.moe_mx_quantize(dev, form, num_rows=num, out=out)
        for got, want in zip(out, (codes, scales)):
            got = got.cpu().numpy()
            assert np.array_equal(got[:n], want[:n]) and np.all(got[n:] == 0xAB), count
        back = poison((G * O, H + 8), torch.bfloat16)
        moe.moe_mx_dequantize(q, form, num_rows=num, out=back[:, :H])
        got = bf16_bits(back)
        assert np.array_equal(got[:n, :H], values[:n]) and np.all(got[n:] == 0xABAB) and np.all(got[:, H:] == 0xABAB), count
    if form == E4M3:
        return
    counts = [3, 0, 0, 7] + [0] * 12 + [5]
    base = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    a = mx_random(rng, (int(base[-1]), H), 0, 0)
    got = moe.moe_mx_product(moe.MxRows(*map(to_dev, a)), moe.MxRows(q.codes.view(G, O, H // 2), q.scales.view(G, O, 1)), to_dev(base))
    av, wv = oracle.mx_values(*a, E2M1), oracle.mx_values(codes, scales, E2M1).reshape(G, O, H)
    want, size = oracle.mx_product(av, wv, base), oracle.mx_product(np.abs(av), np.abs(wv), base)
    # 32 roundings or truncations of partial sums, then half a bf16 step
    assert np.all(np.abs(oracle.bf16_bits_to_f32(bf16_bits(got)).astype(np.float64) - want) <= H * 2.0**-23 * size + 2.0**-8 * np.abs(want))


def test_more_rows_on_a_stream_and_refused(moe):  # noqa: F811
    """The same with a stream of its own, behind a delayed count, and buffers that overlap in different parts."""
    rng = np.random.default_rng(41)
    n, H = 2**20 + 64, 32
    rows = bits(rng.standard_normal((n, H)))
    codes, scales = oracle.mx_quantize(rows, E4M3)
    dev, num, most = bf16_dev(rows), torch.zeros(1, dtype=torch.int32, device=DEV), torch.tensor([n - 3], dtype=torch.int32, device=DEV)
    out = moe.MxRows(poison(codes.shape, torch.uint8), poison(scales.shape, torch.uint8))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        num.copy_(most)
    moe.moe_mx_quantize(dev, E4M3, num_rows=num, out=out, stream=side)
    side.synchronize()
    for got, want in zip(out, (codes, scales)):
        got = got.cpu().numpy()
        assert np.array_equal(got[: n - 3], want[: n - 3]) and np.all(got[n - 3 :] == 0xAB)
    both = torch.zeros(n * H * 2 + n * H - 64 * H, dtype=torch.uint8, device=DEV)
    x = both[: n * H * 2].view(torch.bfloat16).view(n, H)
    over = both[n * H * 2 - 64 * H :].view(n, H)  # its first rows lie over the last of x
    with pytest.raises(ValueError, match="overlap"):
        moe.moe_mx_quantize(x, E4M3, out=moe.MxRows(over, out.scales))
    with pytest.raises(ValueError, match="overlap"):
        moe.moe_mx_dequantize(moe.MxRows(over, out.scales), E4M3, out=x)
    with pytest.raises(ValueError):
        moe.moe_mx_quantize(torch.zeros((n, 48), dtype=torch.bfloat16, device=DEV), E4M3)
    with pytest.raises(ValueError):
        moe.moe_mx_quantize(dev, 3)
    torch.cuda.synchronize()
    assert not both.any()


# ---------------------------------------------------------------- the stream argument


class Handle:
    """A stream of another library: an object with the raw handle."""

    def __init__(self, stream):
        self.stream, self.cuda_stream = stream, stream.cuda_stream


@pytest.mark.parametrize("kind", [lambda s: s, lambda s: s.cuda_stream, Handle], ids=["stream", "handle", "object"])
def test_every_call_runs_on_the_stream_it_is_given(moe, kind):  # noqa: F811
    """The inputs are produced late on a stream, the calls are given that stream while the current one is idle, and
    only that stream is waited for: a call on any other reads the inputs' old contents."""
    S, K, E, H, G, O = 64, 4, 8, 512, 3, 96

    def inputs(seed):
        rng = np.random.default_rng(seed)
        slot = table(rng, S, K, E, 0.1)
        a, w = mx_random(rng, (S * K, H), -1, 1), mx_random(rng, (G, O, H), -1, 1)
        return [bf16_dev(spread_rows(rng, S * K, H)), bf16_dev(spread_rows(rng, S, H)), to_dev(slot), to_dev(rng.random((S, K), dtype=np.float32)),
                *map(to_dev, a), *map(to_dev, w), to_dev(np.array([0, 100, 120, S * K], dtype=np.int32)),
                to_dev(rng.integers(0, 127, (S * K, H)).astype(np.uint8)), to_dev(rng.integers(100, 140, (S * K, H // 32)).astype(np.uint8))]

    calls = {
        "combine_backward": lambda v, **kw: moe.moe_combine_backward(v[1], v[0], v[2], v[3], **kw)[1:],
        "combine_checkpoint": lambda v, **kw: moe.moe_combine_checkpoint(v[0], v[2], v[3], **kw)[:1],
        "combine_backward_mx": lambda v, **kw: moe.moe_combine_backward_mx(v[1], (v[9], v[10]), v[2], v[3], **kw)[1:],
        "dispatch_backward": lambda v, **kw: (moe.moe_dispatch_backward(v[0], v[2], **kw),),
        "quantize": lambda v, **kw: moe.moe_mx_quantize(v[0], E2M1, **kw),
        "dequantize": lambda v, **kw: (moe.moe_mx_dequantize((v[9], v[10]), E4M3, **kw),),
        "product": lambda v, **kw: (moe.moe_mx_product((v[4], v[5]), (v[6], v[7]), v[8], **kw),),
    }
    old, new = inputs(50), inputs(51)
    want = {name: [t.clone() for t in call(new)] for name, call in calls.items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        for mine, fresh in zip(old, new):
            mine.copy_(fresh)
    got = {name: call(old, stream=kind(side)) for name, call in calls.items()}
    late = not side.query()
    side.synchronize()
    assert late, "the producer was done before the calls were made"
    for name in calls:
        for g, w in zip(got[name], want[name]):
            assert torch.equal(g.view(torch.uint8), w.view(torch.uint8)), name
