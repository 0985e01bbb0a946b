"""GPU tests of the gradients, the MX rows, the 8-bit checkpoints and the experts' product against the oracle.

Exact wherever the result is one defined sequence of roundings: MX codes and scales, the row and dispatch
gradients, the checkpointed combine's y. Tolerances elsewhere, derived before the first run:

* d_topk_weights, an fp32 sum of H products in an order fixed by H. Every term passes at most `depth` additions
  (each a rounding of 2^-24 relative to a partial sum that the terms' magnitudes bound), so the error is
  at most depth * 2^-24 * sum|terms|, up to second order. depth <= 128 covers any tree of lanes (64) whose
  leaves are sequential sums of up to 64 terms with 64 joins; products are fused, or add one more.
* the product: with scales 2^-1, 1 and 2 every product is a multiple of 2^-4 and every partial sum below
  36 * 4 * H < 2^24 * 2^-4 for H <= 7168, so fp32 accumulation is exact in any order and the plain result is the
  exact sum rounded once: bit for bit. With free scales: H roundings (or truncations, 2^-23) of partial sums
  bounded by sum|terms|, then half a bf16 step: H * 2^-23 * sum|terms| + 2^-8 * |c|.
* the gated product of exact sums: exp is exp2(v * log2(e)), whose argument is off by two roundings, 2 * |v| * 1.45 *
  2^-24 absolute, hence 2 * |v| * 2^-24 relative in the result, |v| <= 88, plus a few ulps for exp2, sum, quotient
  and product: below 2^-16; then half a bf16 step 2^-8. Below v = -88 the exact value is under 88 * exp(-88)
  = 6e-37 times the up projection, and 0 may stand for it.
"""

import numpy as np
import pytest
import torch

import oracle
from workloads import f32_to_bf16_input, random_tiny_routing

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
POISON = 0xAB
E2M1, E4M3 = 1, 2


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    import combine_moe_layout_02_amd as m

    return m


def note(*a):
    print(*a, flush=True)


def to_dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def bf16_dev(bits):
    return to_dev(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16)


def bf16_bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def bits(a):
    return f32_to_bf16_input(np.asarray(a, dtype=np.float32))


def poison(shape, dtype):
    t = torch.empty(shape, dtype=dtype, device=DEV)
    t.view(torch.uint8).fill_(POISON)
    return t


def strided(bits_rows, gap):
    """Device rows at a stride of H + gap values, with poison between them."""
    R, H = bits_rows.shape
    t = poison((R, H + gap), torch.bfloat16)
    t[:, :H] = bf16_dev(bits_rows)
    return t[:, :H]


def same_bits(got, want, what=""):
    """Equal bit patterns; a NaN equals any NaN."""
    g, w = oracle.bf16_bits_to_f32(got), oracle.bf16_bits_to_f32(want)
    bad = (got != want) & ~(np.isnan(g) & np.isnan(w))
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what} at {i}: {g[i]!r} for {w[i]!r}, {int(bad.sum())} differ")


def table(rng, S, K, E, p_mask):
    idx = random_tiny_routing(rng, S, K, E, p_mask=p_mask)
    return oracle.layout(idx, E, 1, 1)["slot_idx"]


def spread_rows(rng, R, H):
    return bits(rng.standard_normal((R, H)) * np.exp2(rng.integers(-6, 6, (R, 1))))


# ---------------------------------------------------------------- MX rows


def mx_case(moe, rows, form, what):
    want_codes, want_scales = oracle.mx_quantize(rows, form)
    got = moe.moe_mx_quantize(bf16_dev(rows), form)
    assert np.array_equal(got.scales.cpu().numpy(), want_scales), what
    codes = got.codes.cpu().numpy()
    if not np.array_equal(codes, want_codes):
        r, c = np.argwhere(codes != want_codes)[0]
        raise AssertionError(f"{what} row {r} byte {c}: {codes[r, c]:#x} for {want_codes[r, c]:#x}, "
                             f"{int((codes != want_codes).sum())} differ")
    back = bf16_bits(moe.moe_mx_dequantize(got, form))
    same_bits(back, bits(oracle.mx_values(want_codes, want_scales, form).astype(np.float32)), what)


@pytest.mark.parametrize("form", [E2M1, E4M3])
def test_every_bf16_value(moe, form):
    """All 65536 bf16 bit patterns, in order (blocks of neighbours) and in shuffles of the finite ones (blocks
    whose largest value is huge), and blocks of one exponent range each."""
    rng = np.random.default_rng(1)
    every = np.arange(65536, dtype=np.uint16)
    mx_case(moe, every.reshape(64, 1024), form, "in order")
    finite = every[(every & 0x7F80) != 0x7F80]
    mx_case(moe, rng.permutation(finite)[: 65024].reshape(-1, 256), form, "shuffled")
    # every mantissa against every block maximum, exponents up to 12 below it
    rows = []
    for E in range(0, 255):
        e = np.clip(E - rng.integers(0, 13, 512), 0, E)
        rows.append((e << 7) | rng.integers(0, 128, 512) | (rng.integers(0, 2, 512) << 15))
    mx_case(moe, np.array(rows).astype(np.uint16), form, "one exponent range")


@pytest.mark.parametrize("form", [E2M1, E4M3])
@pytest.mark.parametrize("R,H,gap", [(1, 32, 0), (3, 64, 8), (17, 2080, 0), (5, 7168, 512), (2, 16384, 0), (130, 96, 40)])
def test_mx_rows_and_strides(moe, form, R, H, gap):
    rng = np.random.default_rng(R * H)
    rows = spread_rows(rng, R, H)
    want_codes, want_scales = oracle.mx_quantize(rows, form)
    out = moe.MxRows(poison(want_codes.shape, torch.uint8), poison(want_scales.shape, torch.uint8))
    n = R - 1 if R > 2 else R  # a device count below the buffer's rows: the last row stays as it was
    count = torch.tensor([n], dtype=torch.int32, device=DEV)
    moe.moe_mx_quantize(strided(rows, gap), form, num_rows=count, out=out)
    codes, scales = out.codes.cpu().numpy(), out.scales.cpu().numpy()
    assert np.array_equal(codes[:n], want_codes[:n]) and np.array_equal(scales[:n], want_scales[:n])
    assert np.all(codes[n:] == POISON) and np.all(scales[n:] == POISON)
    back = poison((R, H + gap), torch.bfloat16)
    full = moe.MxRows(to_dev(want_codes), to_dev(want_scales))
    moe.moe_mx_dequantize(full, form, num_rows=count, out=back[:, :H])
    got = bf16_bits(back)
    same_bits(got[:n, :H], bits(oracle.mx_values(want_codes, want_scales, form).astype(np.float32))[:n])
    assert np.all(got[n:] == 0xABAB) and np.all(got[:, H:] == 0xABAB)


@pytest.mark.parametrize("count", [-3, 0, 1, 9, 1000])
def test_mx_counts(moe, count):
    rows = spread_rows(np.random.default_rng(3), 9, 64)
    want = oracle.mx_quantize(rows, E4M3)
    out = moe.MxRows(poison((9, 64), torch.uint8), poison((9, 2), torch.uint8))
    moe.moe_mx_quantize(bf16_dev(rows), E4M3, num_rows=torch.tensor([count], dtype=torch.int32, device=DEV), out=out)
    n = min(max(count, 0), 9)
    assert np.array_equal(out.codes.cpu().numpy()[:n], want[0][:n]) and np.all(out.codes.cpu().numpy()[n:] == POISON)
    assert np.array_equal(out.scales.cpu().numpy()[:n], want[1][:n]) and np.all(out.scales.cpu().numpy()[n:] == POISON)


def test_mx_of_no_rows(moe):
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    q = moe.moe_mx_quantize(x, E2M1)
    assert tuple(q.codes.shape) == (0, 32) and tuple(moe.moe_mx_dequantize(q, E2M1).shape) == (0, 64)
    w = moe.MxRows(torch.zeros((2, 8, 32), dtype=torch.uint8, device=DEV), torch.zeros((2, 8, 2), dtype=torch.uint8, device=DEV))
    base = torch.zeros(3, dtype=torch.int32, device=DEV)
    assert tuple(moe.moe_mx_product(q, w, base).shape) == (0, 8)


# ---------------------------------------------------------------- gradients

TABLES = [  # S, K, E, H, masked share
    (1, 1, 1, 16, 0.0), (1, 8, 16, 7168, 0.0), (3, 2, 4, 1024, 0.5), (33, 3, 7, 2064, 0.2), (128, 2, 16, 1024, 0.0),
    (40, 16, 64, 96, 0.1), (7, 5, 9, 8192, 0.1), (5, 4, 6, 16384, 0.1), (9, 9, 20, 8208, 0.0), (21, 6, 48, 2080, 1.0),
    (700, 8, 64, 512, 0.05), (6, 16, 40, 16384, 0.1),
]
MX_TABLES = [(s, k, e, (h + 31) // 32 * 32, p) for s, k, e, h, p in TABLES]


def weight_error_bound(magnitude):
    return 128 * 2.0**-24 * magnitude + 1e-37


def check_combine_backward(moe, run, rows_value, dy, slot, w, R, H, gap=0):
    S, K = slot.shape
    before = np.full((R, H), 0xABAB, dtype=np.uint16)
    want_rows, want_w, magnitude = oracle.combine_backward(dy, rows_value, slot, w, before)
    d_rows, d_w = poison((R, H + gap), torch.bfloat16), poison((S, K), torch.float32)
    run(d_rows[:, :H], d_w)
    got = bf16_bits(d_rows)
    same_bits(got[:, :H], want_rows, "d_rows")
    assert np.all(got[:, H:] == 0xABAB)
    got_w = d_w.cpu().numpy().astype(np.float64)
    finite = np.isfinite(want_w)
    assert np.array_equal(np.isnan(got_w), np.isnan(want_w)) and np.array_equal(got_w[~finite & ~np.isnan(want_w)], want_w[~finite & ~np.isnan(want_w)])
    err = np.abs(got_w - want_w)[finite]
    assert np.all(err <= weight_error_bound(magnitude)[finite]), float(np.max(err / (magnitude[finite] + 1e-37))) * 2**24


@pytest.mark.parametrize("S,K,E,H,p", TABLES)
@pytest.mark.parametrize("gap", [0, 24])
def test_combine_backward(moe, S, K, E, H, p, gap):
    rng = np.random.default_rng(S * 31 + H)
    slot = table(rng, S, K, E, p)
    R = S * K
    rows, dy = spread_rows(rng, R, H), spread_rows(rng, S, H)
    w = rng.random((S, K), dtype=np.float32)
    note("combine_backward", S, K, E, H, p, gap)
    src = strided(rows, gap)
    check_combine_backward(
        moe, lambda d, dw: moe.moe_combine_backward(bf16_dev(dy), src, to_dev(slot), to_dev(w), d, dw),
        oracle.bf16_bits_to_f32(rows).astype(np.float64), dy, slot, w, R, H, gap)


def test_combine_backward_skips_rows_out_of_range(moe):
    """Entries at or past expert_rows, and any negative entry, take no part: fewer rows than the table names."""
    rng = np.random.default_rng(2)
    S, K, H, R = 20, 4, 256, 50
    slot = table(rng, S, K, 8, 0.1)
    slot[3, 1] = -2147483648
    slot[4, 2] = 2147483647
    rows, dy, w = spread_rows(rng, R, H), spread_rows(rng, S, H), rng.random((S, K), dtype=np.float32)
    check_combine_backward(
        moe, lambda d, dw: moe.moe_combine_backward(bf16_dev(dy), bf16_dev(rows), to_dev(slot), to_dev(w), d, dw),
        oracle.bf16_bits_to_f32(rows).astype(np.float64), dy, slot, w, R, H)
    dx = bf16_bits(moe.moe_dispatch_backward(bf16_dev(rows), to_dev(slot)))
    same_bits(dx, oracle.dispatch_backward(rows, slot))


def test_combine_backward_non_finite(moe):
    """NaN and infinities in rows that no entry names stay out of every result; in named rows they reach their own
    entry's weight gradient only; in dy and in a weight they go where IEEE products take them."""
    rng = np.random.default_rng(4)
    S, K, H = 12, 3, 128
    slot = table(rng, S, K, 6, 0.3)
    R = S * K
    rows, dy, w = spread_rows(rng, R, H), spread_rows(rng, S, H), rng.random((S, K), dtype=np.float32)
    rows[int(slot.max()) + 1 :] = 0x7FC0
    rows[slot[slot >= 0][0], 5] = 0x7F80  # +inf
    dy[5, 7] = 0x7FC0
    w[0, 0] = np.inf
    with np.errstate(invalid="ignore"):
        check_combine_backward(
            moe, lambda d, dw: moe.moe_combine_backward(bf16_dev(dy), bf16_dev(rows), to_dev(slot), to_dev(w), d, dw),
            oracle.bf16_bits_to_f32(rows).astype(np.float64), dy, slot, w, R, H)
        same_bits(bf16_bits(moe.moe_dispatch_backward(bf16_dev(rows), to_dev(slot))), oracle.dispatch_backward(rows, slot))


@pytest.mark.parametrize("S,K,E,H,p", TABLES)
@pytest.mark.parametrize("gap", [0, 8])
def test_dispatch_backward(moe, S, K, E, H, p, gap):
    rng = np.random.default_rng(S * 37 + H)
    slot = table(rng, S, K, E, p)
    rows = spread_rows(rng, S * K, H)
    note("dispatch_backward", S, K, E, H, p, gap)
    dx = poison((S, H), torch.bfloat16)
    moe.moe_dispatch_backward(strided(rows, gap), to_dev(slot), dx=dx)
    same_bits(bf16_bits(dx), oracle.dispatch_backward(rows, slot))


def test_gradients_are_differences(moe):
    """The calls' own forwards, moved by small integers: every value and sum is exact, so are the differences."""
    rng = np.random.default_rng(30)
    S, K, E, H = 33, 3, 7, 64
    idx = to_dev(random_tiny_routing(rng, S, K, E, p_mask=0.2))
    lay = moe.moe_layout(idx, E, 1, 1)
    slot, R = lay.slot_idx, S * K
    small = lambda shape, n: torch.from_numpy(rng.integers(-n, n + 1, shape).astype(np.float32)).to(DEV)  # noqa: E731
    rows, dy, w, x = small((R, H), 3), small((S, H), 3), small((S, K), 4), small((S, H), 3)
    as_bf16 = lambda t: t.to(torch.bfloat16).contiguous()  # noqa: E731

    def loss(rows, w):
        return float((dy.double() * moe.moe_combine(as_bf16(rows), slot, w.contiguous()).double()).sum())

    start = torch.zeros((R, H), dtype=torch.bfloat16, device=DEV)
    d_rows, d_w = moe.moe_combine_backward(as_bf16(dy), as_bf16(rows), slot, w, d_expert_out=start)
    for _ in range(3):
        step, w_step = small((R, H), 2), small((S, K), 2)
        assert loss(rows + step, w) - loss(rows, w) == float((step.double() * d_rows.double()).sum())
        assert loss(rows, w + w_step) - loss(rows, w) == float((w_step.double() * d_w.double()).sum())

    g = small((R, H), 3)
    dx = moe.moe_dispatch_backward(as_bf16(g), slot)
    N = int(lay.expert_slot_base[-1])

    def sent(x):
        win = torch.zeros(moe.moe_window_bytes(S, K, H), dtype=torch.uint8, device=DEV)
        moe.moe_dispatch(as_bf16(x), slot, win, moe.MOE_QUANT_NONE)
        rows = win.view(R, -1)[:N, : 2 * H].contiguous().view(torch.bfloat16)
        return float((g[:N].double() * rows.double()).sum())

    for _ in range(3):
        step = small((S, H), 2)
        assert sent(x + step) - sent(x) == float((step.double() * dx.double()).sum())


def test_one_row_in_two_entries(moe):
    """A table that names rows twice: sums and weight gradients count each entry, 16 bytes of a gradient row are
    those of one of its products, the checkpoint holds the row."""
    rng = np.random.default_rng(31)
    S, K, H, R = 24, 4, 512, 9
    slot = rng.integers(-1, R, (S, K)).astype(np.int32)
    slot[:, 3] = slot[:, 0]
    rows, dy, w = spread_rows(rng, R, H), spread_rows(rng, S, H), rng.random((S, K), dtype=np.float32)
    y, kept = moe.moe_combine_checkpoint(bf16_dev(rows), to_dev(slot), to_dev(w))
    same_bits(bf16_bits(y), oracle.combine(rows, slot, w), "y")
    codes, scales = oracle.mx_quantize(rows, E4M3)
    assert np.array_equal(kept.codes.cpu().numpy(), codes) and np.array_equal(kept.scales.cpu().numpy(), scales)
    same_bits(bf16_bits(moe.moe_dispatch_backward(bf16_dev(rows), to_dev(slot))), oracle.dispatch_backward(rows, slot), "dx")
    kept_values = oracle.mx_values(codes, scales, E4M3)
    for got, values in ((moe.moe_combine_backward(bf16_dev(dy), bf16_dev(rows), to_dev(slot), to_dev(w)), oracle.bf16_bits_to_f32(rows)),
                        (moe.moe_combine_backward_mx(bf16_dev(dy), kept, to_dev(slot), to_dev(w)), kept_values)):
        _, want_w, magnitude = oracle.combine_backward(dy, values.astype(np.float64), slot, w, np.zeros((R, H)))
        assert np.all(np.abs(got[1].cpu().numpy() - want_w) <= weight_error_bound(magnitude))
        d_rows = bf16_bits(got[0])
        for s in range(R):
            t, k = np.nonzero(slot == s)
            products = bits(w[t, k, None] * oracle.bf16_bits_to_f32(dy[t])).reshape(-1, H // 8, 8)
            assert np.all((products == d_rows[s].reshape(-1, 8)).all(axis=2).any(axis=0)), s


def test_the_most_entries(moe):
    """65536 tokens of 16 entries, the smallest rows."""
    rng = np.random.default_rng(32)
    S, K, H = 65536, 16, 32
    R = S * K
    slot = rng.permutation(R).astype(np.int32).reshape(S, K)
    slot[rng.random((S, K)) < 0.1] = -1
    rows, dy, w = bits(rng.standard_normal((R, H))), bits(rng.standard_normal((S, H))), rng.random((S, K), dtype=np.float32)
    src, idx, weights = bf16_dev(rows), to_dev(slot), to_dev(w)
    check_combine_backward(moe, lambda d, dw: moe.moe_combine_backward(bf16_dev(dy), src, idx, weights, d, dw),
                           oracle.bf16_bits_to_f32(rows).astype(np.float64), dy, slot, w, R, H)
    same_bits(bf16_bits(moe.moe_dispatch_backward(src, idx)), oracle.dispatch_backward(rows, slot))
    y, kept = moe.moe_combine_checkpoint(src, idx, weights)
    same_bits(bf16_bits(y), oracle.combine(rows, slot, w), "y")
    codes, scales = oracle.mx_quantize(rows, E4M3)
    live = np.sort(slot[slot >= 0])
    assert np.array_equal(kept.codes.cpu().numpy()[live], codes[live]) and np.array_equal(kept.scales.cpu().numpy()[live], scales[live])
    all_rows = moe.moe_mx_quantize(src, E2M1)  # the most rows
    codes, scales = oracle.mx_quantize(rows, E2M1)
    assert np.array_equal(all_rows.codes.cpu().numpy(), codes) and np.array_equal(all_rows.scales.cpu().numpy(), scales)


def test_rows_past_4_gib(moe):
    """Rows, checkpoints and gradients whose offsets pass 32 bits."""
    rng = np.random.default_rng(33)
    S, K, H, R = 3, 2, 16384, 300_000
    slot = np.array([[299_999, 5], [-1, 262_143], [140_000, 262_144]], dtype=np.int32)
    named = slot[slot >= 0]
    values, dy, w = spread_rows(rng, len(named), H), spread_rows(rng, S, H), rng.random((S, K), dtype=np.float32)
    place = np.full((S, K), -1, dtype=np.int32)  # the same table over the named rows alone
    place[slot >= 0] = np.arange(len(named))
    rows, where = torch.empty((R, H), dtype=torch.bfloat16, device=DEV), to_dev(named.astype(np.int64))
    rows[where] = bf16_dev(values)
    y, kept = moe.moe_combine_checkpoint(rows, to_dev(slot), to_dev(w))
    same_bits(bf16_bits(y), oracle.combine(values, place, w), "y")
    codes, scales = oracle.mx_quantize(values, E4M3)
    assert np.array_equal(kept.codes[where].cpu().numpy(), codes) and np.array_equal(kept.scales[where].cpu().numpy(), scales)
    same_bits(bf16_bits(moe.moe_dispatch_backward(rows, to_dev(slot))), oracle.dispatch_backward(values, place), "dx")
    d_rows = torch.empty_like(rows)
    for call, v in ((lambda: moe.moe_combine_backward(bf16_dev(dy), rows, to_dev(slot), to_dev(w), d_rows), oracle.bf16_bits_to_f32(values)),
                    (lambda: moe.moe_combine_backward_mx(bf16_dev(dy), kept, to_dev(slot), to_dev(w), d_rows), oracle.mx_values(codes, scales, E4M3))):
        d_w = call()[1]
        want, want_w, magnitude = oracle.combine_backward(dy, v.astype(np.float64), place, w, values)
        same_bits(bf16_bits(d_rows[where]), want, "d_rows")
        assert np.all(np.abs(d_w.cpu().numpy() - want_w) <= weight_error_bound(magnitude))
    back = moe.moe_mx_dequantize(moe.moe_mx_quantize(rows[299_990:], E2M1), E2M1)
    assert np.array_equal(bf16_bits(back[9:]), bits(oracle.mx_values(*oracle.mx_quantize(values[:1], E2M1), E2M1)))
    whole = moe.moe_mx_quantize(rows, E2M1, out=moe.MxRows(kept.codes.view(-1)[: R * H // 2].view(R, H // 2), kept.scales))
    codes, scales = oracle.mx_quantize(values, E2M1)
    assert np.array_equal(whole.codes[where].cpu().numpy(), codes) and np.array_equal(whole.scales[where].cpu().numpy(), scales)
    back = moe.moe_mx_dequantize(whole, E2M1, out=d_rows)
    assert np.array_equal(bf16_bits(back[where]), bits(oracle.mx_values(codes, scales, E2M1)))


# ---------------------------------------------------------------- 8-bit checkpoints


@pytest.mark.parametrize("S,K,E,H,p", MX_TABLES)
@pytest.mark.parametrize("gap", [0, 16])
def test_checkpoint_and_its_gradient(moe, S, K, E, H, p, gap):
    rng = np.random.default_rng(S * 41 + H)
    slot = table(rng, S, K, E, p)
    R = S * K
    rows, dy, w = spread_rows(rng, R, H), spread_rows(rng, S, H), rng.random((S, K), dtype=np.float32)
    note("checkpoint", S, K, E, H, p, gap)
    kept = moe.MxRows(poison((R, H), torch.uint8), poison((R, H // 32), torch.uint8))
    y = poison((S, H), torch.bfloat16)
    moe.moe_combine_checkpoint(strided(rows, gap), to_dev(slot), to_dev(w), y=y, checkpoint=kept)
    same_bits(bf16_bits(y), oracle.combine(rows, slot, w), "y")
    codes, scales = oracle.mx_quantize(rows, E4M3)
    named = np.zeros(R, dtype=bool)
    named[slot[slot >= 0]] = True
    got_codes, got_scales = kept.codes.cpu().numpy(), kept.scales.cpu().numpy()
    assert np.array_equal(got_codes[named], codes[named]) and np.array_equal(got_scales[named], scales[named])
    assert np.all(got_codes[~named] == POISON) and np.all(got_scales[~named] == POISON)
    check_combine_backward(
        moe, lambda d, dw: moe.moe_combine_backward_mx(bf16_dev(dy), kept, to_dev(slot), to_dev(w), d, dw),
        oracle.mx_values(codes, scales, E4M3), dy, slot, w, R, H, gap)


def test_checkpoint_of_non_finite_rows(moe):
    """A NaN or an infinity makes its block of the checkpoint NaN, and with it that entry's weight gradient, and
    nothing else; y is the combine's."""
    rng = np.random.default_rng(9)
    S, K, H = 10, 2, 64
    slot = table(rng, S, K, 4, 0.2)
    R = S * K
    rows, dy, w = spread_rows(rng, R, H), spread_rows(rng, S, H), rng.random((S, K), dtype=np.float32)
    first, second = slot[slot >= 0][:2]
    rows[first, 40], rows[second, 3] = 0x7F80, 0xFFC0
    with np.errstate(invalid="ignore"):
        y, kept = moe.moe_combine_checkpoint(bf16_dev(rows), to_dev(slot), to_dev(w))
        same_bits(bf16_bits(y), oracle.combine(rows, slot, w), "y")
        codes, scales = oracle.mx_quantize(rows, E4M3)
        check_combine_backward(
            moe, lambda d, dw: moe.moe_combine_backward_mx(bf16_dev(dy), kept, to_dev(slot), to_dev(w), d, dw),
            oracle.mx_values(codes, scales, E4M3), dy, slot, w, R, H)


# ---------------------------------------------------------------- the product


def mx_random(rng, shape, low, high):
    """Random E2M1 rows [..., H]: any code, scale exponents in [low, high]."""
    codes = rng.integers(0, 256, (*shape[:-1], shape[-1] // 2)).astype(np.uint8)
    scales = rng.integers(127 + low, 127 + high + 1, (*shape[:-1], shape[-1] // 32)).astype(np.uint8)
    return codes, scales


def product_case(moe, rng, counts, H, O, gated, low=-1, high=1, behind=0, before=0, gap=0):
    """Runs a product on random codes; returns what came out, the exact sums and the sums of magnitudes (of the
    grouped rows), having checked that nothing else was written."""
    G = len(counts)
    base = (before + np.concatenate([[0], np.cumsum(counts)])).astype(np.int32)
    R = int(base[-1]) + behind
    a, w = mx_random(rng, (R, H), low, high), mx_random(rng, (G, O, H), low, high)
    width = O // 2 if gated else O
    out = poison((R, width + gap), torch.bfloat16)
    moe.moe_mx_product(moe.MxRows(*map(to_dev, a)), moe.MxRows(*map(to_dev, w)), to_dev(base),
                       moe.MOE_MX_GATED if gated else moe.MOE_MX_PLAIN, out=out[:, :width])
    got = bf16_bits(out)
    rows = slice(before, int(base[-1]))
    untouched = np.ones(got.shape, dtype=bool)
    untouched[rows, :width] = False
    assert np.all(got[untouched] == 0xABAB), "wrote outside the groups' rows"
    av, wv = oracle.mx_values(*a, E2M1), oracle.mx_values(*w, E2M1)
    exact = oracle.mx_product(av, wv, base)[rows]
    magnitude = oracle.mx_product(np.abs(av), np.abs(wv), base)[rows]
    return got[rows, :width], exact, magnitude


PRODUCTS = [  # rows of each group, H, O
    ([1], 32, 1), ([1], 32, 2), ([3, 0, 1], 64, 16), ([0, 0, 5], 96, 18), ([16, 17, 15], 128, 64), ([0, 33, 0, 1, 0], 160, 100),
    ([130, 7], 288, 130), ([256, 255, 257], 256, 256), ([1] * 40, 512, 72), ([300], 1056, 1000), ([2, 600, 61], 544, 322),
    ([8] * 3, 7168, 258), ([9] * 5, 7168, 96), ([20, 3, 0, 31], 512, 66), ([12, 40], 736, 32), ([1, 2], 480, 48),
    ([200, 170, 300, 0] * 4, 512, 4100),
    ([200, 170, 300, 0] * 4, 1056, 4100), ([50] * 30, 544, 2500), ([300, 90, 0, 260] * 8, 512, 300), ([7] * 64, 544, 1500),
    ([7] * 64, 1024, 700), ([1000], 768, 6200), ([65, 0, 64, 63], 2048, 510), ([5, 1, 0, 2], 7168, 130), ([40] * 20, 608, 90), ([513, 0, 1023], 992, 514),
    ([700, 690], 480, 9000), ([90] * 20, 96, 1300), ([30000, 20000], 32, 66), ([2, 1], 32, 65536), ([50, 3] * 8, 224, 700),
    ([30, 31], 1024, 3840), ([30, 31], 544, 3842), ([40, 44, 30, 46], 1056, 2400), ([40, 44, 0, 46], 1120, 2402), ([40, 44, 30, 46], 2080, 7200),
    ([60, 1, 64, 33], 2144, 7202), ([90, 60, 100, 30], 4128, 7200), ([127, 1, 128, 5], 4192, 7202), ([400, 380], 4096, 12960), ([500, 290], 4128, 12801),
    ([7400, 7500, 7690, 7410], 96, 1680),
]


@pytest.mark.parametrize("counts,H,O", PRODUCTS)
def test_product_exact(moe, counts, H, O):
    rng = np.random.default_rng(H + O)
    note("product", counts, H, O)
    got, exact, _ = product_case(moe, rng, counts, H, O, False, before=2, behind=3, gap=O % 3)
    same_bits(got, bits(exact.astype(np.float32)), "product")


@pytest.mark.parametrize("counts", [[0] * 8 + [3], [0] * 7 + [300, 200]])
def test_product_of_weights_past_4_gib(moe, counts):
    """The largest matrices and rows: 9 x 65536 x 16384 codes, of which the last groups' first and last rows are
    compared. Scales of 1: products are multiples of 1/4 and sums below 36 * 16384 < 2^24 / 4, exact in fp32."""
    rng = np.random.default_rng(34)
    G, O, H = len(counts), 65536, 16384
    base = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R = int(base[-1])
    codes = torch.zeros((G, O, H // 2), dtype=torch.uint8, device=DEV)
    picked = np.array([0, 1, 130, 40_000, 65_407, 65_534, 65_535])
    some = mx_random(rng, (G, len(picked), H), 0, 0)
    for g in range(G):
        codes[g, to_dev(picked)] = to_dev(some[0][g])
    scales = torch.full((G, O, H // 32), 127, dtype=torch.uint8, device=DEV)
    a = mx_random(rng, (R, H), 0, 0)
    got = moe.moe_mx_product(moe.MxRows(*map(to_dev, a)), moe.MxRows(codes, scales), to_dev(base))
    want = oracle.mx_product(oracle.mx_values(*a, E2M1), oracle.mx_values(*some, E2M1), base)
    same_bits(bf16_bits(got[:, to_dev(picked)]), bits(want.astype(np.float32)))
    got[:, to_dev(picked)] = 0
    assert not got.any()


@pytest.mark.parametrize("counts,H,O", [c for c in PRODUCTS if c[2] % 2 == 0])
def test_product_gated(moe, counts, H, O):
    rng = np.random.default_rng(H * 3 + O)
    note("gated product", counts, H, O)
    got, exact, _ = product_case(moe, rng, counts, H, O, True, low=-3, high=-1, before=1, behind=2, gap=O % 5)
    gate, up = exact[:, : O // 2], exact[:, O // 2 :]
    with np.errstate(over="ignore"):
        want = gate / (1 + np.exp(-gate)) * up
    err = np.abs(oracle.bf16_bits_to_f32(got).astype(np.float64) - want)
    assert np.all(err <= np.abs(want) * (2.0**-8 + 2.0**-16) + 6e-37 * np.abs(up) + 1e-38)


@pytest.mark.parametrize("counts,H,O", [([70, 0, 9], 512, 96), ([4, 3], 1024, 64), ([600], 256, 272)])
def test_product_free_scales(moe, counts, H, O):
    rng = np.random.default_rng(H + 11)
    got, exact, magnitude = product_case(moe, rng, counts, H, O, False, low=-40, high=40)
    err = np.abs(oracle.bf16_bits_to_f32(got).astype(np.float64) - exact)
    assert np.all(err <= H * 2.0**-23 * magnitude + 2.0**-8 * np.abs(exact))


NAN_CASES = [(H, counts, O) for H in (160, 544, 1056, 2080) for counts in ([2, 3], [9, 14], [40, 30], [300, 100]) for O in (48, 3900)]
NAN_CASES += [(1056, [40, 44, 30, 46], 2400), (2080, [40, 44, 30, 46], 7200), (4128, [90, 60, 100, 30], 7200), (4128, [400, 380], 12801)]


@pytest.mark.parametrize("H,counts,O", NAN_CASES)
def test_product_nan_blocks(moe, H, counts, O):
    """A NaN scale of a row makes that row NaN and no other; one of a weight row its column of its group. The last
    block (H is no multiple of the tile's depth) as well as the first."""
    rng = np.random.default_rng(12)
    G, end = len(counts), H // 32 - 1
    base = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R = int(base[-1])
    a, w = mx_random(rng, (R, H), -1, 1), mx_random(rng, (G, O, H), -1, 1)
    a[1][1, end], a[1][R - 1, 0], w[1][1, 7, end], w[1][0, 0, 0] = 255, 255, 255, 255
    a[1][2 % R, end // 2], w[1][1, 9, end // 2 + 1] = 255, 255  # inside, where waves that share H hand over
    out = moe.moe_mx_product(moe.MxRows(*map(to_dev, a)), moe.MxRows(*map(to_dev, w)), to_dev(base))
    want = oracle.mx_product(oracle.mx_values(*a, E2M1), oracle.mx_values(*w, E2M1), base)
    same_bits(bf16_bits(out), bits(want.astype(np.float32)), "nan blocks")


def test_product_part_of_the_groups(moe):
    """A part of a layout's bases with the weights of those groups: rows of the other groups stay as they were."""
    rng = np.random.default_rng(13)
    counts, H, O = [9, 20, 0, 33, 4], 128, 40
    base = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    a, w = mx_random(rng, (int(base[-1]), H), -1, 1), mx_random(rng, (5, O, H), -1, 1)
    dev_base, out = to_dev(base), poison((int(base[-1]), O), torch.bfloat16)
    part = moe.MxRows(to_dev(w[0][1:4]), to_dev(w[1][1:4]))
    moe.moe_mx_product(moe.MxRows(*map(to_dev, a)), part, dev_base[1:5], out=out)
    want = oracle.mx_product(oracle.mx_values(*a, E2M1), oracle.mx_values(*w, E2M1), base)
    got = bf16_bits(out)
    same_bits(got[9:62], bits(want.astype(np.float32))[9:62])
    assert np.all(got[:9] == 0xABAB) and np.all(got[62:] == 0xABAB)


@pytest.mark.parametrize("base", [[0, 100, 200], [-5, 3, 6], [2, 2, 1 << 30], [6, 3, 0], [0, 0, 0]])
def test_product_bases_out_of_range(moe, base):
    """Bases outside [0, a_rows] are clamped: rows inside are computed, nothing else is touched."""
    rng = np.random.default_rng(14)
    R, H, O = 6, 64, 24
    a, w = mx_random(rng, (R, H), -1, 1), mx_random(rng, (2, O, H), -1, 1)
    out = poison((R, O), torch.bfloat16)
    moe.moe_mx_product(moe.MxRows(*map(to_dev, a)), moe.MxRows(*map(to_dev, w)), to_dev(np.array(base, dtype=np.int32)), out=out)
    clamped = np.clip(base, 0, R)
    want = oracle.mx_product(oracle.mx_values(*a, E2M1), oracle.mx_values(*w, E2M1), clamped)
    got = bf16_bits(out)
    has = ~np.isnan(want[:, 0])
    same_bits(got[has], bits(want[has].astype(np.float32)))
    assert np.all(got[~has] == 0xABAB)


@pytest.mark.parametrize("O", [24, 300])
def test_product_descending_bases(moe, O):
    """Bases that go up and down: nothing outside the rows is touched, and rows of ascending parts are computed."""
    rng = np.random.default_rng(16)
    R, H, G = 500, 544, 512
    base = np.zeros(G + 1, dtype=np.int32)
    base[1::2] = 1 << 30
    a, w = mx_random(rng, (R, H), -1, 1), mx_random(rng, (1, O, H), -1, 1)
    w = [np.broadcast_to(m, (G, *m.shape[1:])) for m in w]
    out = poison((R + 64, O), torch.bfloat16)
    moe.moe_mx_product(moe.MxRows(*map(to_dev, a)), moe.MxRows(*map(to_dev, w)), to_dev(base), out=out[:R])
    want = oracle.mx_product(oracle.mx_values(*a, E2M1), oracle.mx_values(w[0][:1], w[1][:1], E2M1), np.array([0, R]))
    got = bf16_bits(out)
    assert np.all(got[R:] == 0xABAB)
    same_bits(got[:R], bits(want.astype(np.float32)))  # every group has the same weights


def test_product_of_many_groups(moe):
    """The largest number of groups, most of them empty, and a misaligned scale pitch."""
    rng = np.random.default_rng(15)
    counts = np.zeros(512, dtype=int)
    counts[[0, 63, 64, 200, 511]] = [3, 1, 20, 0, 5]
    got, exact, _ = product_case(moe, rng, counts.tolist(), 96, 34, False)
    same_bits(got, bits(exact.astype(np.float32)))


# ---------------------------------------------------------------- as they are used


def test_refusals_on_the_device(moe):
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device=DEV)
    slot, w = torch.zeros((4, 2), dtype=torch.int32, device=DEV), torch.zeros((4, 2), device=DEV)
    q = moe.moe_mx_quantize(x, E2M1)
    base = torch.zeros(3, dtype=torch.int32, device=DEV)
    bad = [
        lambda: moe.moe_combine_backward(x[:3].contiguous(), x, slot, w),           # tokens
        lambda: moe.moe_combine_backward(x, x[:, :48], slot, w),                    # hidden size
        lambda: moe.moe_combine_backward(x, x.float(), slot, w),                    # type
        lambda: moe.moe_combine_backward(x, x.t().contiguous().t(), slot, w),       # columns apart
        lambda: moe.moe_combine_backward(x, x[:1].expand(4, 64), slot, w),          # rows on one another
        lambda: moe.moe_combine_backward(x, x, slot, w, d_expert_out=x),            # in place
        lambda: moe.moe_combine_backward(x, x, slot, w, d_expert_out=x[:2].clone()),
        lambda: moe.moe_combine_backward(x, x, slot, w, d_topk_weights=w[:2].clone()),
        lambda: moe.moe_combine_backward(x, x, slot, w.double()),
        lambda: moe.moe_combine_backward(x, x, slot, w[:, :1].contiguous()),
        lambda: moe.moe_dispatch_backward(x, slot.long()),
        lambda: moe.moe_dispatch_backward(x, slot, dx=x),
        lambda: moe.moe_combine_checkpoint(x, slot, w, checkpoint=q),               # E2M1 rows
        lambda: moe.moe_combine_backward_mx(x, q, slot, w),
        lambda: moe.moe_mx_quantize(x, 3),
        lambda: moe.moe_mx_quantize(x[:, :48], E2M1),                               # no whole blocks
        lambda: moe.moe_mx_quantize(x[:, 8:40], E2M1, out=q),
        lambda: moe.moe_mx_dequantize(q, E4M3),
        lambda: moe.moe_mx_product(q, q, base),                                     # weights [G, O, H]
        lambda: moe.moe_mx_product(q, moe.MxRows(q.codes[None], q.scales[None]), base),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
            pytest.fail(f"call {i} was not refused")
    g = moe.MxRows(torch.zeros((2, 3, 32), dtype=torch.uint8, device=DEV), torch.zeros((2, 3, 2), dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        moe.moe_mx_product(q, g, base, moe.MOE_MX_GATED)  # an odd O
    torch.cuda.synchronize()


def whole_step(moe, s):
    """Serving and training around one table, each call fed by the one before: every result."""
    lay = moe.moe_layout(s["idx"], s["E"], s["P"], s["C"])
    moe.moe_dispatch(s["x"], lay.slot_idx, s["win"])
    S, K, H = s["S"], s["K"], s["H"]
    up = moe.moe_unpack(s["win"], lay.expert_slot_base[s["E"]:], S, K, H, out=s["unpacked"])
    a = moe.moe_mx_quantize(up.expand_x, E2M1, num_rows=lay.expert_slot_base[s["E"]:], out=s["a"])
    mid = moe.moe_mx_product(a, s["w_up"], lay.expert_slot_base, moe.MOE_MX_GATED, out=s["mid"])
    b = moe.moe_mx_quantize(mid, E2M1, num_rows=lay.expert_slot_base[s["E"]:], out=s["b"])
    rows = moe.moe_mx_product(b, s["w_down"], lay.expert_slot_base, out=s["rows"])
    y, kept = moe.moe_combine_checkpoint(rows, lay.slot_idx, s["weights"], y=s["y"], checkpoint=s["kept"])
    d_rows, d_w = moe.moe_combine_backward_mx(s["dy"], kept, lay.slot_idx, s["weights"], s["d_rows"], s["d_w"])
    dx = moe.moe_dispatch_backward(d_rows, lay.slot_idx, dx=s["dx"])
    return dict(slot=lay.slot_idx, base=lay.expert_slot_base, expand=up.expand_x, a_codes=a.codes, a_scales=a.scales, mid=mid,
                b_codes=b.codes, b_scales=b.scales, rows=rows, y=y, codes=kept.codes, scales=kept.scales, d_rows=d_rows, d_w=d_w,
                dx=dx)


def step_state(moe, seed, S=96, K=4, E=16, P=4, H=256, inner=160):
    rng = np.random.default_rng(seed)
    R, s = S * K, dict(S=S, K=K, E=E, P=P, C=min(S, 8), H=H, inner=inner)
    s["idx"] = to_dev(random_tiny_routing(rng, S, K, E, p_mask=0.1))
    s["x"], s["dy"] = bf16_dev(spread_rows(rng, S, H)), bf16_dev(spread_rows(rng, S, H))
    s["weights"] = to_dev(rng.random((S, K), dtype=np.float32))
    s["win"] = poison((moe.moe_window_bytes(S, K, H),), torch.uint8)
    s["unpacked"] = moe.Unpacked(poison((R, H), torch.bfloat16), None, poison((R, 3), torch.int32))
    s["w_host"] = {}
    for name, (o, h) in dict(w_up=(2 * inner, H), w_down=(H, inner)).items():
        codes, scales = oracle.mx_quantize(bits(rng.standard_normal((E * o, h)) / np.sqrt(h)), E2M1)
        s["w_host"][name] = oracle.mx_values(codes, scales, E2M1).reshape(E, o, h)
        s[name] = moe.MxRows(to_dev(codes).view(E, o, h // 2), to_dev(scales).view(E, o, h // 32))
    mx = lambda h, c: moe.MxRows(poison((R, c), torch.uint8), poison((R, h // 32), torch.uint8))  # noqa: E731
    s["a"], s["b"], s["kept"] = mx(H, H // 2), mx(inner, inner // 2), mx(H, H)
    s["mid"], s["rows"], s["d_rows"] = (poison((R, h), torch.bfloat16) for h in (inner, H, H))
    s["y"], s["dx"], s["d_w"] = poison((S, H), torch.bfloat16), poison((S, H), torch.bfloat16), poison((S, K), torch.float32)
    return s


def host(r):
    torch.cuda.synchronize()
    return {k: (bf16_bits(v) if v.dtype == torch.bfloat16 else v.cpu().numpy()) for k, v in r.items()}


def equal_runs(a, b, what):
    for k in a:
        x, y = a[k], b[k]
        assert np.array_equal(x, y, equal_nan=x.dtype.kind == "f"), f"{what}: {k}"


def test_whole_step(moe):
    s = step_state(moe, 20)
    g = host(whole_step(moe, s))
    slot, base = g["slot"], g["base"]
    N = int(base[-1])
    x, dy, w = bf16_bits(s["x"]), bf16_bits(s["dy"]), s["weights"].cpu().numpy()
    codes, scales = oracle.mx_quantize(g["expand"][:N], E2M1)
    assert np.array_equal(g["a_codes"][:N], codes) and np.array_equal(g["a_scales"][:N], scales)
    av = oracle.mx_values(codes, scales, E2M1)
    sums = oracle.mx_product(av, s["w_host"]["w_up"], base)
    size = oracle.mx_product(np.abs(av), np.abs(s["w_host"]["w_up"]), base)
    I = s["inner"]
    # each sum is off by at most H * 2^-23 of its magnitudes; silu's slope is at most 1.1
    slack = s["H"] * 2.0**-23 * (1.1 * size[:, :I] * np.abs(sums[:, I:]) + np.abs(sums[:, :I]) * size[:, I:])
    want = sums[:, :I] / (1 + np.exp(-sums[:, :I])) * sums[:, I:]
    assert np.all(np.abs(oracle.bf16_bits_to_f32(g["mid"][:N]) - want) <= slack + np.abs(want) * (2.0**-8 + 2.0**-16) + 1e-30)
    codes, scales = oracle.mx_quantize(g["mid"][:N], E2M1)
    assert np.array_equal(g["b_codes"][:N], codes) and np.array_equal(g["b_scales"][:N], scales)
    bv = oracle.mx_values(codes, scales, E2M1)
    want = oracle.mx_product(bv, s["w_host"]["w_down"], base)
    size = oracle.mx_product(np.abs(bv), np.abs(s["w_host"]["w_down"]), base)
    assert np.all(np.abs(oracle.bf16_bits_to_f32(g["rows"][:N]) - want) <= I * 2.0**-23 * size + 2.0**-8 * np.abs(want))
    same_bits(g["y"], oracle.combine(g["rows"], slot, w), "y")
    codes, scales = oracle.mx_quantize(g["rows"][:N], E4M3)
    assert np.array_equal(g["codes"][:N], codes) and np.array_equal(g["scales"][:N], scales)
    d_rows, d_w, magnitude = oracle.combine_backward(dy, oracle.mx_values(codes, scales, E4M3), slot, w, np.full_like(g["d_rows"], 0xABAB))
    same_bits(g["d_rows"], d_rows, "d_rows")
    assert np.all(np.abs(g["d_w"] - d_w) <= weight_error_bound(magnitude))
    same_bits(g["dx"], oracle.dispatch_backward(g["d_rows"], slot), "dx")
    for k in ("expand", "mid", "rows", "d_rows"):
        assert np.all(g[k][N:] == 0xABAB), f"{k}: rows behind the last were written"
    for k in ("a_codes", "a_scales", "b_codes", "b_scales", "codes", "scales"):
        assert np.all(g[k][N:] == POISON), f"{k}: rows behind the last were written"


def test_repeated_and_on_another_stream(moe):
    ref = host(whole_step(moe, step_state(moe, 21)))
    equal_runs(ref, host(whole_step(moe, step_state(moe, 21))), "again")
    first, second = torch.cuda.Stream(), torch.cuda.Stream()
    a, b = step_state(moe, 21), step_state(moe, 22)
    other = host(whole_step(moe, step_state(moe, 22)))
    torch.cuda.synchronize()
    got = []
    for stream, s in ((first, a), (second, b)):  # both in flight at once
        with torch.cuda.stream(stream):
            got.append(whole_step(moe, s))
    equal_runs(ref, host(got[0]), "first stream")
    equal_runs(other, host(got[1]), "second stream")


def test_stream_argument(moe):
    """An explicit stream orders the call there, its new outputs included."""
    rng = np.random.default_rng(23)
    slot, rows = table(rng, 64, 4, 8, 0.1), spread_rows(rng, 256, 512)
    src, idx, w, dy = bf16_dev(rows), to_dev(slot), to_dev(rng.random((64, 4), dtype=np.float32)), bf16_dev(spread_rows(rng, 64, 512))
    torch.cuda.synchronize()
    want = host(dict(dx=moe.moe_dispatch_backward(src, idx), d_w=moe.moe_combine_backward(dy, src, idx, w)[1]))
    for stream in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        got = dict(dx=moe.moe_dispatch_backward(src, idx, stream=stream), d_w=moe.moe_combine_backward(dy, src, idx, w, stream=stream)[1])
        equal_runs(want, host(got), "stream")


def test_graph_replays(moe):
    """The whole step captured, and replayed on changed inputs with eager work in between."""
    s = step_state(moe, 24)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        whole_step(moe, s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = whole_step(moe, s)
    for seed in (25, 26, 27):
        fresh = step_state(moe, seed)
        for k in ("idx", "x", "dy", "weights"):
            s[k].copy_(fresh[k])
        for name in ("w_up", "w_down"):
            for mine, new in zip(s[name], fresh[name]):
                mine.copy_(new)
        for k in ("mid", "rows", "d_rows"):  # what an earlier replay left behind the last row
            s[k].view(torch.uint8).fill_(POISON)
        for k in ("a", "b", "kept"):
            for t in s[k]:
                t.fill_(POISON)
        s["unpacked"].expand_x.view(torch.uint8).fill_(POISON)
        graph.replay()
        equal_runs(host(whole_step(moe, fresh)), host(out), f"replay {seed}")
