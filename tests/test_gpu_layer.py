"""GPU tests of the rows in 8 bits, the INT8 product, the RMS norm and the balance loss against the oracle.

Exact wherever the result is one defined sequence of roundings: codes, scales and their values, the plain product, the
norm's sum, output and codes (1 / rms is rounded from 64 bits, and the fixed seeds have none at a border), counts.
Tolerances elsewhere, derived before the first run; u = 2^-24 is fp32's rounding, 2^-8 bf16's:

* the gated product of exact values g and v: silu(g) * v is right to 2^-14 for g >= -174 (0 may stand for it below),
  then half a step: (2^-8 + 2^-13) |result|, and 2^-133 for what underflows in bf16;
* the norm's dx = r (g - n m) + d: r, n, g, m are each off by at most 3 roundings, the three sums and products add
  four: 2^-21 (|r g| + |r n m| + |d|), then half a step of the result;
* d_weight: each term is off by 4 u and passes the additions of its part's rows (S / 256 of them, or one, in 256 to 1024 parts),
  of every 64th part (16 at most) and of those 64 sums: (S / 256 + 85) u of the sum of magnitudes;
* scores: exp's argument l - max is rounded (d u for a distance d), exp is good to 2 u, sum and quotient add 16 u:
  (24 + d) u of each score; the loss sums S of them in an order of at most 300 additions, so (324 + max d) u, where d is
  at most 88 for a score that is not 0 in fp32;
* d_logits = c s (g - dot): (64 + d) u (|g| + sum s |g|) c s, then half a step in bf16; scores below fp32's normal range
  count as up to 2^-120.
"""

import numpy as np
import pytest
import torch

import oracle
from workloads import f32_to_bf16_input

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
POISON = 0xAB
E4M3, INT8 = 1, 2
PLAIN, GATED = 0, 1
U = 2.0**-24


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


def values(t):
    return oracle.bf16_bits_to_f32(bf16_bits(t)) if t.dtype == torch.bfloat16 else t.cpu().numpy()


def bits(a):
    return f32_to_bf16_input(np.asarray(a, dtype=np.float32))


def poison(shape, dtype):
    t = torch.empty(shape, dtype=dtype, device=DEV)
    t.view(torch.uint8).fill_(POISON)
    return t


def poisoned(t):
    return bool((t.contiguous().view(torch.uint8) == POISON).all())


def strided(bits_rows, gap):
    """Device rows at a stride of H + gap values, with poison between them."""
    R, H = bits_rows.shape
    t = poison((R, H + gap), torch.bfloat16)
    t[:, :H] = bf16_dev(bits_rows)
    return t[:, :H]


def same_bits(got, want, what=""):
    g, w = oracle.bf16_bits_to_f32(got), oracle.bf16_bits_to_f32(want)
    bad = (got != want) & ~(np.isnan(g) & np.isnan(w))
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what} at {i}: {g[i]!r} for {w[i]!r}, {int(bad.sum())} of {bad.size} differ")


def same_rows8(got, codes, scales, what=""):
    g = got.codes.view(torch.uint8).cpu().numpy()
    if not np.array_equal(g, codes):
        i = tuple(np.argwhere(g != codes)[0])
        raise AssertionError(f"{what} code at {i}: {g[i]:#x} for {codes[i]:#x}, {int((g != codes).sum())} of {g.size} differ")
    assert np.array_equal(got.scales.cpu().numpy(), scales, equal_nan=True), what


def spread_rows(rng, R, H):
    return bits(rng.standard_normal((R, H)) * np.exp2(rng.integers(-6, 6, (R, 1))))


def near(got, want, tol, what=""):
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want, dtype=np.float64)
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what} at {i}: {got[i]!r} for {want[i]!r}, tolerance {np.broadcast_to(tol, got.shape)[i]:.3g}, "
                             f"{int(bad.sum())} of {bad.size} differ")


# ---------------------------------------------------------------- rows in 8 bits


@pytest.mark.parametrize("quant", [E4M3, INT8])
@pytest.mark.parametrize("R,H,gap", [(1, 16, 0), (3, 48, 8), (17, 2064, 0), (5, 7168, 512), (2, 16384, 0), (130, 80, 40)])
def test_rows_and_strides(moe, quant, R, H, gap):
    rng = np.random.default_rng(R * H + quant)
    rows = spread_rows(rng, R, H)
    rows[0] = 0
    if R > 2:
        rows[1, H // 2] = bits([np.nan])[0]
    codes, scales = oracle.row_quantize(rows, quant)
    n = R - 1 if R > 2 else R  # a device count below the buffer's rows: the last row stays as it was
    count = torch.tensor([n], dtype=torch.int32, device=DEV)
    out = moe.ScaledRows(poison((R, H), torch.uint8), poison(R, torch.float32))
    moe.moe_row_quantize(strided(rows, gap), quant, num_rows=count, out=out)
    same_rows8(moe.ScaledRows(out.codes[:n], out.scales[:n]), codes[:n], scales[:n])
    assert poisoned(out.codes[n:]) and poisoned(out.scales[n:])
    back = poison((R, H + gap), torch.bfloat16)
    moe.moe_row_dequantize(out, quant, num_rows=count, out=back[:, :H])
    same_bits(bf16_bits(back[:n, :H]), bits(oracle.row_values(codes, scales, quant))[:n])
    assert poisoned(back[n:]) and poisoned(back[:, H:])


@pytest.mark.parametrize("quant", [E4M3, INT8])
def test_rows_of_every_scale(moe, quant):
    """Every bf16 magnitude as a row's largest, with values down to 2^-12 of it, and infinities and NaNs."""
    rng = np.random.default_rng(quant)
    top = np.arange(0, 0x8000, 37, dtype=np.uint16)
    e = np.maximum((top >> 7).astype(np.int64)[:, None] - rng.integers(0, 13, (len(top), 32)), 0)
    rows = ((e << 7) | rng.integers(0, 128, e.shape)).astype(np.uint16)
    rows = np.minimum(rows, top[:, None]) | (rng.integers(0, 2, e.shape).astype(np.uint16) << 15)
    rows[:, 5] = top
    codes, scales = oracle.row_quantize(rows, quant)
    got = moe.moe_row_quantize(bf16_dev(rows), quant)
    same_rows8(got, codes, scales)
    same_bits(bf16_bits(moe.moe_row_dequantize(got, quant)), bits(oracle.row_values(codes, scales, quant)))


def test_rows_match_an_unpacked_dispatch(moe):
    """What the quantised dispatch leaves of the same rows, and counts below zero and above the rows."""
    rng = np.random.default_rng(6)
    S, H, E, K = 40, 272, 8, 2
    x = spread_rows(rng, S, H)
    idx = to_dev(rng.integers(0, E, (S, K)).astype(np.int32))
    for quant in (E4M3, INT8):
        lay = moe.moe_layout(idx, E, 1, 1)
        win = torch.empty(moe.moe_window_bytes(S, K, H), dtype=torch.uint8, device=DEV)
        moe.moe_dispatch(bf16_dev(x), lay.slot_idx, win, quant)
        un = moe.moe_unpack(win, lay.expert_slot_base[E:], S, K, H, quant)
        rows = moe.moe_row_quantize(bf16_dev(x), quant)
        at = lay.slot_idx.long()
        for k in range(K):
            assert torch.equal(un.expand_x[at[:, k]], rows.codes) and torch.equal(un.expand_scales[at[:, k]], rows.scales)
        for n, want in ((-3, 0), (1 << 30, S)):
            out = moe.ScaledRows(poison((S, H), torch.uint8), poison(S, torch.float32))
            moe.moe_row_quantize(bf16_dev(x), quant, num_rows=torch.tensor([n], dtype=torch.int32, device=DEV), out=out)
            assert torch.equal(out.codes[:want], rows.codes[:want]) and poisoned(out.codes[want:])


# ---------------------------------------------------------------- the product


def int8_rows(rng, R, H):
    a = rng.integers(-128, 128, (R, H)).astype(np.int8)
    return a, np.exp2(rng.uniform(-12, -6, R)).astype(np.float32)


def product_case(moe, rng, base, R, G, H, O, epilogue, gap=0, what="", a=None, a_scales=None):
    base = np.asarray(base, dtype=np.int32)
    assert len(base) == G + 1
    note(what, "R", R, "G", G, "H", H, "O", O, "epilogue", epilogue, "gap", gap)
    if a is None:
        a, a_scales = int8_rows(rng, R, H)
    w = rng.integers(-128, 128, (G, O, H)).astype(np.int8)
    w_scales = (np.exp2(rng.uniform(-5, 0, (G, O))) / (np.sqrt(H) * 4)).astype(np.float32)
    v, group = oracle.int8_product(a, a_scales, base, w, w_scales)
    width = O // 2 if epilogue == GATED else O
    buf = poison((R, width + gap), torch.bfloat16)
    got = moe.moe_scaled_product(moe.ScaledRows(to_dev(a).view(torch.uint8), to_dev(a_scales)), moe.ScaledRows(to_dev(w), to_dev(w_scales)),
                               to_dev(base), epilogue, out=buf[:, :width])
    inside = group >= 0
    if epilogue == PLAIN:
        same_bits(bf16_bits(got)[inside], bits(v)[inside], what)
    else:
        gate, up = v[:, :width].astype(np.float64), v[:, width:].astype(np.float64)
        with np.errstate(over="ignore"):
            want = gate / (1 + np.exp(-gate)) * up
        tol = (2.0**-8 + 2.0**-13) * np.abs(want) + 2.0**-133 + np.where(gate < -174, np.abs(want), 0)
        ok = inside[:, None] & np.isfinite(want)
        near(np.where(ok, values(got), 0), np.where(ok, want, 0), np.where(ok, tol, 0), what)
        assert np.array_equal(np.isnan(values(got))[inside], np.isnan(want)[inside]), what
    assert poisoned(buf[:, width:]) and poisoned(buf[to_dev(~inside)])


def spread_base(rng, R, G):
    return np.concatenate(([0], np.sort(rng.integers(0, R + 1, G - 1)), [R]))


@pytest.mark.parametrize("epilogue", [PLAIN, GATED])
@pytest.mark.parametrize("R,G,H,O", [(1, 1, 16, 2), (1, 3, 7168, 64), (5, 2, 48, 34), (16, 1, 64, 32), (17, 1, 80, 66), (33, 7, 1040, 200),
                                     (64, 4, 2048, 258), (100, 64, 112, 130), (129, 1, 272, 514), (300, 5, 528, 96), (257, 2, 3088, 1000),
                                     (1000, 3, 400, 770), (3, 2, 16384, 40)])
def test_product_sizes(moe, R, G, H, O, epilogue):
    rng = np.random.default_rng(R * 31 + H + O + epilogue)
    product_case(moe, rng, spread_base(rng, R, G), R, G, H, O, epilogue, what="sizes")


@pytest.mark.parametrize("epilogue", [PLAIN, GATED])
@pytest.mark.parametrize("R,G,H,O,gap", [(40, 2, 96, 25 * 2, 3), (70, 2, 160, 64, 8), (200, 3, 512, 300, 1), (530, 2, 1040, 520, 24), (2000, 4, 2064, 258, 2)])
def test_product_strides_and_odd_widths(moe, R, G, H, O, gap, epilogue):
    rng = np.random.default_rng(R + gap)
    product_case(moe, rng, spread_base(rng, R, G), R, G, H, O, epilogue, gap, "strides")
    if epilogue == PLAIN:
        product_case(moe, rng, spread_base(rng, R, G), R, G, H, O - 1, epilogue, gap, "odd width")


@pytest.mark.parametrize("R,G,H,O,epilogue,gap", [
    (12288, 1, 80, 1024, PLAIN, 0), (9000, 3, 144, 1606, PLAIN, 0), (5000, 4, 208, 4096, GATED, 8),           # tiles of 256 x 256
    (900, 3, 2064, 2100, PLAIN, 0), (512, 4, 2064, 4096, GATED, 0), (700, 1, 2096, 5000, PLAIN, 3),          # 128 x 128, one a unit
    (9000, 3, 144, 1030, PLAIN, 0), (2000, 16, 144, 2050, PLAIN, 0), (1500, 20, 1040, 2048, GATED, 4),       # 128 x 128 in turns
    (64, 20, 1552, 1800, PLAIN, 0), (300, 60, 1552, 1100, GATED, 6), (2500, 7, 3088, 600, PLAIN, 0),         # 64 x 64, 64 x 128, one each
    (1024, 32, 272, 4096, PLAIN, 0), (3001, 16, 1040, 1000, PLAIN, 0), (900, 40, 528, 4100, GATED, 0),       # 64 x 128 in turns
    (600, 2, 96, 2000, PLAIN, 0), (250, 3, 1088, 1100, GATED, 2), (40, 5, 2000, 2222, PLAIN, 0),            # smaller ones
    (600, 512, 64, 64, GATED, 0), (9000, 512, 96, 320, PLAIN, 0)])                                           # the most groups
def test_product_kernels(moe, R, G, H, O, epilogue, gap):
    """Every tile, with uneven groups, partly filled tiles, odd widths and ends of H inside a stage, and last rounds that leave
    workgroups without a tile of their own."""
    rng = np.random.default_rng(R + G)
    share = rng.dirichlet(np.full(G, 4.0))
    base = np.concatenate(([0], np.floor(np.cumsum(share) * R).astype(np.int64)))
    base[-1] = R
    product_case(moe, rng, base, R, G, H, O, epilogue, gap, "kernels")


@pytest.mark.parametrize("R,base", [(50, [3, 3, 20, 20, 44]), (50, [0, 0, 0, 0, 50]), (50, [50, 50, 50, 50, 50]), (50, [-7, 10, 5, 30, 99]),
                                    (50, [30, 10, 20, 45, 40]), (700, [100, 99, 400, 400, 650]), (700, [-5, 300, 200, 690, 800])])
@pytest.mark.parametrize("epilogue", [PLAIN, GATED])
def test_product_bases(moe, R, base, epilogue):
    """Rows before the first group and behind the last, empty groups, bases that descend or leave the rows."""
    product_case(moe, np.random.default_rng(len(base) + R), base, R, 4, 320, 140, epilogue, what=str(base))


@pytest.mark.parametrize("epilogue", [PLAIN, GATED])
def test_product_extremes(moe, epilogue):
    """The largest sums that there are (16384 * 128 * 128), scales near both ends of fp32, and scales of zero, an
    infinity and NaN, which stay in their own rows and outputs."""
    rng = np.random.default_rng(8)
    R, H = 40, 16384
    a = np.full((R, H), -128, dtype=np.int8)
    a[1::2] = 127
    scales = np.full(R, 2.0**-20, dtype=np.float32)
    scales[:8] = [0, np.inf, np.nan, 1e-45, 3e38, 2.0**-126, 1, 2.0**-60]
    with np.errstate(over="ignore", invalid="ignore"):
        product_case(moe, rng, [0, 25, 40], R, 2, H, 64, epilogue, what="extremes", a=a, a_scales=scales)
    w = np.full((1, 32, H), -128, dtype=np.int8)
    got = moe.moe_scaled_product(moe.ScaledRows(to_dev(a), to_dev(np.full(R, 2.0**-28, dtype=np.float32))),
                               moe.ScaledRows(to_dev(w), torch.ones(1, 32, device=DEV)), to_dev(np.array([0, R], dtype=np.int32)))
    assert np.all(values(got)[::2] == 1.0) and np.all(values(got)[1::2] == values(torch.tensor([-127 / 128], dtype=torch.bfloat16, device=DEV)))


def test_product_of_no_rows(moe):
    w = moe.ScaledRows(torch.zeros((2, 8, 32), dtype=torch.int8, device=DEV), torch.zeros((2, 8), device=DEV))
    a = moe.ScaledRows(torch.zeros((0, 32), dtype=torch.int8, device=DEV), torch.zeros(0, device=DEV))
    assert moe.moe_scaled_product(a, w, torch.zeros(3, dtype=torch.int32, device=DEV)).shape == (0, 8)


# ---------------------------------------------------------------- the norm


def norm_weight(rng, H, kind):
    w = (1 + 0.3 * rng.standard_normal(H)).astype(np.float32)
    if kind == "bf16":
        w = oracle.bf16_bits_to_f32(bits(w))
        return w, bf16_dev(bits(w))
    return w, to_dev(w)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("S,H,gap", [(1, 16, 0), (1, 7168, 0), (3, 48, 8), (70, 528, 0), (9, 2064, 16), (33, 4096, 0), (5, 8192, 8), (4, 8208, 0), (3, 16384, 0)])
def test_norm(moe, S, H, gap, residual, kind):
    rng = np.random.default_rng(S * H + residual)
    x, res = spread_rows(rng, S, H), spread_rows(rng, S, H) if residual else None
    x[0] = 0
    if residual and S > 1:
        res[0] = 0
    w, w_dev = norm_weight(rng, H, kind)
    eps = 1e-5
    s, y = oracle.rms_norm(x, res, w, eps)
    for quant in (0, INT8, E4M3):
        note("norm", S, H, gap, residual, kind, "quant", quant)
        total = poison((S, H + gap), torch.bfloat16)[:, :H] if residual else None
        out = poison((S, H), torch.bfloat16)
        got = moe.moe_rms_norm(strided(x, gap), w_dev, eps, residual=strided(res, gap) if residual else None, quant=quant, out=out, sum=total)
        same_bits(bf16_bits(got.sum), s, "sum")
        same_bits(bf16_bits(got.out), bits(y), "out")
        if quant:
            codes, scales = oracle.row_quantize_f32(y, quant)
            same_rows8(got.rows8, codes, scales, "codes")
            alone = moe.moe_rms_norm(bf16_dev(x), w_dev, eps, residual=bf16_dev(res) if residual else None, quant=quant)
            assert alone.out is None and torch.equal(alone.rows8.codes, got.rows8.codes) and torch.equal(alone.rows8.scales, got.rows8.scales)
        if gap and residual:
            assert poisoned(total.as_strided((S - 1, gap), (H + gap, 1), total.storage_offset() + H))


@pytest.mark.parametrize("place", ["x", "residual"])
@pytest.mark.parametrize("H,gap", [(1024, 0), (7168, 8)])
def test_norm_in_place(moe, place, H, gap):
    rng = np.random.default_rng(H)
    x, res = spread_rows(rng, 20, H), spread_rows(rng, 20, H)
    w, w_dev = norm_weight(rng, H, "bf16")
    s, y = oracle.rms_norm(x, res, w, 1e-6)
    a, b = strided(x, gap), strided(res, gap)
    got = moe.moe_rms_norm(a, w_dev, residual=b, sum=a if place == "x" else b)
    same_bits(bf16_bits(a if place == "x" else b), s)
    same_bits(bf16_bits(b if place == "x" else a), res if place == "x" else x)
    same_bits(bf16_bits(got.out), bits(y))
    both = strided(x, gap)  # x + x, over x
    s, y = oracle.rms_norm(x, x, w, 1e-6)
    got = moe.moe_rms_norm(both, w_dev, residual=both, sum=both)
    same_bits(bf16_bits(both), s)
    same_bits(bf16_bits(got.out), bits(y))


@pytest.mark.parametrize("quant", [0, INT8, E4M3])
def test_norm_of_extreme_rows(moe, quant):
    """Squares outside fp32, rows of subnormals, infinities and NaNs, which stay in their own rows."""
    rng = np.random.default_rng(quant)
    S, H = 24, 256
    v = rng.standard_normal((S, H))
    for i, scale in enumerate((1e30, 3e37, 1e-30, 1e-39, 1e-42, 1.0)):
        v[i] *= scale
    x = bits(v)
    x[6, 3], x[7, 9], x[8, 1], x[8, 2] = bits([np.inf])[0], bits([np.nan])[0], bits([np.inf])[0], bits([-np.inf])[0]
    w, w_dev = norm_weight(rng, H, "fp32")
    for eps in (1e-6, 1e-45):
        with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
            s, y = oracle.rms_norm(x, None, w, eps)
            codes, scales = oracle.row_quantize_f32(y, quant) if quant else (None, None)
        out = poison((S, H), torch.bfloat16)
        got = moe.moe_rms_norm(bf16_dev(x), w_dev, eps, quant=quant, out=out)
        same_bits(bf16_bits(out), bits(y), f"eps {eps}")
        if quant:
            same_rows8(got.rows8, codes, scales, f"eps {eps}")


def grad_case(moe, S, H, gap, residual, kind, seed, eps=1e-5, scale=1.0):
    rng = np.random.default_rng(seed)
    h, dy = spread_rows(rng, S, H), spread_rows(rng, S, H)
    if scale != 1.0:
        h = bits(oracle.bf16_bits_to_f32(h) * np.float32(scale))
    d_sum = spread_rows(rng, S, H) if residual else None
    w, w_dev = norm_weight(rng, H, kind)
    note("grad", S, H, gap, residual, kind)
    want_dx, want_dw = oracle.rms_norm_backward(dy, h, w, eps, d_sum)
    dx, dw = moe.moe_rms_norm_backward(strided(dy, gap), strided(h, gap), w_dev, eps, d_sum=strided(d_sum, gap) if residual else None)
    hv, g = oracle.bf16_bits_to_f32(h).astype(np.float64), oracle.bf16_bits_to_f32(dy).astype(np.float64) * w
    r = 1 / np.sqrt((hv * hv).mean(axis=1, keepdims=True) + eps)
    n = hv * r
    terms = np.abs(r * g) + np.abs(r * n * (g * n).mean(axis=1, keepdims=True)) + (np.abs(oracle.bf16_bits_to_f32(d_sum)) if residual else 0)
    near(values(dx), want_dx, 2.0**-21 * terms + 2.0**-8 * np.abs(want_dx) + 2.0**-133, "dx")
    near(values(dw), want_dw, (S / 256 + 85) * U * np.abs(oracle.bf16_bits_to_f32(dy) * n).sum(axis=0), "d_weight")
    return dx, dw


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("S,H,gap", [(1, 16, 0), (2, 7168, 8), (3, 48, 8), (70, 528, 0), (600, 272, 16), (1031, 1040, 0), (5, 8192, 8), (4, 8208, 0), (7, 16384, 0)])
def test_norm_gradient(moe, S, H, gap, residual, kind):
    grad_case(moe, S, H, gap, residual, kind, S * H + residual)


def test_norm_gradient_of_extreme_rows(moe):
    """Sums whose squares and products leave fp32's range."""
    grad_case(moe, 12, 512, 0, False, "fp32", 1, eps=1e-6, scale=1e25)
    grad_case(moe, 12, 512, 0, True, "bf16", 2, eps=1e-6, scale=1e-25)


def test_norm_gradient_of_no_rows(moe):
    w = torch.ones(64, device=DEV)
    empty = torch.zeros((0, 64), dtype=torch.bfloat16, device=DEV)
    dx, dw = moe.moe_rms_norm_backward(empty, empty, w, d_weight=poison(64, torch.float32))
    assert dx.shape == (0, 64) and not dw.any()
    assert moe.moe_rms_norm(empty, w).out.shape == (0, 64)
    assert moe.moe_rms_norm(empty, w, residual=empty, quant=INT8).rows8.scales.shape == (0,)


# ---------------------------------------------------------------- the balance loss


def routing(rng, S, E, K, form):
    idx = np.argsort(rng.random((S, E)), axis=1)[:, :K].astype(np.int32) if K <= E else rng.integers(0, E, (S, K)).astype(np.int32)
    if form == "padded":
        idx[rng.random((S, K)) < 0.3] = -1
        idx[S - S // 4 :] = -1
    elif form == "odd":  # ids out of range, the same id twice, one expert alone
        idx[rng.random((S, K)) < 0.2] = E
        idx[rng.random((S, K)) < 0.2] = -(2**31)
        idx[: S // 2] = min(1, E - 1)
    elif form == "none":
        idx[:] = -1
    return idx


def balance_case(moe, l, idx, score, kind, coef=0.01, gap=0):
    S, E = l.shape
    note("balance", S, E, idx.shape[1], "score", score, kind)
    if kind == "bf16":
        l = oracle.bf16_bits_to_f32(bits(l))
    wide = np.zeros((S, E + gap), dtype=np.float32)
    wide[:, :E] = l
    dev = (bf16_dev(bits(wide)) if kind == "bf16" else to_dev(wide))[:, :E]
    loss, counts, tokens, d = oracle.balance(l, idx, coef, score)
    got = moe.moe_balance_loss(dev, to_dev(idx), coef, score)
    assert np.array_equal(got.num_tokens_per_expert.cpu().numpy(), counts) and int(got.num_tokens) == tokens
    near(values(got.loss), [loss], 412 * U * abs(loss), "loss")
    d_loss = torch.full((1,), -1.5, device=DEV)
    out = poison((S, E), dev.dtype)
    moe.moe_balance_loss_backward(d_loss, dev, to_dev(idx), got.num_tokens_per_expert, got.num_tokens, coef, score, d_logits=out)
    valid = ((idx >= 0) & (idx < E)).any(axis=1)
    g = np.abs(counts - counts.sum() // E).astype(np.float64)
    s, far = np.zeros((S, E)), np.zeros((S, E))
    for row in np.flatnonzero(valid & (l.max(axis=1) > -np.inf)):
        u = l[row].astype(np.float64) if score == 0 else -np.logaddexp(0, -l[row].astype(np.float64))
        far[row] = np.minimum(u.max() - u, 88)
        s[row] = np.exp(u - u.max()) / np.exp(u - u.max()).sum()
    each = 1.5 * coef * E / max(1.0, float(counts.sum()) * tokens)
    tol = each * U * (64 + far) * s * (g + (s * g).sum(axis=1, keepdims=True)) + each * 2.0**-120 * (g.max() + 1) + 2.0**-148
    if kind == "bf16":
        tol = tol + 2.0**-8 * np.abs(1.5 * d) + 2.0**-133
    near(values(out), -1.5 * d, tol, "d_logits")
    return got


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("S,E,K,form", [(1, 1, 1, ""), (1, 2, 2, ""), (3, 7, 2, "odd"), (33, 64, 8, ""), (100, 65, 16, "padded"), (128, 16, 2, ""),
                                        (700, 128, 4, "odd"), (513, 200, 8, "padded"), (1500, 256, 8, "padded"), (90, 512, 6, ""), (64, 40, 3, "none")])
def test_balance(moe, S, E, K, form, score, kind):
    rng = np.random.default_rng(S + E + K + score)
    balance_case(moe, rng.standard_normal((S, E)).astype(np.float32) * 2, routing(rng, S, E, K, form), score, kind, gap=3 if S % 2 else 0)


@pytest.mark.parametrize("score", [0, 1])
def test_balance_masks(moe, score):
    """-inf for experts a token may not go to, rows of nothing else, of the lowest value alone and far from zero; NaN and
    infinities in the logits of padding."""
    rng = np.random.default_rng(score)
    S, E = 80, 96
    l = rng.standard_normal((S, E)).astype(np.float32)
    l[:, ::2] = -np.inf
    l[3], l[4] = -np.inf, np.finfo(np.float32).min
    l[5], l[6] = l[5] - 70, l[6] + 70
    l[7], l[8] = rng.standard_normal(E) * 40, np.finfo(np.float32).min
    l[8, 5] = 0.5
    idx = routing(rng, S, E, 4, "")
    idx[60:] = -1
    l[60:70], l[70:75], l[75:] = np.nan, np.inf, -np.inf
    got = balance_case(moe, l, idx, score, "fp32")
    assert torch.isfinite(got.loss).all()


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("value", [np.nan, np.inf])
def test_balance_of_logits_that_are_no_numbers(moe, score, value):
    """One NaN, alone among -inf or not, makes the loss NaN and its token's gradient at the NaN; +inf does with a softmax. Other
    tokens keep their gradients."""
    rng = np.random.default_rng(4)
    S, E = 40, 70
    l = rng.standard_normal((S, E)).astype(np.float32)
    idx = routing(rng, S, E, 3, "")
    want = oracle.balance(l, idx, 1.0, score)[3]
    l[7] = -np.inf
    l[7, 66] = l[30, 2] = value
    dev, table = to_dev(l), to_dev(idx)
    b = moe.moe_balance_loss(dev, table, 1.0, score)
    d = values(moe.moe_balance_loss_backward(torch.ones(1, device=DEV), dev, table, b.num_tokens_per_expert, b.num_tokens, 1.0, score))
    lost = bool(np.isnan(value)) or score == 0
    assert bool(torch.isnan(b.loss)) == lost and np.isnan(d[7, 66]) == np.isnan(d[30, 2]) == lost
    others = np.delete(np.arange(S), [7, 30])
    # (64 + far) U s (g + the mean of g) as in balance_case, with far below 20 for normal values and s below 1
    near(d[others], want[others], 168 * U * E / (3 * S * S) * np.bincount(idx.ravel(), minlength=E).max(), "d_logits")
    if lost:
        assert np.isnan(d[30]).all()


def test_balance_counts_are_the_layouts(moe):
    rng = np.random.default_rng(3)
    idx = to_dev(routing(rng, 600, 32, 4, "odd"))
    lay = moe.moe_layout(idx, 32, 4, 8)
    got = moe.moe_balance_loss(torch.randn((600, 32), device=DEV), idx, 0.1)
    assert torch.equal(got.num_tokens_per_expert, lay.num_tokens_per_expert)


def test_equal_counts_have_no_gradient(moe):
    idx = to_dev(np.arange(64, dtype=np.int32).reshape(32, 2) % 16)
    l = torch.randn((32, 16), device=DEV)
    b = moe.moe_balance_loss(l, idx, 1.0)
    assert not moe.moe_balance_loss_backward(torch.ones(1, device=DEV), l, idx, b.num_tokens_per_expert, b.num_tokens, 1.0).any()


@pytest.mark.parametrize("score", [0, 1])
def test_balance_gradient_is_the_losss_difference(moe, score):
    """(L(l + h v) - L(l - h v)) / 2h of the GPU's own losses against <d_logits, v>, as far as the oracle's own quotient is
    from its gradient, and twice the loss's tolerance over 2h."""
    rng = np.random.default_rng(score)
    S, E, K, h = 200, 24, 3, 0.25
    l, v = rng.standard_normal((S, E)).astype(np.float32), rng.standard_normal((S, E)).astype(np.float32)
    idx = routing(rng, S, E, K, "odd")
    up, down = (l + np.float32(h) * v).astype(np.float32), (l - np.float32(h) * v).astype(np.float32)
    d = oracle.balance(l, idx, 1.0, score)[3]
    losses = [oracle.balance(at, idx, 1.0, score)[0] for at in (up, down)]
    off = abs((losses[0] - losses[1]) / (2 * h) - (d * v).sum())
    b = moe.moe_balance_loss(to_dev(l), to_dev(idx), 1.0, score)
    got = moe.moe_balance_loss_backward(torch.ones(1, device=DEV), to_dev(l), to_dev(idx), b.num_tokens_per_expert, b.num_tokens, 1.0, score)
    quotient = (float(moe.moe_balance_loss(to_dev(up), to_dev(idx), 1.0, score).loss) - float(moe.moe_balance_loss(to_dev(down), to_dev(idx), 1.0, score).loss)) / (2 * h)
    inner = float((got.double().cpu().numpy() * v).sum())
    assert abs(quotient - inner) <= off + 2 * 412 * U * max(losses) / (2 * h) + 100 * U * float(np.abs(d * v).sum())


# ---------------------------------------------------------------- workspaces and ends of buffers


def inside(shape, dtype, front=64, back=64):
    """A poisoned device buffer and the part of it, 64 bytes aligned, that a call gets."""
    n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
    whole = poison(front + n + back, torch.uint8)
    return whole, whole[front : front + n].view(dtype).view(shape)


def untouched(whole, front=64, back=64):
    return poisoned(whole[:front]) and poisoned(whole[len(whole) - back :])


@pytest.mark.parametrize("S,H", [(1, 16), (2, 528), (300, 2064), (1531, 1040), (700, 16384)])
def test_norm_gradient_workspace(moe, S, H):
    """Exactly the bytes that are asked for, whatever they hold, and none around them or around the outputs."""
    rng = np.random.default_rng(S)
    dy, h, w = bf16_dev(spread_rows(rng, S, H)), bf16_dev(spread_rows(rng, S, H)), torch.ones(H, device=DEV)
    note("workspace", S, H)
    want = moe.moe_rms_norm_backward(dy, h, w)
    need = moe.moe_rms_norm_backward_workspace_bytes(S, H)
    ws, dx, dw = inside((need,), torch.uint8), inside((S, H), torch.bfloat16), inside((H,), torch.float32)
    for _ in range(2):  # the second time over the first one's parts
        moe.moe_rms_norm_backward(dy, h, w, dx=dx[1], d_weight=dw[1], workspace=ws[1])
        assert torch.equal(dx[1], want[0]) and torch.equal(dw[1], want[1])
    assert all(untouched(b[0]) for b in (ws, dx, dw))
    if need:
        with pytest.raises(ValueError):
            moe.moe_rms_norm_backward(dy, h, w, workspace=ws[1][:-16])


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("S,E,K", [(1, 1, 1), (128, 63, 3), (129, 5, 2), (700, 65, 4), (4001, 130, 8), (9000, 511, 6)])
def test_balance_workspace(moe, S, E, K, kind):
    rng = np.random.default_rng(S)
    idx, l = to_dev(routing(rng, S, E, K, "padded")), torch.randn((S, E), device=DEV).to(kind)
    note("balance workspace", S, E, K)
    want = moe.moe_balance_loss(l, idx, 0.1)
    one = torch.ones(1, device=DEV)
    want_d = moe.moe_balance_loss_backward(one, l, idx, want.num_tokens_per_expert, want.num_tokens, 0.1)
    need = moe.moe_balance_loss_workspace_bytes(S, E)
    bufs = [inside(s, d) for s, d in (((1,), torch.float32), ((E,), torch.int32), ((1,), torch.int32), ((S, E), kind), ((need,), torch.uint8))]
    loss, counts, tokens, d, ws = (b[1] for b in bufs)
    for _ in range(3):
        moe.moe_balance_loss(l, idx, 0.1, out=(loss, counts, tokens), workspace=ws)
        moe.moe_balance_loss_backward(one, l, idx, counts, tokens, 0.1, d_logits=d)
        assert torch.equal(loss, want.loss) and torch.equal(counts, want.num_tokens_per_expert) and torch.equal(tokens, want.num_tokens)
        assert torch.equal(d, want_d)
    assert all(untouched(b[0]) for b in bufs)
    if need:
        with pytest.raises(ValueError):
            moe.moe_balance_loss(l, idx, 0.1, workspace=ws[:-16])


@pytest.mark.parametrize("quant", [E4M3, INT8])
@pytest.mark.parametrize("S,H", [(1, 16), (3, 1040), (258, 7184)])
def test_dense_outputs_end_where_they_end(moe, S, H, quant):
    rng = np.random.default_rng(H)
    x, w = bf16_dev(spread_rows(rng, S, H)), torch.ones(H, device=DEV)
    want = moe.moe_rms_norm(x, w, residual=x, quant=quant, out=poison((S, H), torch.bfloat16))
    bufs = [inside(s, d) for s, d in (((S, H), torch.bfloat16), ((S, H), torch.bfloat16), ((S, H), torch.uint8), ((S,), torch.float32))]
    total, out, codes, scales = (b[1] for b in bufs)
    moe.moe_rms_norm(x, w, residual=x, quant=quant, sum=total, out=out, rows8=(codes, scales))
    assert torch.equal(total, want.sum) and torch.equal(out, want.out)
    assert torch.equal(codes, want.rows8.codes) and torch.equal(scales, want.rows8.scales)
    rows = moe.moe_row_quantize(x, quant)
    moe.moe_row_quantize(x, quant, out=(codes, scales))
    assert torch.equal(codes, rows.codes) and torch.equal(scales, rows.scales)
    back = moe.moe_row_dequantize(rows, quant)
    moe.moe_row_dequantize(rows, quant, out=total)
    assert torch.equal(total, back) and all(untouched(b[0]) for b in bufs)


def test_shared_workspace_in_order(moe):
    """Calls one behind the other may share a workspace, in a graph as well, and two graphs of one stream too."""
    rng = np.random.default_rng(5)
    S, E, K, H = 900, 200, 4, 528
    idx = [to_dev(routing(rng, S, E, K, f)) for f in ("", "padded")]
    l = [torch.randn((S, E), device=DEV) for _ in idx]
    dy, h, w = bf16_dev(spread_rows(rng, S, H)), bf16_dev(spread_rows(rng, S, H)), torch.ones(H, device=DEV)
    ws = poison(max(moe.moe_balance_loss_workspace_bytes(S, E), moe.moe_rms_norm_backward_workspace_bytes(S, H)), torch.uint8)

    def both():
        a = [moe.moe_balance_loss(x, t, 1.0, workspace=ws) for x, t in zip(l, idx)]
        return [v for b in a for v in b] + list(moe.moe_rms_norm_backward(dy, h, w, workspace=ws))

    want = both()
    alone = [v for x, t in zip(l, idx) for v in moe.moe_balance_loss(x, t, 1.0)] + list(moe.moe_rms_norm_backward(dy, h, w))
    assert all(torch.equal(a, b) for a, b in zip(want, alone))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = both()
        graphs.append((g, out))
    for _ in range(3):
        for g, out in graphs:
            ws.fill_(POISON)
            for t in l:
                t.normal_()
            eager = both()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, eager))


# ---------------------------------------------------------------- together, streams, graphs


class Step:
    """One pass through a layer in 8 bits, forward and the gradients around it, on buffers of its own."""

    def __init__(self, moe, seed, S=96, H=512, I=192, E=16, K=2):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.moe, self.S, self.H, self.E, self.K = moe, S, H, E, K
        rand = lambda *shape: torch.randn(shape, generator=g, device=DEV)  # noqa: E731
        self.x, self.residual, self.dy = (rand(S, H).to(torch.bfloat16) for _ in range(3))
        self.norm_weight = 1 + 0.1 * rand(H)
        self.router = rand(H, E) / H**0.5

        def weights(n, o, h):
            r = moe.moe_row_quantize((rand(n * o, h) / h**0.5).to(torch.bfloat16), INT8)
            return moe.ScaledRows(r.codes.view(n, o, h), r.scales.view(n, o))

        self.up, self.down = weights(E, 2 * I, H), weights(E, H, I)
        self.shared_up, self.shared_down = weights(1, 2 * I, H), weights(1, H, I)
        self.all_rows = torch.tensor([0, S], dtype=torch.int32, device=DEV)
        self.window = torch.zeros(moe.moe_window_bytes(S, K, H), dtype=torch.uint8, device=DEV)
        self.topk_idx, self.topk_weights = self.route()

    def route(self):
        normed = self.moe.moe_rms_norm(self.x, self.norm_weight, residual=self.residual)
        w, idx = torch.topk(torch.softmax(normed.out.float() @ self.router, dim=1), self.K, dim=1)
        return idx.to(torch.int32).contiguous(), w.contiguous()

    def __call__(self):
        moe, S, H, K, E = self.moe, self.S, self.H, self.K, self.E
        out = torch.empty((S, H), dtype=torch.bfloat16, device=DEV)
        normed = moe.moe_rms_norm(self.x, self.norm_weight, residual=self.residual, quant=INT8, out=out)
        logits = normed.out.float() @ self.router
        lay = moe.moe_layout(self.topk_idx, E, 1, 1)
        loss = moe.moe_balance_loss(logits, self.topk_idx, 0.01)
        moe.moe_dispatch(normed.out, lay.slot_idx, self.window, INT8)
        rows = lay.expert_slot_base[E:]
        un = moe.moe_unpack(self.window, rows, S, K, H, INT8)
        mid = moe.moe_scaled_product(moe.ScaledRows(un.expand_x, un.expand_scales), self.up, lay.expert_slot_base, GATED)
        mid8 = moe.moe_row_quantize(mid, INT8, num_rows=rows)
        expert_out = moe.moe_scaled_product(mid8, self.down, lay.expert_slot_base)
        y = moe.moe_combine(expert_out, lay.slot_idx, self.topk_weights)
        shared = moe.moe_scaled_product(normed.rows8, self.shared_up, self.all_rows, GATED)
        shared = moe.moe_scaled_product(moe.moe_row_quantize(shared, INT8), self.shared_down, self.all_rows)
        d_rows, d_weights = moe.moe_combine_backward(self.dy, expert_out, lay.slot_idx, self.topk_weights)
        d_out = moe.moe_dispatch_backward(d_rows, lay.slot_idx)
        d_logits = moe.moe_balance_loss_backward(torch.ones(1, device=DEV), logits, self.topk_idx, loss.num_tokens_per_expert, loss.num_tokens, 0.01)
        dx, d_norm = moe.moe_rms_norm_backward(d_out, normed.sum, self.norm_weight, d_sum=self.dy)
        return normed.sum, normed.out, normed.rows8.codes, loss.loss, loss.num_tokens_per_expert, y, shared, d_weights, d_logits, dx, d_norm


def equal(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)) for x, y in zip(a, b))


def test_whole_step(moe):
    """The chain against the oracle's; every later call reads what the earlier ones left on the GPU."""
    step = Step(moe, 1)
    total, out, codes, loss, counts, y, shared, d_weights, d_logits, dx, d_norm = step()
    s, yn = oracle.rms_norm(bf16_bits(step.x), bf16_bits(step.residual), step.norm_weight.cpu().numpy(), 1e-6)
    same_bits(bf16_bits(total), s)
    same_bits(bf16_bits(out), bits(yn))
    idx = step.topk_idx.cpu().numpy()
    lay = oracle.layout(idx, step.E, 1, 1)
    a, sa = oracle.row_quantize(bf16_bits(out), INT8)
    slots = lay["slot_idx"]
    token = np.empty(slots.size, dtype=np.int64)
    token[slots.ravel()] = np.arange(slots.size) // step.K

    def through(a, sa, base, up, down):
        up_w, up_s, down_w, down_s = (t.cpu().numpy() for t in (*up, *down))
        v, _ = oracle.int8_product(a.view(np.int8), sa, base, up_w.view(np.int8), up_s)
        half = v.shape[1] // 2
        gate = v[:, :half].astype(np.float64)
        mid = bits(gate / (1 + np.exp(-gate)) * v[:, half:])
        b, sb = oracle.row_quantize(mid, INT8)
        return oracle.int8_product(b.view(np.int8), sb, base, down_w.view(np.int8), down_s)[0]

    base = lay["expert_slot_base"]
    rows = through(a[token], sa[token], base, step.up, step.down)
    want = oracle.combine(bits(rows), slots, step.topk_weights.cpu().numpy())
    # the activation may round to the other bf16 value, and a code of the second product's rows then to its neighbour:
    # a step of the row's scale, 1/127 of its largest value, in few of its 192 places
    scale = np.abs(rows).max()
    assert np.abs(values(y) - oracle.bf16_bits_to_f32(want)).max() <= 0.02 * scale
    codes8, scales8 = oracle.row_quantize_f32(yn, INT8)
    assert np.array_equal(codes.cpu().numpy(), codes8)
    want = through(codes8, scales8, [0, step.S], step.shared_up, step.shared_down)
    assert np.abs(values(shared) - want).max() <= 0.02 * np.abs(want).max()
    assert np.array_equal(counts.cpu().numpy(), lay["num_tokens_per_expert"])


def test_repeat_runs_and_streams(moe):
    """The same bytes on every run, with two steps at once on two streams, and with calls that are given their stream."""
    a, b = Step(moe, 2), Step(moe, 3)
    want_a, want_b = a(), b()
    assert equal(a(), want_a)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            got_a = a()
        with torch.cuda.stream(t):
            got_b = b()
        torch.cuda.synchronize()
        assert equal(got_a, want_a) and equal(got_b, want_b)
    n = moe.moe_rms_norm(a.x, a.norm_weight, residual=a.residual, quant=INT8, stream=s)
    v = moe.moe_row_dequantize(n.rows8, INT8, stream=s)
    dx, dw = moe.moe_rms_norm_backward(a.dy, n.sum, a.norm_weight, stream=s)
    loss = moe.moe_balance_loss(torch.zeros((a.S, a.E), device=DEV), a.topk_idx, 1.0, stream=t)
    torch.cuda.synchronize()
    assert torch.equal(n.rows8.codes, want_a[2]) and v.shape == n.sum.shape and torch.isfinite(dx.float()).all() and abs(float(loss.loss) - 1) < 1e-5


def test_graph(moe):
    """Captured once and replayed with new inputs between eager runs, two graphs of steps that share nothing."""
    step, other = Step(moe, 4), Step(moe, 5)
    stream = torch.cuda.Stream()
    graphs = []
    for s in (step, other):
        with torch.cuda.stream(stream):
            s()
            stream.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                outs = s()
        graphs.append((g, outs))
    for k in range(3):
        for s, (g, outs) in zip((step, other), graphs):
            s.x.copy_(torch.randn(s.S, s.H, device=DEV).to(torch.bfloat16))
            want = s()
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert equal(outs, want), k


def test_most_rows(moe):
    """2^20 rows of 16 values: a wave a row, and as many parts of the gradient as there are."""
    rng = np.random.default_rng(11)
    R, H = 1 << 20, 16
    x = bits(rng.standard_normal((R, H)))
    at = np.concatenate((np.arange(64), rng.integers(0, R, 400), np.arange(R - 64, R)))
    w, w_dev = norm_weight(rng, H, "fp32")
    dev = bf16_dev(x)
    for quant in (INT8, E4M3):
        note("most rows", quant)
        got = moe.moe_row_quantize(dev, quant)
        codes, scales = oracle.row_quantize(x[at], quant)
        index = to_dev(at)
        same_rows8(moe.ScaledRows(got.codes[index], got.scales[index]), codes, scales)
        same_bits(bf16_bits(moe.moe_row_dequantize(got, quant)[index]), bits(oracle.row_values(codes, scales, quant)))
    n = moe.moe_rms_norm(dev, w_dev, 1e-6, residual=dev)
    s, y = oracle.rms_norm(x[at], x[at], w, 1e-6)
    same_bits(bf16_bits(n.sum[index]), s)
    same_bits(bf16_bits(n.out[index]), bits(y))
    dx, dw = moe.moe_rms_norm_backward(dev, n.sum, w_dev)
    total = bits(2 * oracle.bf16_bits_to_f32(x))
    want_dx, want_dw = oracle.rms_norm_backward(x, total, w, 1e-6)
    hv, g = oracle.bf16_bits_to_f32(total).astype(np.float64), oracle.bf16_bits_to_f32(x).astype(np.float64)
    r = 1 / np.sqrt((hv * hv).mean(axis=1, keepdims=True) + 1e-6)
    terms = np.abs(r * g * w) + np.abs(hv * r * r * (g * w * hv * r).mean(axis=1, keepdims=True))
    near(values(dx), want_dx, 2.0**-21 * terms + 2.0**-8 * np.abs(want_dx), "dx")
    # 1024 parts of 1024 rows, 64 sums of 16 parts: 1024 + 16 + 64 additions and 4 roundings of a term
    near(values(dw), want_dw, 1108 * U * np.abs(g * hv * r).sum(axis=0), "d_weight")


def test_most_tokens_and_experts(moe):
    """The largest router call: counts exactly, the loss and some tokens' gradients."""
    rng = np.random.default_rng(12)
    S, E, K = 65536, 512, 16
    idx = rng.integers(-1, E, (S, K)).astype(np.int32)
    l = rng.standard_normal((S, E)).astype(np.float32)
    dev = to_dev(l)
    note("most tokens")
    got = moe.moe_balance_loss(dev, to_dev(idx), 0.5)
    counts = np.bincount(idx[idx >= 0], minlength=E)
    live = (idx >= 0).any(axis=1)
    assert np.array_equal(got.num_tokens_per_expert.cpu().numpy(), counts) and int(got.num_tokens) == live.sum()
    p = np.exp(l.astype(np.float64) - l.max(axis=1, keepdims=True))
    p = np.where(live[:, None], p / p.sum(axis=1, keepdims=True), 0)
    each = 0.5 * E / (counts.sum() * float(live.sum()))
    loss = each * float((p.sum(axis=0) * counts).sum())
    near(values(got.loss), [loss], 412 * U * loss, "loss")  # 16 tokens a wave, 16 waves, 256 parts as 4, 4 and 16: 16 + 16 + 4 + 4 + 16 additions
    d = moe.moe_balance_loss_backward(torch.ones(1, device=DEV), dev, to_dev(idx), got.num_tokens_per_expert, got.num_tokens, 0.5)
    g = counts - counts.sum() // E
    at = np.concatenate((np.arange(100), np.arange(S - 100, S)))
    dot = (p * g).sum(axis=1, keepdims=True)
    tol = each * U * 96 * p * (np.abs(g) + (p * np.abs(g)).sum(axis=1, keepdims=True))
    near(values(d)[at], (each * p * (g - dot))[at], tol[at] + 2.0**-148, "d_logits")


def test_buffers_past_4_gib(moe):
    """Rows and weights whose offsets pass 32 bits: the last group's products and the last rows."""
    R, H = 300000, 16384  # 4.9 GB of codes
    a = torch.zeros((R, H), dtype=torch.int8, device=DEV)
    sa = torch.ones(R, device=DEV)
    rng = np.random.default_rng(9)
    tail, tail_scales = int8_rows(rng, 40, H)
    a[-40:], sa[-40:] = to_dev(tail), to_dev(tail_scales)
    w = torch.zeros((300, 1024, H), dtype=torch.int8, device=DEV)  # 5 GB
    ws = torch.ones((300, 1024), device=DEV)
    last = rng.integers(-128, 128, (1024, H)).astype(np.int8)
    w[-1], ws[-1] = to_dev(last), 2.0**-10
    base = torch.full((301,), R - 40, dtype=torch.int32, device=DEV)
    base[300] = R
    note("product past 4 GiB")
    got = moe.moe_scaled_product(moe.ScaledRows(a, sa), moe.ScaledRows(w, ws), base)
    v, _ = oracle.int8_product(tail, tail_scales, [0, 40], last[None], np.full((1, 1024), 2.0**-10, dtype=np.float32))
    same_bits(bf16_bits(got[-40:]), bits(v))
    del w, got
    note("rows past 4 GiB")
    back = moe.moe_row_dequantize(moe.ScaledRows(a.view(torch.uint8), sa), INT8)
    same_bits(bf16_bits(back[-40:]), bits(oracle.row_values(tail.view(np.uint8), tail_scales, INT8)))
    again = moe.moe_row_quantize(back, INT8)
    codes, scales = oracle.row_quantize(bf16_bits(back[-40:]), INT8)
    same_rows8(moe.ScaledRows(again.codes[-40:], again.scales[-40:]), codes, scales)
    del a, again
    note("norm past 4 GiB")
    weight = torch.ones(H, device=DEV)
    n = moe.moe_rms_norm(back, weight, residual=back, quant=E4M3)
    s, y = oracle.rms_norm(bf16_bits(back[-40:]), bf16_bits(back[-40:]), np.ones(H, dtype=np.float32), 1e-6)
    same_bits(bf16_bits(n.sum[-40:]), s)
    codes, scales = oracle.row_quantize_f32(y, E4M3)
    same_rows8(moe.ScaledRows(n.rows8.codes[-40:], n.rows8.scales[-40:]), codes, scales)
    dx, _ = moe.moe_rms_norm_backward(back, n.sum, weight)
    want, _ = oracle.rms_norm_backward(bf16_bits(back[-40:]), s, np.ones(H), 1e-6)
    # dy is half the sum, so g = n / 2r and its mean with n is 1 / 2r: both terms of dx are about r g = n / 2 and cancel, and the
    # error stays the terms', as derived above
    h = oracle.bf16_bits_to_f32(s).astype(np.float64)
    n = h / np.sqrt((h * h).mean(axis=1, keepdims=True) + 1e-6)
    near(values(dx[-40:]), want, 2.0**-21 * np.abs(n) + 2.0**-8 * np.abs(want), "dx")
