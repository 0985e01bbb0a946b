"""Refusals of the calls of the 8-bit layer: every argument check of the C ABI on the host, before any HIP call (fake,
never-dereferenced pointers), and the binding's own checks. Needs no GPU."""

import math

import pytest
import torch

import combine_moe_layout_02_amd as moe

A = 0x100000000  # a fake, aligned device address; buffers below are far enough apart not to overlap
GAP = 1 << 40
NULL = None
ARG, ALIGN, WINDOW, UNSUPPORTED = moe.MOE_ERR_ARG, moe.MOE_ERR_ALIGN, moe.MOE_ERR_WINDOW, moe.MOE_ERR_UNSUPPORTED
E4M3, INT8 = moe.MOE_QUANT_FP8_E4M3_DYN, moe.MOE_QUANT_INT8_DYN


def at(i):
    return A + i * GAP


CALLS = {
    "moe_row_quantize": dict(rows=at(1), stride=2048, num=NULL, n=64, H=1024, quant=INT8, codes=at(5), scales=at(6), stream=None),
    "moe_row_dequantize": dict(codes=at(5), scales=at(6), num=NULL, n=64, H=1024, quant=E4M3, rows=at(1), stride=2048, stream=None),
    "moe_scaled_product": dict(ac=at(0), asc=at(1), n=64, base=at(2), G=8, wc=at(3), ws=at(4), O=100, H=1024, epilogue=0, out=at(5),
                             stride=200, stream=None),
    "moe_rms_norm": dict(x=at(0), stride=2048, res=at(1), res_stride=2048, w=at(2), kind=2, eps=1e-6, n=64, H=1024, quant=INT8, sum=at(3),
                         sum_stride=2048, out=at(4), codes=at(5), scales=at(6), stream=None),
    "moe_rms_norm_backward": dict(dy=at(0), stride=2048, sum=at(1), sum_stride=2048, w=at(2), kind=1, eps=1e-6, ds=at(3), ds_stride=2048,
                                  n=64, H=1024, dx=at(4), dw=at(5), ws=at(6), bytes=1 << 30, stream=None),
    "moe_balance_loss": dict(logits=at(0), stride=256, kind=2, topk=at(1), S=500, K=4, E=64, score=0, coef=0.01, loss=at(2), counts=at(3),
                             tokens=at(4), ws=at(5), bytes=1 << 30, stream=None),
    "moe_balance_loss_backward": dict(dl=at(6), logits=at(0), stride=256, kind=2, topk=at(1), counts=at(3), tokens=at(4), S=500, K=4, E=64,
                                      score=1, coef=0.01, d=at(5), stream=None),
}
OPTIONAL = {("moe_row_quantize", "num"), ("moe_row_dequantize", "num"), ("moe_rms_norm", "out"), ("moe_rms_norm_backward", "ds")}
POINTERS = {"rows", "codes", "scales", "ac", "asc", "base", "wc", "ws", "out", "x", "res", "w", "sum", "dy", "ds", "dx", "dw", "logits", "topk",
            "loss", "counts", "tokens", "dl", "d"}


def call(name, **kw):
    args = dict(CALLS[name])
    assert set(kw) <= set(args)
    args.update(kw)
    return getattr(moe._lib, name)(*args.values())


@pytest.mark.parametrize("name,arg", [(n, a) for n, args in CALLS.items() for a in args if a in POINTERS and (n, a) not in OPTIONAL])
def test_null_pointers(name, arg):
    assert call(name, **{arg: NULL}) == ARG


@pytest.mark.parametrize("name", [n for n in CALLS if "H" in CALLS[n]])
@pytest.mark.parametrize("H,err", [(0, ARG), (8, ARG), (1000, UNSUPPORTED), (16400, ARG), (-16, ARG)])
def test_hidden(name, H, err):
    assert call(name, H=H) == err


@pytest.mark.parametrize("name", [n for n in CALLS if "n" in CALLS[n]])
def test_row_counts(name):
    assert call(name, n=-1) == ARG
    assert call(name, n=(1 << 20) + 1) == ARG
    assert call(name, n=1 << 62) == ARG


@pytest.mark.parametrize("name", [n for n in CALLS if "n" in CALLS[n] and n != "moe_rms_norm_backward"])
def test_no_rows_enqueue_nothing(name):
    assert call(name, n=0) == moe.MOE_OK


@pytest.mark.parametrize("name", ["moe_balance_loss", "moe_balance_loss_backward"])
@pytest.mark.parametrize("kw,err", [
    (dict(S=0), ARG), (dict(S=-1), ARG), (dict(S=65537), UNSUPPORTED), (dict(K=0), ARG), (dict(K=17), ARG), (dict(E=0), ARG),
    (dict(E=513, stride=4096), ARG), (dict(kind=0), ARG), (dict(kind=3), ARG), (dict(score=2), ARG), (dict(score=-1), ARG),
    (dict(coef=math.nan), ARG), (dict(coef=math.inf), ARG), (dict(stride=252), ARG), (dict(stride=258), ALIGN),
    (dict(stride=1 << 61), ARG), (dict(logits=at(0) + 2), ALIGN), (dict(topk=at(1) + 2), ALIGN), (dict(counts=at(3) + 1), ALIGN),
    (dict(tokens=at(4) + 2), ALIGN),
])
def test_router_arguments(name, kw, err):
    assert call(name, **kw) == err


@pytest.mark.parametrize("name,kw,err", [
    ("moe_row_quantize", dict(quant=0), ARG),
    ("moe_row_quantize", dict(quant=3), ARG),
    ("moe_row_quantize", dict(stride=2032), ARG),
    ("moe_row_quantize", dict(stride=2056), ALIGN),
    ("moe_row_quantize", dict(rows=at(1) + 8), ALIGN),
    ("moe_row_quantize", dict(codes=at(5) + 8), ALIGN),
    ("moe_row_quantize", dict(scales=at(6) + 2), ALIGN),
    ("moe_row_quantize", dict(num=at(7) + 2), ALIGN),
    ("moe_row_quantize", dict(codes=at(1)), ARG),
    ("moe_row_quantize", dict(scales=at(5) + 64 * 1024 - 4), ARG),
    ("moe_row_quantize", dict(num=at(6) + 252), ARG),
    ("moe_row_dequantize", dict(quant=0), ARG),
    ("moe_row_dequantize", dict(rows=at(5) + 63 * 1024), ARG),
    ("moe_row_dequantize", dict(rows=at(6)), ARG),
    ("moe_row_dequantize", dict(rows=at(1) + 8), ALIGN),
    ("moe_row_dequantize", dict(stride=2032), ARG),
    ("moe_scaled_product", dict(G=0), ARG),
    ("moe_scaled_product", dict(G=513), ARG),
    ("moe_scaled_product", dict(O=0), ARG),
    ("moe_scaled_product", dict(O=65537, stride=200000), ARG),
    ("moe_scaled_product", dict(epilogue=2), ARG),
    ("moe_scaled_product", dict(epilogue=1, O=101), UNSUPPORTED),
    ("moe_scaled_product", dict(stride=198), ARG),
    ("moe_scaled_product", dict(stride=201), ALIGN),
    ("moe_scaled_product", dict(stride=1 << 62), ARG),
    ("moe_scaled_product", dict(out=at(5) + 1), ALIGN),
    ("moe_scaled_product", dict(ac=at(0) + 8), ALIGN),
    ("moe_scaled_product", dict(asc=at(1) + 2), ALIGN),
    ("moe_scaled_product", dict(wc=at(3) + 8), ALIGN),
    ("moe_scaled_product", dict(ws=at(4) + 1), ALIGN),
    ("moe_scaled_product", dict(base=at(2) + 2), ALIGN),
    ("moe_scaled_product", dict(out=at(0)), ARG),
    ("moe_scaled_product", dict(out=at(1) + 252), ARG),
    ("moe_scaled_product", dict(out=at(2) + 32), ARG),
    ("moe_scaled_product", dict(out=at(3) + 8 * 100 * 1024 - 2), ARG),
    ("moe_scaled_product", dict(out=at(4) + 8 * 100 * 4 - 2), ARG),
    ("moe_rms_norm", dict(kind=0), ARG),
    ("moe_rms_norm", dict(kind=3), ARG),
    ("moe_rms_norm", dict(quant=3), ARG),
    ("moe_rms_norm", dict(quant=0), ARG),                            # codes without a type
    ("moe_rms_norm", dict(quant=0, codes=NULL, scales=NULL, out=NULL), ARG),
    ("moe_rms_norm", dict(eps=0.0), ARG),
    ("moe_rms_norm", dict(eps=-1e-6), ARG),
    ("moe_rms_norm", dict(eps=math.nan), ARG),
    ("moe_rms_norm", dict(eps=math.inf), ARG),
    ("moe_rms_norm", dict(res=NULL), ARG),                           # a sum without a residual
    ("moe_rms_norm", dict(stride=2032), ARG),
    ("moe_rms_norm", dict(res_stride=2056), ALIGN),
    ("moe_rms_norm", dict(sum_stride=2032), ARG),
    ("moe_rms_norm", dict(x=at(0) + 8), ALIGN),
    ("moe_rms_norm", dict(w=at(2) + 8), ALIGN),
    ("moe_rms_norm", dict(out=at(4) + 8), ALIGN),
    ("moe_rms_norm", dict(codes=at(5) + 8), ALIGN),
    ("moe_rms_norm", dict(sum=at(0), sum_stride=4096), ARG),         # over x, but not row on row
    ("moe_rms_norm", dict(sum=at(0) + 2048), ARG),
    ("moe_rms_norm", dict(sum=at(1) + 16), ARG),
    ("moe_rms_norm", dict(sum=at(2)), ARG),
    ("moe_rms_norm", dict(sum=at(0), res=at(0) + 2048), ARG),        # over x, and over other rows of residual
    ("moe_rms_norm", dict(out=at(0)), ARG),
    ("moe_rms_norm", dict(out=at(3) + 63 * 2048), ARG),
    ("moe_rms_norm", dict(out=at(1)), ARG),
    ("moe_rms_norm", dict(codes=at(4) + 64 * 2048 - 16), ARG),
    ("moe_rms_norm", dict(scales=at(2) + 4092), ARG),
    ("moe_rms_norm_backward", dict(kind=4), ARG),
    ("moe_rms_norm_backward", dict(eps=0.0), ARG),
    ("moe_rms_norm_backward", dict(stride=2032), ARG),
    ("moe_rms_norm_backward", dict(sum_stride=2056), ALIGN),
    ("moe_rms_norm_backward", dict(ds_stride=2032), ARG),
    ("moe_rms_norm_backward", dict(dx=at(4) + 8), ALIGN),
    ("moe_rms_norm_backward", dict(dw=at(5) + 4), ALIGN),
    ("moe_rms_norm_backward", dict(ws=at(6) + 8), ALIGN),
    ("moe_rms_norm_backward", dict(bytes=-1), WINDOW),
    ("moe_rms_norm_backward", dict(dx=at(0)), ARG),
    ("moe_rms_norm_backward", dict(dx=at(3)), ARG),
    ("moe_rms_norm_backward", dict(dw=at(2)), ARG),
    ("moe_rms_norm_backward", dict(dw=at(4) + 64 * 2048 - 16), ARG),
    ("moe_rms_norm_backward", dict(ws=at(1)), ARG),
    ("moe_rms_norm_backward", dict(ws=at(5) + 4080), ARG),
    ("moe_balance_loss", dict(bytes=-1), WINDOW),
    ("moe_balance_loss", dict(loss=at(2) + 2), ALIGN),
    ("moe_balance_loss", dict(ws=at(5) + 4), ALIGN),
    ("moe_balance_loss", dict(loss=at(3) + 252), ARG),
    ("moe_balance_loss", dict(counts=at(0) + 499 * 256 + 252), ARG),
    ("moe_balance_loss", dict(tokens=at(1) + 500 * 16 - 4), ARG),
    ("moe_balance_loss", dict(ws=at(0)), ARG),
    ("moe_balance_loss_backward", dict(dl=at(6) + 2), ALIGN),
    ("moe_balance_loss_backward", dict(d=at(5) + 2), ALIGN),
    ("moe_balance_loss_backward", dict(d=at(0)), ARG),
    ("moe_balance_loss_backward", dict(d=at(6) - 500 * 256 + 4), ARG),
    ("moe_balance_loss_backward", dict(d=at(3) + 252), ARG),
])
def test_refusals(name, kw, err):
    assert call(name, **kw) == err


def test_workspaces():
    for n, H in ((1, 16), (64, 1024), (4096, 7168), (1 << 20, 16384)):
        need = moe.moe_rms_norm_backward_workspace_bytes(n, H)
        assert need >= 0 and need % 16 == 0
        if need:
            assert call("moe_rms_norm_backward", n=n, H=H, stride=2 * H, sum_stride=2 * H, ds_stride=2 * H, bytes=need - 1) == WINDOW
    assert moe.moe_rms_norm_backward_workspace_bytes(0, 1024) >= 0
    for S, E in ((1, 1), (500, 64), (65536, 512)):
        need = moe.moe_balance_loss_workspace_bytes(S, E)
        assert need >= 0
        if need:
            assert call("moe_balance_loss", S=S, E=E, stride=4 * E, bytes=need - 1) == WINDOW
    for bad in (lambda: moe.moe_rms_norm_backward_workspace_bytes(-1, 1024), lambda: moe.moe_rms_norm_backward_workspace_bytes(4, 1000),
                lambda: moe.moe_balance_loss_workspace_bytes(0, 8), lambda: moe.moe_balance_loss_workspace_bytes(8, 513)):
        with pytest.raises(ValueError):
            bad()


def test_binding_refuses_host_tensors():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    w, idx, one = torch.zeros(64), torch.zeros((4, 2), dtype=torch.int32), torch.zeros(1)
    rows8 = moe.ScaledRows(torch.zeros((4, 64), dtype=torch.int8), torch.zeros(4))
    for fn in (lambda: moe.moe_row_quantize(x, INT8), lambda: moe.moe_row_dequantize(rows8, INT8),
               lambda: moe.moe_scaled_product(rows8, rows8, idx), lambda: moe.moe_rms_norm(x, w),
               lambda: moe.moe_rms_norm_backward(x, x, w), lambda: moe.moe_balance_loss(torch.zeros((4, 8)), idx, 0.1),
               lambda: moe.moe_balance_loss_backward(one, torch.zeros((4, 8)), idx, idx, idx, 0.1)):
        with pytest.raises(ValueError, match="device tensor"):
            fn()


def test_binding_refuses_other_types():
    for fn in (lambda: moe.moe_row_quantize([1.0], INT8), lambda: moe.moe_rms_norm(None, None),
               lambda: moe.moe_scaled_product(moe.ScaledRows([1], [2]), None, None)):
        with pytest.raises(TypeError, match="torch.Tensor"):
            fn()
