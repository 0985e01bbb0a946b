"""Refusals of the gradient, MX and product calls: every argument check of the C ABI on the host, before any HIP
call (fake, never-dereferenced pointers), and the binding's own checks. Needs no GPU."""

import pytest
import torch

import combine_moe_layout_02_amd as moe

A = 0x100000000  # a fake, aligned device address; buffers below are far enough apart not to overlap
GAP = 1 << 40
NULL = None
ARG, ALIGN, UNSUPPORTED = moe.MOE_ERR_ARG, moe.MOE_ERR_ALIGN, moe.MOE_ERR_UNSUPPORTED


def at(i):
    return A + i * GAP


CALLS = {
    "moe_combine_backward": dict(dy=at(0), rows=at(1), stride=2048, n=64, slot=at(2), w=at(3), S=16, H=1024, K=4, d=at(4),
                                 d_stride=2048, dw=at(5), stream=None),
    "moe_combine_backward_mx": dict(dy=at(0), codes=at(1), scales=at(6), n=64, slot=at(2), w=at(3), S=16, H=1024, K=4, d=at(4),
                                    d_stride=2048, dw=at(5), stream=None),
    "moe_dispatch_backward": dict(rows=at(1), stride=2048, n=64, slot=at(2), S=16, H=1024, K=4, dx=at(4), stream=None),
    "moe_combine_checkpoint": dict(rows=at(1), stride=2048, n=64, slot=at(2), w=at(3), S=16, H=1024, K=4, y=at(4), codes=at(5),
                                   scales=at(6), stream=None),
    "moe_mx_quantize": dict(rows=at(1), stride=2048, num=NULL, n=64, H=1024, format=1, codes=at(5), scales=at(6), stream=None),
    "moe_mx_dequantize": dict(codes=at(5), scales=at(6), num=NULL, n=64, H=1024, format=2, rows=at(1), stride=2048, stream=None),
    "moe_mx_product": dict(ac=at(0), asc=at(1), n=64, base=at(2), G=8, wc=at(3), ws=at(4), O=100, H=1024, epilogue=0, out=at(5),
                           stride=200, stream=None),
}
POINTERS = {"dy", "rows", "slot", "w", "d", "dw", "codes", "scales", "dx", "y", "ac", "asc", "base", "wc", "ws", "out"}


def call(name, **kw):
    args = dict(CALLS[name])
    assert set(kw) <= set(args)
    args.update(kw)
    return getattr(moe._lib, name)(*args.values())


@pytest.mark.parametrize("name,arg", [(n, a) for n, args in CALLS.items() for a in args if a in POINTERS])
def test_null_pointers(name, arg):
    assert call(name, **{arg: NULL}) == ARG


TABLE = [n for n in CALLS if "S" in CALLS[n]]


@pytest.mark.parametrize("name", TABLE)
@pytest.mark.parametrize("kw,err", [
    (dict(S=0), ARG), (dict(S=-1), ARG), (dict(S=65537), UNSUPPORTED), (dict(K=0), ARG), (dict(K=17), ARG),
    (dict(n=-1), ARG), (dict(slot=at(2) + 2), ALIGN),
])
def test_table_arguments(name, kw, err):
    assert call(name, **kw) == err


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("H,err", [(0, ARG), (8, ARG), (1000, UNSUPPORTED), (16400, ARG)])
def test_hidden(name, H, err):
    assert call(name, H=H) == err


@pytest.mark.parametrize("name", [n for n in CALLS if n not in ("moe_combine_backward", "moe_dispatch_backward")])
def test_mx_hidden_is_whole_blocks(name):
    assert call(name, H=1008) == UNSUPPORTED


@pytest.mark.parametrize("name,kw,err", [
    ("moe_combine_backward", dict(stride=2032), ARG),
    ("moe_combine_backward", dict(stride=2056), ALIGN),
    ("moe_combine_backward", dict(d_stride=2032), ARG),
    ("moe_combine_backward", dict(d_stride=2056), ALIGN),
    ("moe_combine_backward", dict(rows=at(1) + 8), ALIGN),
    ("moe_combine_backward", dict(dy=at(0) + 8), ALIGN),
    ("moe_combine_backward", dict(d=at(4) + 8), ALIGN),
    ("moe_combine_backward", dict(dw=at(5) + 2), ALIGN),
    ("moe_combine_backward", dict(w=at(3) + 1), ALIGN),
    ("moe_combine_backward", dict(n=1 << 60), ARG),                 # rows * stride wraps
    ("moe_combine_backward", dict(stride=1 << 58), ARG),
    ("moe_combine_backward", dict(d=at(1)), ARG),                   # in place
    ("moe_combine_backward", dict(d=at(1) + 63 * 2048 + 2032), ARG),
    ("moe_combine_backward", dict(d=at(0) - 63 * 2048 - 2032), ARG),
    ("moe_combine_backward", dict(dw=at(4) + 4096), ARG),
    ("moe_combine_backward", dict(dw=at(3)), ARG),
    ("moe_combine_backward_mx", dict(d_stride=2056), ALIGN),
    ("moe_combine_backward_mx", dict(codes=at(1) + 8), ALIGN),
    ("moe_combine_backward_mx", dict(n=1 << 60), ARG),
    ("moe_combine_backward_mx", dict(d=at(1) + 1024 * 63), ARG),
    ("moe_combine_backward_mx", dict(d=at(6)), ARG),
    ("moe_dispatch_backward", dict(stride=2032), ARG),
    ("moe_dispatch_backward", dict(stride=2056), ALIGN),
    ("moe_dispatch_backward", dict(dx=at(4) + 8), ALIGN),
    ("moe_dispatch_backward", dict(dx=at(1) + 2048), ARG),
    ("moe_combine_checkpoint", dict(y=at(4) + 8), ALIGN),
    ("moe_combine_checkpoint", dict(codes=at(5) + 8), ALIGN),
    ("moe_combine_checkpoint", dict(codes=at(1)), ARG),
    ("moe_combine_checkpoint", dict(scales=at(5) + 1024 * 64 - 1), ARG),
    ("moe_combine_checkpoint", dict(scales=at(4)), ARG),
    ("moe_mx_quantize", dict(format=0), ARG),
    ("moe_mx_quantize", dict(format=3), ARG),
    ("moe_mx_quantize", dict(n=1048577), ARG),
    ("moe_mx_quantize", dict(n=-1), ARG),
    ("moe_mx_quantize", dict(stride=2040), ARG),
    ("moe_mx_quantize", dict(stride=2056), ALIGN),
    ("moe_mx_quantize", dict(codes=at(5) + 4), ALIGN),
    ("moe_mx_quantize", dict(num=at(7) + 2), ALIGN),
    ("moe_mx_quantize", dict(codes=at(1)), ARG),
    ("moe_mx_quantize", dict(num=at(6)), ARG),
    ("moe_mx_dequantize", dict(format=3), ARG),
    ("moe_mx_dequantize", dict(rows=at(1) + 8), ALIGN),
    ("moe_mx_dequantize", dict(stride=2032), ARG),
    ("moe_mx_dequantize", dict(rows=at(5)), ARG),
    ("moe_mx_product", dict(n=-1), ARG),
    ("moe_mx_product", dict(n=1048577), ARG),
    ("moe_mx_product", dict(G=0), ARG),
    ("moe_mx_product", dict(G=513), ARG),
    ("moe_mx_product", dict(O=0), ARG),
    ("moe_mx_product", dict(O=65537), ARG),
    ("moe_mx_product", dict(epilogue=2), ARG),
    ("moe_mx_product", dict(epilogue=-1), ARG),
    ("moe_mx_product", dict(epilogue=1, O=101), UNSUPPORTED),
    ("moe_mx_product", dict(stride=198), ARG),
    ("moe_mx_product", dict(stride=201), ALIGN),
    ("moe_mx_product", dict(stride=1 << 62), ARG),
    ("moe_mx_product", dict(out=at(5) + 1), ALIGN),
    ("moe_mx_product", dict(ac=at(0) + 8), ALIGN),
    ("moe_mx_product", dict(wc=at(3) + 8), ALIGN),
    ("moe_mx_product", dict(base=at(2) + 2), ALIGN),
    ("moe_mx_product", dict(out=at(0)), ARG),
    ("moe_mx_product", dict(out=at(4) + 8 * 100 * 32 - 2), ARG),
    ("moe_mx_product", dict(out=at(2) + 32), ARG),
])
def test_refusals(name, kw, err):
    assert call(name, **kw) == err


@pytest.mark.parametrize("name", ["moe_mx_quantize", "moe_mx_dequantize", "moe_mx_product"])
def test_no_rows_enqueue_nothing(name):
    assert call(name, n=0) == moe.MOE_OK


def test_row_bytes():
    assert moe.moe_mx_row_bytes(7168, moe.MOE_MX_E2M1) == 3584
    assert moe.moe_mx_row_bytes(7168, moe.MOE_MX_E4M3) == 7168
    assert moe._lib.moe_mx_row_bytes(7168, 0) == ARG
    assert moe._lib.moe_mx_row_bytes(7168 + 16, 1) == UNSUPPORTED
    with pytest.raises(ValueError):
        moe.moe_mx_row_bytes(16400, 1)


def test_binding_refuses_host_tensors():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    slot, w = torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 2))
    mx = moe.MxRows(torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8))
    for fn in (lambda: moe.moe_combine_backward(x, x, slot, w), lambda: moe.moe_dispatch_backward(x, slot),
               lambda: moe.moe_combine_checkpoint(x, slot, w), lambda: moe.moe_combine_backward_mx(x, mx, slot, w),
               lambda: moe.moe_mx_quantize(x, 1), lambda: moe.moe_mx_dequantize(mx, 1),
               lambda: moe.moe_mx_product(mx, mx, slot)):
        with pytest.raises(ValueError, match="device tensor"):
            fn()
