"""The row operators' C ABI and their Python checks, without a GPU: every refusal comes before any device work."""
import ctypes

import pytest
import torch

import dispatch_fp8_grouped_amd as mm
from dispatch_fp8_grouped_amd import ops

P = ctypes.c_void_p(4096)          # aligned, never read: a refusal must come first


def at(address):
    return ctypes.c_void_p(address)


def norm(x=P, residual=P, weight=P, h=P, y=P, codes=P, scales=P, rows=4, hidden=64, eps=1e-6, dtype=mm.BF16, rdtype=mm.BF16,
         wdtype=mm.BF16):
    return mm.lib().mega_moe_rms_norm(x, residual, weight, h, y, codes, scales, rows, hidden, eps, dtype, rdtype, wdtype, None)


def norm_backward(dy=P, h=P, h_scales=None, weight=P, dresidual=P, dx=P, dweight=P, rows=4, hidden=64, eps=1e-6, dtype=mm.BF16,
                  rdtype=mm.BF16, wdtype=mm.BF16, ws=P, nbytes=1 << 40):
    return mm.lib().mega_moe_rms_norm_backward(dy, h, h_scales, weight, dresidual, dx, dweight, rows, hidden, eps, dtype, rdtype,
                                               wdtype, ws, nbytes, None)


SIZES = (dict(hidden=0), dict(hidden=16385), dict(rows=(1 << 26) + 1), dict(dtype=3), dict(dtype=-1), dict(rdtype=mm.FP16),
         dict(wdtype=mm.FP16), dict(dtype=mm.FP32, rdtype=mm.BF16), dict(eps=-1e-6), dict(eps=float("inf")), dict(eps=float("nan")))


def test_norm_refusals():
    for kw in (dict(x=None, residual=None), dict(weight=None), dict(y=None, codes=None, scales=None, h=None), dict(codes=None),
               dict(scales=None), dict(rows=-1), dict(hidden=-1), dict(x=at(4097)), dict(residual=at(4097)), dict(weight=at(4097)),
               dict(h=at(4097)), dict(y=at(4097)), dict(scales=at(4098)), dict(rdtype=mm.FP32, residual=at(4098)),
               dict(wdtype=mm.FP32, weight=at(4098))):
        assert norm(**kw) == mm.ERR_INVALID_ARG, kw
    for kw in SIZES:
        assert norm(**kw) == mm.ERR_UNSUPPORTED, kw
    assert norm(x=None, residual=None, weight=None, h=None, y=None, codes=None, scales=None, rows=0) == mm.OK


def test_norm_backward_refusals():
    need = mm.mega_moe_norm_workspace_bytes(4, 64)
    assert need >= 4 * 64
    for kw in (dict(dy=None), dict(h=None), dict(weight=None), dict(dx=None), dict(dweight=None), dict(ws=None), dict(rows=-1),
               dict(hidden=-1), dict(dy=at(4097)), dict(h=at(4097)), dict(h_scales=at(4098)), dict(weight=at(4097)),
               dict(dresidual=at(4097)), dict(dx=at(4097)), dict(dweight=at(4098)), dict(ws=at(4098))):
        assert norm_backward(**kw) == mm.ERR_INVALID_ARG, kw
    for kw in SIZES:
        assert norm_backward(**kw) == mm.ERR_UNSUPPORTED, kw
    assert norm_backward(nbytes=need - 1) == mm.ERR_WORKSPACE_TOO_SMALL
    out, lib = ctypes.c_uint64(0), mm.lib()
    assert lib.mega_moe_norm_workspace_bytes(4, 64, None) == mm.ERR_INVALID_ARG
    assert lib.mega_moe_norm_workspace_bytes(-1, 64, ctypes.byref(out)) == mm.ERR_INVALID_ARG
    assert lib.mega_moe_norm_workspace_bytes(4, 16385, ctypes.byref(out)) == mm.ERR_UNSUPPORTED
    assert mm.mega_moe_norm_workspace_bytes(0, 64) == 0


def test_rows_refusals():
    lib = mm.lib()
    for fn in (lib.mega_moe_quantize_rows, lib.mega_moe_dequantize_rows):
        for args in ((None, P, P, 4, 64, mm.BF16), (P, None, P, 4, 64, mm.BF16), (P, P, None, 4, 64, mm.BF16), (P, P, P, -1, 64, mm.BF16),
                     (P, P, P, 4, -1, mm.BF16)):
            assert fn(*args, None) == mm.ERR_INVALID_ARG, args
        for args in ((P, P, P, 4, 0, mm.BF16), (P, P, P, 4, 65537, mm.BF16), (P, P, P, (1 << 26) + 1, 64, mm.BF16), (P, P, P, 4, 64, 3)):
            assert fn(*args, None) == mm.ERR_UNSUPPORTED, args
        assert fn(None, None, None, 0, 64, mm.FP32, None) == mm.OK
    assert lib.mega_moe_quantize_rows(at(4097), P, P, 4, 64, mm.BF16, None) == mm.ERR_INVALID_ARG
    assert lib.mega_moe_quantize_rows(at(4098), P, P, 4, 64, mm.FP32, None) == mm.ERR_INVALID_ARG
    assert lib.mega_moe_quantize_rows(P, P, at(4098), 4, 64, mm.BF16, None) == mm.ERR_INVALID_ARG
    assert lib.mega_moe_dequantize_rows(P, at(4098), P, 4, 64, mm.BF16, None) == mm.ERR_INVALID_ARG
    assert lib.mega_moe_dequantize_rows(P, P, at(4097), 4, 64, mm.FP16, None) == mm.ERR_INVALID_ARG


def swiglu(gate_up=P, act=P, codes=P, scales=P, offsets=None, groups=0, rows=4, inter=64, dtype=mm.BF16, status=None):
    return mm.lib().mega_moe_swiglu(gate_up, act, codes, scales, offsets, groups, rows, inter, dtype, status, None)


def swiglu_backward(dact=P, gate_up=P, scales=None, dgate_up=P, act=None, offsets=None, groups=0, rows=4, inter=64, dtype=mm.BF16,
                    status=None):
    return mm.lib().mega_moe_swiglu_backward(dact, gate_up, scales, dgate_up, act, offsets, groups, rows, inter, dtype, status, None)


def test_swiglu_refusals():
    for call in (swiglu, swiglu_backward):
        for kw in (dict(gate_up=None), dict(rows=-1), dict(inter=-1), dict(groups=-1), dict(gate_up=at(4097)), dict(scales=at(4098)),
                   dict(act=at(4097)), dict(offsets=at(4098), groups=2), dict(status=at(4098))):
            assert call(**kw) == mm.ERR_INVALID_ARG, kw
        for kw in (dict(inter=0), dict(inter=65537), dict(rows=(1 << 26) + 1), dict(dtype=mm.FP32), dict(offsets=P, groups=0),
                   dict(offsets=P, groups=1025)):
            assert call(**kw) == mm.ERR_UNSUPPORTED, kw
        assert call(rows=0, gate_up=None, act=None) == mm.OK
    for kw in (dict(act=None), dict(codes=None), dict(scales=None)):
        assert swiglu(**kw) == mm.ERR_INVALID_ARG, kw
    for kw in (dict(dact=None), dict(dgate_up=None), dict(dact=at(4097)), dict(dgate_up=at(4097))):
        assert swiglu_backward(**kw) == mm.ERR_INVALID_ARG, kw


def weight(dy=P, codes=P, scales=P, off=P, dw=P, rows=4, n=16, k=16, groups=2, dtype=mm.BF16, out=mm.FP32, accumulate=0, ws=P,
           nbytes=1 << 40, status=None):
    return mm.lib().mega_moe_grouped_backward_weight_codes(dy, codes, scales, off, dw, rows, n, k, groups, dtype, out, accumulate, ws,
                                                           nbytes, status, None)


def test_weight_gradient_refusals():
    for kw in (dict(dy=None), dict(codes=None), dict(scales=None), dict(off=None), dict(dw=None), dict(dy=at(4104)), dict(codes=at(4100)),
               dict(scales=at(4098)), dict(off=at(4098)), dict(dw=at(4104)), dict(status=at(4097)), dict(rows=-1), dict(n=-8),
               dict(k=-8), dict(groups=-1)):
        assert weight(**kw) == mm.ERR_INVALID_ARG, kw
    for kw in (dict(n=0), dict(n=12), dict(k=4), dict(k=65544), dict(groups=0), dict(groups=1025), dict(dtype=mm.FP32), dict(dtype=9),
               dict(rows=(1 << 26) + 1), dict(out=mm.FP16), dict(out=mm.BF16, accumulate=1), dict(n=65536, k=65536, groups=1024)):
        assert weight(**kw) == mm.ERR_UNSUPPORTED, kw
    # a split sum, rows that are restored because there are many tiles, and because they are shorter than a load
    for rows, n, k, groups in ((9000, 16, 16, 2), (100, 8200, 8200, 3), (100, 16, 8, 2)):
        need = mm.mega_moe_grouped_codes_workspace_bytes(rows, n, k, groups)
        assert need > 0
        sizes = dict(rows=rows, n=n, k=k, groups=groups)
        assert weight(**sizes, nbytes=need - 1) == mm.ERR_WORKSPACE_TOO_SMALL
        assert weight(**sizes, ws=None, nbytes=need) == mm.ERR_INVALID_ARG
        assert weight(**sizes, ws=at(4104), nbytes=need) == mm.ERR_INVALID_ARG
    assert mm.mega_moe_grouped_codes_workspace_bytes(2000, 1000, 2056, 10) == 0      # no 16-bit copy of the rows
    out, lib = ctypes.c_uint64(0), mm.lib()
    assert lib.mega_moe_grouped_codes_workspace_bytes(4, 16, 16, 2, None) == mm.ERR_INVALID_ARG
    assert lib.mega_moe_grouped_codes_workspace_bytes(-4, 16, 16, 2, ctypes.byref(out)) == mm.ERR_INVALID_ARG
    assert lib.mega_moe_grouped_codes_workspace_bytes(4, 12, 16, 2, ctypes.byref(out)) == mm.ERR_UNSUPPORTED


def test_python_checks_refuse_before_the_library():
    x, w = torch.zeros(4, 16), torch.zeros(16)
    codes, scales = torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 1)
    off = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: mm.rms_norm(x, w), lambda: mm.rms_norm(None, w), lambda: mm.rms_norm(x, w, quantize="y"),
                 lambda: mm.rms_norm_backward(x, x, w), lambda: mm.rms_norm_backward(None, x, w), lambda: mm.rms_norm_backward(x, None, w),
                 lambda: mm.swiglu(x.bfloat16()), lambda: mm.swiglu(None), lambda: mm.swiglu_backward(x.bfloat16(), x.bfloat16()),
                 lambda: mm.swiglu_backward(None, None), lambda: mm.quantize_rows(x), lambda: mm.quantize_rows(None),
                 lambda: mm.dequantize_rows(codes, scales), lambda: mm.dequantize_rows(None, None),
                 lambda: mm.dequantize_rows(codes, scales, dtype=torch.float64),
                 lambda: mm.grouped_backward_weight(x.bfloat16(), (codes, scales), off),
                 lambda: mm.grouped_backward_weight(x.bfloat16(), (None, None), off)):
        with pytest.raises(ValueError):
            call()


def test_sizes_beyond_32_bits_are_refused_and_not_cut():
    far = (1 << 32) + 8
    for call in (lambda: ops._codes_bytes(0, far, 8, 1), lambda: ops._codes_bytes(0, 8, far, 1), lambda: ops._codes_bytes(0, 8, 8, far),
                 lambda: ops._norm_bytes(0, far)):
        with pytest.raises(ValueError, match="32-bit"):
            call()
