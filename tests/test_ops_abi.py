"""The operators' C ABI and their Python checks, without a GPU: every refusal comes before any device work."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import dispatch_fp8_grouped_amd as mm

from conftest import ROOT

HEADER = os.path.join(ROOT, "include", "mega_moe_ops.h")
P = ctypes.c_void_p(4096)          # aligned, never read: a refusal must come first
ODD = ctypes.c_void_p(4104)


def test_library_exports_every_declared_operator():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(mega_moe_[a-z_]+)\s*\(", text))
    assert names == set(mm.OPS_EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", mm.LIB_PATH], capture_output=True, text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if " T " in line}
    assert names <= exported
    for n in names:
        assert callable(getattr(mm, n))


def grouped(fn, p=P, q=P, off=P, out=P, rows=4, n=16, k=16, groups=2, dtype=mm.BF16, status=None, more=()):
    return getattr(mm.lib(), fn)(p, q, off, out, rows, n, k, groups, dtype, *more, status, None)


@pytest.mark.parametrize("fn,more", [("mega_moe_grouped_forward", ()), ("mega_moe_grouped_backward_rows", ()),
                                     ("mega_moe_grouped_backward_weight", (mm.FP32, 0))])
def test_grouped_refusals(fn, more):
    for kw in (dict(p=None), dict(q=None), dict(off=None), dict(out=None), dict(p=ODD), dict(q=ODD), dict(out=ODD),
               dict(off=ctypes.c_void_p(4098)), dict(status=ctypes.c_void_p(4097)), dict(rows=-1), dict(n=-8),
               dict(k=-8), dict(groups=-1)):
        assert grouped(fn, more=more, **kw) == mm.ERR_INVALID_ARG, kw
    for kw in (dict(n=0), dict(n=12), dict(k=4), dict(k=65544), dict(n=1 << 20), dict(groups=0), dict(groups=1025),
               dict(dtype=mm.FP32), dict(dtype=9), dict(rows=(1 << 26) + 1)):
        assert grouped(fn, more=more, **kw) == mm.ERR_UNSUPPORTED, kw
    if more:
        assert grouped(fn, more=(mm.FP16, 0)) == mm.ERR_UNSUPPORTED          # bf16 operands, fp16 output
        assert grouped(fn, more=(mm.BF16, 1)) == mm.ERR_UNSUPPORTED          # accumulating in 16 bits
        assert grouped(fn, more=more, n=65536, k=65536, groups=1024) == mm.ERR_UNSUPPORTED   # too many tiles
    else:
        assert grouped(fn, p=None, out=None, rows=0) == mm.OK                # nothing to do


def test_python_checks_refuse_before_the_library():
    x, w, off = torch.zeros(4, 16), torch.zeros(2, 16, 16), torch.zeros(3, dtype=torch.int32)
    for call in (lambda: mm.grouped_forward(x, w, off), lambda: mm.grouped_forward(None, None, None),
                 lambda: mm.grouped_backward_rows(x.bfloat16(), w.bfloat16(), off),
                 lambda: mm.grouped_backward_weight(x.bfloat16(), x.bfloat16(), off)):
        with pytest.raises(ValueError):
            call()
