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


def grouped(fn, p=P, q=P, off=P, out=P, rows=4, n=16, k=16, groups=2, dtype=mm.BF16, status=None, more=(), ws=()):
    if more and not ws:
        ws = (P, 1 << 40)
    return getattr(mm.lib(), fn)(p, q, off, out, rows, n, k, groups, dtype, *more, *ws, status, None)


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
        need = mm.mega_moe_grouped_weight_workspace_bytes(9000, 16, 16, 2)
        assert need > 0 and mm.mega_moe_grouped_weight_workspace_bytes(9000, 4096, 7168, 32) == 0
        assert grouped(fn, more=more, rows=9000, ws=(P, need - 1)) == mm.ERR_WORKSPACE_TOO_SMALL
        assert grouped(fn, more=more, rows=9000, ws=(None, need)) == mm.ERR_INVALID_ARG
        assert grouped(fn, more=more, rows=9000, ws=(ODD, need)) == mm.ERR_INVALID_ARG
        out = ctypes.c_uint64(0)
        lib = mm.lib()
        assert lib.mega_moe_grouped_weight_workspace_bytes(4, 16, 16, 2, None) == mm.ERR_INVALID_ARG
        assert lib.mega_moe_grouped_weight_workspace_bytes(-4, 16, 16, 2, ctypes.byref(out)) == mm.ERR_INVALID_ARG
        assert lib.mega_moe_grouped_weight_workspace_bytes(4, 12, 16, 2, ctypes.byref(out)) == mm.ERR_UNSUPPORTED
    else:
        assert grouped(fn, rows=1 << 26, n=65536, k=65536) == mm.ERR_UNSUPPORTED       # too many tiles
        assert grouped(fn, p=None, out=None, rows=0) == mm.OK                # nothing to do


def test_python_checks_refuse_before_the_library():
    x, w, off = torch.zeros(4, 16), torch.zeros(2, 16, 16), torch.zeros(3, dtype=torch.int32)
    for call in (lambda: mm.grouped_forward(x, w, off), lambda: mm.grouped_forward(None, None, None),
                 lambda: mm.grouped_backward_rows(x.bfloat16(), w.bfloat16(), off),
                 lambda: mm.grouped_backward_weight(x.bfloat16(), x.bfloat16(), off)):
        with pytest.raises(ValueError):
            call()


def router_cfg(**kw):
    base = dict(tokens=4, num_experts=16, topk=2, score=0, num_groups=4, topk_groups=2, group_top=2, renormalize=1,
                scale=1.0, dtype=mm.FP32)
    base.update(kw)
    return mm.mega_moe_router_config(*[base[n] for n, _ in mm.mega_moe_router_config._fields_])


def test_router_refusals():
    lib = mm.lib()
    for kw in (dict(num_experts=0), dict(num_experts=4097), dict(topk=0), dict(topk=17), dict(topk=65, num_experts=256),
               dict(score=2), dict(num_groups=0), dict(num_groups=3), dict(num_groups=128, num_experts=256),
               dict(topk_groups=0), dict(topk_groups=5), dict(group_top=0), dict(group_top=3), dict(dtype=3),
               dict(scale=float("inf")), dict(scale=float("nan")), dict(tokens=1 << 31), dict(tokens=1 << 30, topk=4)):
        c = router_cfg(**kw)
        assert lib.mega_moe_router_topk(ctypes.byref(c), P, P, P, P, None) == mm.ERR_UNSUPPORTED, kw
        assert lib.mega_moe_router_backward(ctypes.byref(c), P, P, P, P, None) == mm.ERR_UNSUPPORTED, kw
    c = router_cfg()
    assert lib.mega_moe_router_topk(None, P, P, P, P, None) == mm.ERR_INVALID_ARG
    assert lib.mega_moe_router_backward(None, P, P, P, P, None) == mm.ERR_INVALID_ARG
    neg = router_cfg(tokens=-1)
    assert lib.mega_moe_router_topk(ctypes.byref(neg), P, P, P, P, None) == mm.ERR_INVALID_ARG
    for i in (0, 1, 2, 3):
        args = [P, P, P, P]
        args[i] = ODD
        assert lib.mega_moe_router_topk(ctypes.byref(c), *args, None) == mm.ERR_INVALID_ARG, i
        assert lib.mega_moe_router_backward(ctypes.byref(c), *args, None) == mm.ERR_INVALID_ARG, i
        args[i] = None
        if i != 1:                                     # the bias may be missing
            assert lib.mega_moe_router_topk(ctypes.byref(c), *args, None) == mm.ERR_INVALID_ARG, i
        assert lib.mega_moe_router_backward(ctypes.byref(c), *args, None) == mm.ERR_INVALID_ARG, i
    none = router_cfg(tokens=0)
    assert lib.mega_moe_router_topk(ctypes.byref(none), None, None, None, None, None) == mm.OK
    assert lib.mega_moe_router_backward(ctypes.byref(none), None, None, None, None, None) == mm.OK


def test_ordering_refusals():
    lib = mm.lib()
    out = ctypes.c_uint64(0)
    assert lib.mega_moe_group_workspace_bytes(10, 4, None) == mm.ERR_INVALID_ARG
    assert lib.mega_moe_group_workspace_bytes(-1, 4, ctypes.byref(out)) == mm.ERR_INVALID_ARG
    for pairs, experts in ((1 << 31, 4), ((1 << 31) - 1, 4), (10, 0), (10, 4097)):
        assert lib.mega_moe_group_workspace_bytes(pairs, experts, ctypes.byref(out)) == mm.ERR_UNSUPPORTED
        assert lib.mega_moe_group_by_expert(P, pairs, 0, experts, P, P, P, P, 1 << 40, None) == mm.ERR_UNSUPPORTED
    need = mm.mega_moe_group_workspace_bytes(100000, 256)
    assert lib.mega_moe_group_by_expert(P, 100000, 0, 256, P, P, P, P, need - 1, None) == mm.ERR_WORKSPACE_TOO_SMALL
    assert lib.mega_moe_group_by_expert(P, 10, -1, 4, P, P, P, P, need, None) == mm.ERR_INVALID_ARG
    for i in range(5):
        args = [P] * 5
        args[i] = ODD
        a = (args[0], 100000, 0, 256, *args[1:])
        assert lib.mega_moe_group_by_expert(*a, need, None) == mm.ERR_INVALID_ARG, i


@pytest.mark.parametrize("experts", [513, 1000, 4096])
def test_ordering_of_no_pairs_asks_for_the_tables_its_launches_write(experts):
    """More than 512 experts take the three launches: counts of one chunk at least, and totals, an int32 per expert
    in each, whether there are pairs or not."""
    need = mm.mega_moe_group_workspace_bytes(0, experts)
    assert need >= 2 * 4 * experts
    assert need == mm.mega_moe_group_workspace_bytes(1, experts)
    assert mm.lib().mega_moe_group_by_expert(None, 0, 0, experts, P, None, None, P, need - 1, None) == \
        mm.ERR_WORKSPACE_TOO_SMALL


def test_router_python_checks():
    x = torch.zeros(4, 16)
    for call in (lambda: mm.router_topk(x, 2), lambda: mm.router_topk(None, 2), lambda: mm.group_by_expert(x.long(), 4),
                 lambda: mm.router_backward(x[:, :2], x, x[:, :2].long()), lambda: mm.router_backward(x, x, None)):
        with pytest.raises(ValueError):
            call()


def adapter_call(x=P, w=P, a=P, b=P, scales=P, off=P, adapter=P, y=P, rows=4, n=16, k=16, rank=8, requests=2, adapters=3,
                 dtype=mm.BF16, ws=P, nbytes=1 << 40, status=None):
    return mm.lib().mega_moe_adapter_forward(x, w, a, b, scales, off, adapter, y, rows, n, k, rank, requests, adapters,
                                             dtype, ws, nbytes, status, None)


def test_adapter_refusals():
    for name in ("x", "w", "a", "b", "scales", "off", "adapter", "y", "ws"):
        assert adapter_call(**{name: None}) == mm.ERR_INVALID_ARG, name
        assert adapter_call(**{name: ctypes.c_void_p(4098)}) == mm.ERR_INVALID_ARG, name
    for kw in (dict(rows=-1), dict(n=-8), dict(k=-8), dict(rank=-8), dict(requests=-1), dict(adapters=-1),
               dict(status=ctypes.c_void_p(4097))):
        assert adapter_call(**kw) == mm.ERR_INVALID_ARG, kw
    for kw in (dict(rank=0), dict(rank=12), dict(rank=264), dict(n=12), dict(k=20), dict(n=65544), dict(adapters=0),
               dict(adapters=65537), dict(requests=4097), dict(dtype=mm.FP32), dict(rows=(1 << 26) + 1)):
        assert adapter_call(**kw) == mm.ERR_UNSUPPORTED, kw
    assert adapter_call(nbytes=mm.mega_moe_adapter_workspace_bytes(4, 16, 16, 8, 2) - 1) == mm.ERR_WORKSPACE_TOO_SMALL
    assert adapter_call(rows=0, x=None, y=None) == mm.OK
    out = ctypes.c_uint64(0)
    lib = mm.lib()
    assert lib.mega_moe_adapter_workspace_bytes(4, 16, 16, 8, 2, None) == mm.ERR_INVALID_ARG
    assert lib.mega_moe_adapter_workspace_bytes(-1, 16, 16, 8, 2, ctypes.byref(out)) == mm.ERR_INVALID_ARG
    assert lib.mega_moe_adapter_workspace_bytes(4, 16, 16, 12, 2, ctypes.byref(out)) == mm.ERR_UNSUPPORTED
    x = torch.zeros(4, 16)
    with pytest.raises(ValueError):
        mm.adapter_forward(x, x, x, x, x, x, x)
