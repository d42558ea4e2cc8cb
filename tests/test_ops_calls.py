"""What the operators' Python calls do with their caller's tensors before and after the library, without a GPU."""
import pytest
import torch

from dispatch_fp8_grouped_amd import ops


def test_a_result_raises_where_a_gradient_would_be_lost():
    x, w = torch.randn(3, 4, requires_grad=True), torch.randn(4)
    y = ops._unrecorded("op", "do so", torch.zeros(3, 4), w, x)
    assert y.requires_grad and (y == 0).all()
    y.mul_(2)                                          # an ordinary tensor otherwise
    with pytest.raises(RuntimeError, match="op records no autograd graph: do so"):
        (y * x).sum().backward()


def test_a_result_is_left_alone_where_no_gradient_is_asked_for():
    out, x, p = torch.zeros(3), torch.randn(3), torch.randn(3, requires_grad=True)
    assert ops._unrecorded("op", "", out, x) is out
    with torch.no_grad():
        assert ops._unrecorded("op", "", out, p) is out

    class Own(torch.autograd.Function):                # a program's own node around the calls
        @staticmethod
        def forward(ctx, a):
            return ops._unrecorded("op", "", a * 2, a)

        @staticmethod
        def backward(ctx, g):
            return 2 * g
    Own.apply(p).sum().backward()
    assert (p.grad == 2).all()


def test_sizes_beyond_32_bits_are_refused_and_not_cut():
    far = (1 << 32) + 8
    for call in (lambda: ops._weight_bytes(0, far, 8, 1), lambda: ops._weight_bytes(0, 8, far, 1),
                 lambda: ops._weight_bytes(0, 8, 8, far), lambda: ops._group_bytes(10, far),
                 lambda: ops._group_bytes(10, 8 - (1 << 32)), lambda: ops._adapter_bytes(1, far, 8, 8, 1, 1),
                 lambda: ops._adapter_bytes(1, 8, far, 8, 1, 1), lambda: ops._adapter_bytes(1, 8, 8, far, 1, 1),
                 lambda: ops._adapter_bytes(1, 8, 8, 8, far, 1), lambda: ops._adapter_bytes(1, 8, 8, 8, 1, far)):
        with pytest.raises(ValueError, match="32-bit"):
            call()
    good = (4, 16, 2, 0, 4, 2, 1, 1, 1.0, ops.FP32)
    assert ops._config(*good).topk == 2
    for i in (1, 2, 4, 5, 6):
        with pytest.raises(ValueError, match="32-bit"):
            ops._config(*good[:i], good[i] + (1 << 32), *good[i + 1:])


def test_outputs_that_share_memory_with_an_input():
    whole = torch.zeros(100)
    ops._apart("out", whole[:50], whole[50:], None, torch.zeros(100), torch.zeros(0), whole[10:10])
    for other in (whole, whole[49:], whole[:1], whole[20:30].view(torch.int32), whole.view(torch.uint8)[199:201]):
        with pytest.raises(ValueError, match="out overlaps"):
            ops._apart("out", whole[:50], torch.zeros(3), other)
    for a, b in ((whole[:50], whole[50:]), (whole[50:], whole[:50])):
        ops._apart("out", a, b)
