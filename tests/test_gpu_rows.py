"""The norm, SwiGLU and 8-bit rows against their definitions in 64 bits.

Tolerances, counted in u = 2^-24 (half a step of fp32, relative), before the output's own rounding:
- 8-bit rows: the definition's scale and grid, exactly; of values computed in fp32 first, half a step of the grid beside
  the error of the value.
- norm: v is one addition (1 u).  A sum over a row adds at most 32 squares in a lane, 6 times within a wave and 16 waves:
  54 additions, and 3 u in each square, so 57 u of the sum and 29 of its root; root, division and the mean 4 u: r is off by at
  most 33 u, y by 33 + 1 + 3: below 40 u of |y|.
- its gradient: mean(g n) adds 54 times products with 2 roundings and one r: 56 + 34 u of mean |g n|; in dx it meets r twice
  more and 4 roundings: 56 + 3 * 34 + 4 < 192 u of the terms' magnitudes.  dweight adds at most `rows` products of 35 u.
- SwiGLU: exp's argument g log2(e) is off by 2 u of itself, which is 2 |g| u of the exponential; exp2, reciprocal and addition 5 u:
  sigmoid s is off by (2 |g| + 5) u, act by (2 |g| + 8) u.  dgate = dact up (s + g s (1 - s)): 1 - s is off by s's error, so
  by (2 |g| + 8) u of each term, twice: (4 |g| + 20) u of |dact up| s (1 + |g|).  Below gate -87 the exponential passes fp32's
  range and s is 0 for less than 2^-125."""
import pytest
import torch

import dispatch_fp8_grouped_amd as mm
import row_refs as ref
from row_refs import U
from test_gpu_grouped import check_weight, make

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
KINDS = {"bf16": BF16, "fp16": FP16, "fp32": FP32}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(shape, dtype, seed, std=1.0):
    return (torch.randn(*shape, generator=gen(seed), device="cuda") * std).to(dtype)


def check_rows8(codes, scales, want, error, what="rows8"):
    """codes * scales is `want` (finite), which was known up to `error` when it was rounded."""
    top, block_error = ref.blocks(want).abs().amax(-1), ref.blocks(error.expand_as(want)).amax(-1)
    s = scales.double()
    assert torch.equal(torch.exp2(torch.log2(s).round()), s), f"{what}: scale no power of two"
    assert ((top - block_error) <= 448 * s).all(), f"{what}: scale too small"
    low = (top + block_error) > 224 * s
    assert (low | (s == 2.0 ** -126)).all(), f"{what}: scale too large"
    half = torch.maximum(2.0 ** -4 * (want.abs() + error), 2.0 ** -10 * s.repeat_interleave(128, -1)[..., :want.shape[-1]])
    d = (ref.decode(codes, scales) - want).abs()
    assert (d <= error + half).all(), f"{what}: worst excess {(d - error - half).max().item():.3g}"


# ------------------------------------------------------------------ 8-bit rows
COLS = [1, 7, 8, 9, 120, 127, 128, 129, 136, 255, 1000, 4104, 7168]


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("cols", COLS)
def test_quantize_and_back(cols, kind):
    print(f"[case] {cols} {kind}", flush=True)
    for rows in (1, 3, 130):
        x = normal((rows, cols), KINDS[kind], rows + cols) * torch.exp2(torch.arange(rows, device="cuda") % 12 - 6)[:, None].to(KINDS[kind])
        x[rows // 2] = 0
        codes, scales = mm.quantize_rows(x)
        assert codes.shape == x.shape and scales.shape == (rows, -(-cols // 128))
        assert torch.equal(scales.double(), ref.scales_of(x))
        assert torch.equal(ref.decode(codes, scales), ref.quantized(x))
        for back in KINDS.values():
            got = mm.dequantize_rows(codes, scales, dtype=back)
            want = ref.quantized(x)
            ref.close(got, want, torch.zeros_like(want), "restored")
            if back != FP16 or kind == "fp16":       # a power of two: nothing is rounded again
                assert torch.equal(got.double(), want)


def test_values_at_the_borders_of_the_scales():
    """448 * 2^e and its neighbours, the ends of fp32's range, ties of the codes, signed zeros."""
    up = torch.tensor([448.0 * 2.0 ** e for e in range(-140, 119)], device="cuda")
    bits = up.view(torch.int32)
    for tops in (up, (bits - 1).view(FP32), (bits + 1).view(FP32)):
        x = tops[:, None] * torch.linspace(-1, 1, 128, device="cuda")[None]
        codes, scales = mm.quantize_rows(x)
        assert torch.equal(scales.double(), ref.scales_of(x))
        assert torch.equal(ref.decode(codes, scales), ref.quantized(x))
    ends = torch.tensor([[0.0, -0.0] * 64, [1e-45] * 128, [-1.17549435e-38] * 128, [3.4028234e38] * 128, [2.0 ** -149, 1.0] * 64], device="cuda")
    codes, scales = mm.quantize_rows(ends)
    assert torch.equal(scales.double(), ref.scales_of(ends))
    assert torch.equal(ref.decode(codes, scales), ref.quantized(ends))
    assert torch.equal(mm.dequantize_rows(codes, scales, dtype=FP32).double(), ref.quantized(ends))
    # halfway between neighbouring codes, scale 1: to the even one
    grid = ref.decode(torch.arange(0, 127, device="cuda"), torch.ones(1, device="cuda"))
    ties = torch.cat([(grid[1:] + grid[:-1]) / 2, grid[-2:]]).float()[None]
    codes, scales = mm.quantize_rows(ties)
    assert (scales == 1).all() and torch.equal(ref.decode(codes, scales), ref.quantized(ties))


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("kind", list(KINDS))
def test_a_block_with_an_infinity_or_nan(kind, bad):
    x = normal((5, 400), KINDS[kind], 1)
    x[2, 130] = bad
    x[4, 399] = bad
    codes, scales = mm.quantize_rows(x)
    got = ref.decode(codes, scales)
    want = ref.quantized(x)
    assert torch.isnan(want[2, 128:256]).all() and torch.isnan(want[4, 384:]).all() and torch.isnan(want).sum() == 128 + 16
    assert torch.equal(got.nan_to_num(-1e30), want.nan_to_num(-1e30)) and (scales[2, 1] == 1)
    for back in KINDS.values():
        assert torch.equal(torch.isnan(mm.dequantize_rows(codes, scales, dtype=back)), torch.isnan(want))


def test_restored_values():
    """Every code with scales that are no powers of two, and fp16's largest numbers."""
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(2, 128)
    for scale in (1.0, 0.37, 3e-5, 1e30, 0.0):
        scales = torch.full((2, 1), scale, device="cuda")
        for back in KINDS.values():
            want = ref.decode(codes, scales)
            ref.close(mm.dequantize_rows(codes, scales, dtype=back), want, U * want.abs() + 2.0 ** -149, f"{scale} {back}")
    x = torch.tensor([[65504.0, -65504.0, 63488.0, 1.0]], dtype=FP16, device="cuda")
    back = mm.dequantize_rows(*mm.quantize_rows(x), dtype=FP16)
    assert torch.equal(back, torch.tensor([[65504.0, -65504.0, 65504.0, 1.0]], dtype=FP16, device="cuda"))
    far = torch.tensor([[1e6, -1e6]], device="cuda")
    assert torch.isinf(mm.dequantize_rows(*mm.quantize_rows(far), dtype=FP16)).all()


# ------------------------------------------------------------------ norm
# columns of each way to lay a row out: 16 lanes, a wave, a work-group; odd ends
HIDDEN = [1, 7, 16, 100, 128, 129, 136, 500, 512, 1000, 2048, 2049, 4096, 7168, 8200, 12289, 16384]
TYPES = [("bf16", "bf16", "bf16"), ("bf16", "fp32", "fp32"), ("fp16", "fp16", "fp32"), ("fp16", "fp32", "fp16"), ("fp32", "fp32", "fp32")]


@pytest.mark.parametrize("dtype,stream,wkind", TYPES)
@pytest.mark.parametrize("hidden", HIDDEN)
def test_norm_forward(hidden, dtype, stream, wkind):
    print(f"[case] {hidden} {dtype} {stream} {wkind}", flush=True)
    w = 1 + normal((hidden,), KINDS[wkind], 3, 0.2)
    for rows, with_residual, quantize in ((1, True, "both"), (37, False, "both"), (18, True, True), (5, True, False)):
        x = normal((rows, hidden), KINDS[dtype], rows, 1.5)
        res = normal((rows, hidden), KINDS[stream], rows + 1, 3.0) if with_residual else None
        if rows > 4:
            x[3] = 0
            if with_residual:
                res[3] = 0
        eps = 1e-5
        y, h, rows8 = mm.rms_norm(x, w, residual=res, eps=eps, quantize=quantize)
        want, v, _ = ref.norm(x, res, w, eps)
        error = 40 * U * want.abs()
        assert (y is None) == (quantize is True) and (h is None) == (res is None) and (rows8 is None) == (quantize is False)
        if y is not None:
            assert y.dtype == x.dtype
            ref.close(y, want, error, "y")
        if h is not None:
            assert h.dtype == res.dtype
            ref.close(h, v, U * v.abs(), "h")
        if rows8 is not None:
            check_rows8(*rows8, want, error)


@pytest.mark.parametrize("out", list(KINDS))
@pytest.mark.parametrize("hidden", [100, 520, 7168])
def test_norm_of_a_stream_as_it_stands(hidden, out):
    """A float32 residual stream without an addition, rows of another type."""
    x = normal((9, hidden), FP32, 1)
    w = normal((hidden,), KINDS[out], 2)
    y, h, rows8 = mm.rms_norm(x, w, dtype=KINDS[out], quantize="both")
    want, _, _ = ref.norm(x, None, w, 1e-6)
    assert h is None and y.dtype == KINDS[out]
    ref.close(y, want, 40 * U * want.abs(), "y")
    check_rows8(*rows8, want, 40 * U * want.abs())


@pytest.mark.parametrize("dtype,stream,wkind", TYPES)
@pytest.mark.parametrize("hidden", HIDDEN)
def test_norm_backward(hidden, dtype, stream, wkind):
    print(f"[case] {hidden} {dtype} {stream} {wkind}", flush=True)
    w = 1 + normal((hidden,), KINDS[wkind], 3, 0.2)
    for rows, with_residual, kept in ((1, True, False), (37, False, False), (18, True, True), (5, False, True), (1300, True, False)):
        dy = normal((rows, hidden), KINDS[dtype], rows)
        h = normal((rows, hidden), KINDS[stream], rows + 1, 3.0)
        dres = normal((rows, hidden), KINDS[stream], rows + 2) if with_residual else None
        if rows > 4:
            h[3] = 0
            dy[4] = 0
        eps = 1e-3
        given = mm.quantize_rows(h) if kept else h
        value = ref.decode(*given) if kept else h
        dx, dw = mm.rms_norm_backward(dy, given, w, eps=eps, dresidual=dres)
        want, want_w, size, size_w = ref.norm_backward(dy, value, w, dres, eps)
        assert dx.dtype == (dres.dtype if dres is not None else dy.dtype if kept else h.dtype) and dw.dtype == FP32
        ref.close(dx, want, 192 * U * size, "dx")
        ref.close(dw, want_w, (rows + 64) * U * size_w, "dweight")


def test_norm_gradient_against_differences():
    """Central differences of the 64-bit definition in every input of a few rows: off by step^2 and by 2^-52 / step."""
    for rows, hidden in ((3, 24), (2, 130)):
        x, res = normal((rows, hidden), FP32, 5).double(), normal((rows, hidden), FP32, 6).double()
        w, dy = normal((hidden,), FP32, 7).double(), normal((rows, hidden), FP32, 8).double()
        dh = normal((rows, hidden), FP32, 9).double()

        def loss(res, w):
            y, v, _ = ref.norm(x, res, w, 1e-5)
            return (y * dy).sum() + (v * dh).sum()
        h = (x + res).float()
        x = h.double() - res
        dx, dw = mm.rms_norm_backward(dy.float(), h, w.float(), eps=1e-5, dresidual=dh.float())
        step = 1e-5
        for i in range(0, rows * hidden, 7):
            e = torch.zeros(rows * hidden, device="cuda", dtype=torch.float64)
            e[i] = step
            e = e.view(rows, hidden)
            diff = (loss(res + e, w) - loss(res - e, w)) / (2 * step)
            assert abs(dx.view(-1)[i].item() - diff.item()) < 1e-4
        for i in range(0, hidden, 5):
            e = torch.zeros(hidden, device="cuda", dtype=torch.float64)
            e[i] = step
            diff = (loss(res, w + e) - loss(res, w - e)) / (2 * step)
            assert abs(dw[i].item() - diff.item()) < 1e-4


def test_norm_of_large_small_and_broken_rows():
    x = normal((8, 1000), FP32, 1)
    x[0] *= 1e15
    x[1] *= 1e-20                                    # far below eps: y = x w / sqrt(eps)
    x[2, 7] = float("inf")
    x[3, 9] = float("nan")
    w = normal((1000,), FP32, 2)
    y, _, rows8 = mm.rms_norm(x, w, quantize="both")
    want, _, _ = ref.norm(x, None, w, 1e-6)
    error = 40 * U * want.abs() + 2.0 ** -126
    for r in (0, 1, 4, 5, 6, 7):
        ref.close(y[r], want[r], error[r], f"row {r}")
    assert torch.isnan(y[2, 7]) and (torch.isnan(y[2]).sum() == 1) and (y[2].nan_to_num(0) == 0).all()
    assert torch.isnan(y[3]).all()
    back = ref.decode(*rows8)
    assert torch.isnan(back[2, :128]).all() and (back[2, 128:] == 0).all() and torch.isnan(back[3]).all()
    check_rows8(rows8[0][4:], rows8[1][4:], want[4:], error[4:])
    # a row of zeros with eps 0 is 0 / 0, as the formula has it
    zero = torch.zeros(1, 64, device="cuda")
    assert torch.isnan(mm.rms_norm(zero, w[:64], eps=0.0)[0]).all() and (mm.rms_norm(zero, w[:64])[0] == 0).all()


# ------------------------------------------------------------------ SwiGLU
INTER = [1, 7, 8, 100, 128, 129, 1000, 2048, 8192]


def sigmoid_error(gate):
    return (2 * gate.abs() + 8) * U


def check_swiglu(act, gate, up):
    want = ref.swiglu(gate, up)
    ref.close(act, want, sigmoid_error(gate) * want.abs() + 2.0 ** -125 * (gate * up).abs(), "act")


def check_swiglu_backward(dgate_up, dact, gate, up):
    dg, du = ref.swiglu_backward(dact.double(), gate, up)
    s, n = torch.sigmoid(gate), gate.shape[-1]
    d = dact.double().abs()
    ref.close(dgate_up[..., :n], dg, ((4 * gate.abs() + 20) * U * s + 2.0 ** -125) * (1 + gate.abs()) * d * up.abs(), "dgate")
    ref.close(dgate_up[..., n:], du, sigmoid_error(gate) * du.abs() + 2.0 ** -125 * d * gate.abs(), "dup")


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("inter", INTER)
def test_swiglu(inter, kind):
    print(f"[case] {inter} {kind}", flush=True)
    for rows in (1, 3, 300):
        gate_up = normal((rows, 2 * inter), KINDS[kind], rows + inter, 2.0)
        gate_up[0, :inter] *= 20                       # gates far out on both sides
        dact = normal((rows, inter), KINDS[kind], inter)
        gate, up = gate_up.double().chunk(2, 1)
        act, none = mm.swiglu(gate_up)
        assert none is None
        check_swiglu(act, gate, up)
        again, kept = mm.swiglu(gate_up, checkpoint=True)
        assert torch.equal(act, again) and kept[0].shape == gate_up.shape and kept[1].shape == (rows, 2 * -(-inter // 128))
        codes, scales = kept[0].view(rows, 2, inter), kept[1].view(rows, 2, -1)
        by_rows = mm.quantize_rows(gate_up.view(2 * rows, inter))
        assert torch.equal(by_rows[0].view_as(codes), codes) and torch.equal(by_rows[1].view_as(scales), scales)
        dgate_up, none = mm.swiglu_backward(dact, gate_up)
        assert none is None
        check_swiglu_backward(dgate_up, dact, gate, up)
        both, act2 = mm.swiglu_backward(dact, gate_up, recompute=True)
        assert torch.equal(both, dgate_up) and torch.equal(act2, act)
        gate, up = ref.decode(codes, scales).unbind(1)
        dgate_up, act = mm.swiglu_backward(dact, kept, recompute=True)
        check_swiglu_backward(dgate_up, dact, gate, up)
        check_swiglu(act, gate, up)
        assert torch.equal(mm.swiglu_backward(dact, kept)[0], dgate_up)


def test_swiglu_gradient_against_differences():
    gate, up, dact = (normal((2, 40), BF16, i).double() for i in (1, 2, 3))
    got, _ = mm.swiglu_backward(dact.to(FP16), torch.cat([gate, up], 1).to(FP16))      # bf16 normals fit fp16
    step = 1e-5
    dg = dact * (ref.swiglu(gate + step, up) - ref.swiglu(gate - step, up)) / (2 * step)
    du = dact * (ref.swiglu(gate, up + step) - ref.swiglu(gate, up - step)) / (2 * step)
    for a, b in ((got[:, :40], dg), (got[:, 40:], du)):
        ref.close(a, b, torch.full_like(b, 1e-6) * (1 + b.abs()), "difference")


def test_swiglu_takes_the_rows_of_the_groups_alone():
    rows, inter = 60, 136
    gate_up, dact = normal((rows, 2 * inter), BF16, 1), normal((rows, inter), BF16, 2)
    want, kept = mm.swiglu(gate_up, checkpoint=True)
    want_d, want_a = mm.swiglu_backward(dact, kept, recompute=True)
    lib = mm.lib()
    p = lambda t: t.data_ptr()      # noqa: E731
    st = torch.cuda.current_stream().cuda_stream
    for offsets, lo, hi, bad in (([5, 9, 9, 40], 5, 40, False), ([0, 60], 0, 60, False), ([7, 7], 7, 7, False), ([-3, 70], 0, 60, True),
                                 ([50, 20], 50, 50, True), ([2 ** 31 - 1, -2 ** 31], 60, 60, True), ([-2 ** 31, 2 ** 31 - 1], 0, 60, True)):
        off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        outs = [torch.full_like(t.view(torch.uint8), 0x5C) for t in (want, kept[0], kept[1], want_d, want_a)]
        assert lib.mega_moe_swiglu(p(gate_up), p(outs[0]), p(outs[1]), p(outs[2]), p(off), len(offsets) - 1, rows, inter, mm.BF16,
                                   p(status), st) == 0
        assert lib.mega_moe_swiglu_backward(p(dact), p(kept[0]), p(kept[1]), p(outs[3]), p(outs[4]), p(off), len(offsets) - 1, rows,
                                            inter, mm.BF16, p(status), st) == 0
        torch.cuda.synchronize()
        assert status.item() == (mm.STATUS_BAD_LAYOUT if bad else 0), offsets
        for got, t in zip(outs, (want, kept[0], kept[1], want_d, want_a)):
            t = t.view(torch.uint8)
            assert torch.equal(got[lo:hi], t[lo:hi]) and (got[:lo] == 0x5C).all() and (got[hi:] == 0x5C).all(), offsets
        act, some = mm.swiglu(gate_up, checkpoint=True, offsets=off, status=status)
        d, a = mm.swiglu_backward(dact, some, recompute=True, offsets=off)
        for got, t in ((act, want), (some[0], kept[0]), (some[1], kept[1]), (d, want_d), (a, want_a)):
            assert torch.equal(got[lo:hi], t[lo:hi])


# ------------------------------------------------------------------ gradient of the weights from 8-bit rows
# counts of the groups, n, k: no rows, odd edges, parts of sums, large tiles and streams of them
WEIGHTS = [([1], 8, 8), ([0, 1, 0], 64, 72), ([3, 0, 17, 16, 15, 1], 264, 520), ([127, 128, 129, 1], 256, 192), ([700, 0, 0, 900], 768, 1096),
           ([2048], 512, 64), ([1] * 100 + [0] * 50 + [7] * 50, 72, 128), ([40] * 8, 2056, 2048), ([3000, 0, 2500, 1300, 257], 4104, 200),
           ([3000, 17, 0, 900], 4104, 2056), ([64], 2056, 7168), ([20000], 72, 64), ([9000, 0, 3, 4000], 136, 264),
           ([63, 64, 65, 0, 1, 2, 129], 2048, 2184), ([5000, 0, 3], 64, 8), ([31, 32, 33, 95, 96, 97], 264, 24),
           # so many tiles that the rows are restored first
           ([40, 0, 25], 8200, 8200)]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("counts,n,k", WEIGHTS)
def test_weight_gradient_from_codes(counts, n, k, kind):
    print(f"[case] {counts} {n} {k} {kind}", flush=True)
    x, dy, _, off_t, off = make(counts, n, k, KINDS[kind], seed=len(counts) + n, extra=3, first=2)
    codes, scales = mm.quantize_rows(x)
    value = ref.decode(codes, scales)
    assert torch.equal(value.to(x.dtype).double(), value)            # exact in the operands' type
    # what lies behind the groups' rows meets no sum
    codes[:2], codes[off[-1]:] = 0x7F, 0x7F
    dy[:2], dy[off[-1]:] = float("nan"), float("nan")
    check_weight(dy, value, off, mm.grouped_backward_weight(dy, (codes, scales), off_t))
    dw = mm.grouped_backward_weight(dy, (codes, scales), off_t, dtype=FP32)
    check_weight(dy, value, off, dw)
    before = dw.clone()
    assert mm.grouped_backward_weight(dy, (codes, scales), off_t, out=dw, accumulate=True) is dw
    check_weight(dy, value, off, dw, before=before)
    assert torch.equal(mm.grouped_backward_weight(dy, (codes, scales), off_t, dtype=FP32), before)


def test_weight_gradient_from_scales_of_any_kind():
    """The layer's own kind of scales, largest / 448: a value is rounded to the operands' type first."""
    x, dy, _, off_t, off = make([300, 0, 77], 136, 264, BF16, seed=4)
    codes = torch.randint(0, 256, x.shape, generator=gen(1), device="cuda").to(torch.uint8)
    codes[(codes & 127) == 127] = 0
    scales = torch.rand(x.shape[0], 3, generator=gen(2), device="cuda") / 448
    value = (ref.decode(codes, scales).float()).to(BF16).double()
    check_weight(dy, value, off, mm.grouped_backward_weight(dy, (codes, scales), off_t, dtype=FP32))


# ------------------------------------------------------------------ sizes
def test_no_rows():
    w = torch.ones(64, device="cuda")
    y, h, rows8 = mm.rms_norm(torch.empty(0, 64, device="cuda"), w, residual=torch.empty(0, 64, device="cuda"), quantize="both")
    assert y.shape == (0, 64) and h.shape == (0, 64) and rows8[0].shape == (0, 64) and rows8[1].shape == (0, 1)
    dx, dw = mm.rms_norm_backward(torch.empty(0, 64, device="cuda"), torch.empty(0, 64, device="cuda"), w)
    assert dx.shape == (0, 64) and (dw == 0).all()
    act, kept = mm.swiglu(torch.empty(0, 64, device="cuda", dtype=BF16), checkpoint=True)
    assert act.shape == (0, 32) and kept[0].shape == (0, 64) and kept[1].shape == (0, 2)
    assert mm.swiglu_backward(act, kept, recompute=True)[0].shape == (0, 64)
    assert mm.dequantize_rows(*mm.quantize_rows(torch.empty(0, 5, device="cuda"))).shape == (0, 5)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    codes, scales = mm.quantize_rows(torch.empty(0, 64, device="cuda"))
    dw = mm.grouped_backward_weight(torch.empty(0, 32, device="cuda", dtype=BF16), (codes, scales), off)
    assert dw.shape == (2, 32, 64) and (dw == 0).all()


@pytest.mark.parametrize("lead", [(), (3,), (2, 3, 4)])
def test_leading_dimensions(lead):
    x, w = normal((*lead, 200), BF16, 1), normal((200,), BF16, 2)
    y, _, rows8 = mm.rms_norm(x, w, quantize="both")
    want = ref.norm(x, None, w, 1e-6)[0]
    ref.close(y, want, 40 * U * want.abs(), "y")
    assert rows8[1].shape == (*lead, 2) and mm.dequantize_rows(*rows8).shape == x.shape
    dx, dw = mm.rms_norm_backward(y, x, w)
    assert dx.shape == x.shape and dw.shape == (200,)


@pytest.mark.parametrize("kind", list(KINDS))
def test_rows_from_anywhere(kind):
    """Slices of tokens whose rows are no multiple of 16 bytes, and tensors from the middle of a buffer."""
    dt = KINDS[kind]
    for cols in (61, 200, 1001, 3001):
        pool = normal((41 * cols + 5,), dt, cols)
        x = pool[3:3 + 41 * cols].view(41, cols)
        w = normal((cols + 1,), dt, 2)[1:]
        whole = mm.rms_norm(x.clone(), w.clone(), residual=x.clone(), quantize="both")
        grads = mm.rms_norm_backward(x.clone(), x.clone(), w.clone(), dresidual=x.clone())
        for lo, hi in ((1, 41), (3, 4), (41, 41)):
            s = x[lo:hi]
            y, h, (codes, scales) = mm.rms_norm(s, w, residual=s, quantize="both")
            for a, b in ((y, whole[0]), (h, whole[1]), (codes, whole[2][0]), (scales, whole[2][1])):
                assert torch.equal(a, b[lo:hi])
            assert torch.equal(mm.rms_norm_backward(s, s, w, dresidual=s)[0], grads[0][lo:hi])
            kept = whole[2][0][lo:hi], whole[2][1][lo:hi]
            assert torch.equal(mm.dequantize_rows(*kept), mm.dequantize_rows(*whole[2])[lo:hi])
            assert torch.equal(mm.quantize_rows(s)[0], mm.quantize_rows(x.clone())[0][lo:hi])
            if dt != FP32 and cols % 2 == 0:
                act, some = mm.swiglu(x.clone(), checkpoint=True)
                got, part = mm.swiglu(s, checkpoint=True)
                assert torch.equal(got, act[lo:hi]) and torch.equal(part[0], some[0][lo:hi])
                assert torch.equal(mm.swiglu_backward(act[lo:hi], part)[0], mm.swiglu_backward(act, some)[0][lo:hi])


def test_more_than_32_bits_of_values():
    """Rows whose last ones lie beyond 2^32 values."""
    rows, cols = (1 << 17) + 3, 32776
    x = torch.empty(rows, cols, dtype=BF16, device="cuda")
    for at in range(0, rows, 8192):
        x[at:at + 8192] = normal((min(8192, rows - at), cols), BF16, at)
    codes, scales = mm.quantize_rows(x)
    for s in (slice(0, 2), slice(65533, 65539), slice(rows - 3, rows)):
        assert torch.equal(ref.decode(codes[s], scales[s]), ref.quantized(x[s]))
    back = mm.dequantize_rows(codes, scales)
    assert torch.equal(back[-3:].double(), ref.quantized(x[-3:]))
    del back, codes, scales
    act, kept = mm.swiglu(x, checkpoint=True)
    check_swiglu(act[-3:], *x[-3:].double().chunk(2, 1))
    d, _ = mm.swiglu_backward(act, kept)
    gate, up = ref.decode(kept[0][-3:].view(3, 2, -1), kept[1][-3:].view(3, 2, -1)).unbind(1)
    check_swiglu_backward(d[-3:], act[-3:], gate, up)
    del act, kept, d, x
    torch.cuda.empty_cache()


def test_more_than_32_bits_of_values_in_a_norm():
    rows, hidden = (1 << 18) + 5, 16384
    x = torch.empty(rows, hidden, dtype=BF16, device="cuda")
    for at in range(0, rows, 16384):
        x[at:at + 16384] = normal((min(16384, rows - at), hidden), BF16, at)
    w = normal((hidden,), BF16, 1)
    y, _, rows8 = mm.rms_norm(x, w, quantize="both")
    want = ref.norm(x[-3:], None, w, 1e-6)[0]
    ref.close(y[-3:], want, 40 * U * want.abs(), "y")
    check_rows8(rows8[0][-3:], rows8[1][-3:], want, 40 * U * want.abs())
    del rows8
    dx, _ = mm.rms_norm_backward(y, x, w)
    want, _, size, _ = ref.norm_backward(y[-3:], x[-3:], w, None, 1e-6)
    ref.close(dx[-3:], want, 192 * U * size, "dx")
    del x, y, dx
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("powers", [True, False])
def test_weight_gradient_takes_the_restored_values(kind, powers):
    """With dy the identity dw is x itself: every code under scales of all sizes, as dequantize_rows restores it."""
    rows, k = 256, 520
    g = gen(11)
    codes = torch.randint(0, 256, (rows, k), generator=g, device="cuda").to(torch.uint8)
    codes[(codes & 127) == 127] = 0                    # NaN would meet dy's zeros in every row
    codes[:, :256] = torch.arange(256, device="cuda").to(torch.uint8)
    codes[:, 127] = codes[:, 255] = 0
    low, high = (-110, 118) if kind == "bf16" else (-30, 7)
    scales = torch.exp2(torch.randint(low, high + 1, (rows, 5), generator=g, device="cuda").float())
    if not powers:
        scales = scales * (1 + torch.rand(rows, 5, generator=g, device="cuda") * 0.75)
    if kind == "fp16" and powers:                      # 256 * 2^8 comes back as 65504
        scales[3, 4], codes[3, 512:] = 256.0, 0x78
    dy = torch.eye(rows, device="cuda", dtype=KINDS[kind])
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    want = mm.dequantize_rows(codes, scales, dtype=KINDS[kind])
    dw = mm.grouped_backward_weight(dy, (codes, scales), off, dtype=FP32)
    fine = torch.isfinite(want).all(0)                 # beyond fp16's range an infinity meets dy's zeros in its column
    assert fine.all() or (kind == "fp16" and not powers and fine.sum() > 100)
    assert torch.equal(dw[0][:, fine], want.float()[:, fine])


def test_weight_gradient_past_32_bits_of_codes():
    """Rows whose codes lie beyond 2^32 bytes, in the last group."""
    counts, n, k = [65530, 0, 4470], 8, 65536
    rows = sum(counts)
    codes = torch.empty(rows, k, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, k // 128, device="cuda")
    for at in range(0, rows, 8192):
        s = slice(at, min(at + 8192, rows))
        codes[s], scales[s] = mm.quantize_rows(normal((s.stop - at, k), BF16, at))
    dy = normal((rows, n), BF16, 3)
    off = [0, 65530, 65530, rows]
    dw = mm.grouped_backward_weight(dy, (codes, scales), torch.tensor(off, dtype=torch.int32, device="cuda"), dtype=FP32)
    assert (dw[1] == 0).all()
    last = slice(off[2], rows)
    check_weight(dy[last], ref.decode(codes[last], scales[last]), [0, counts[2]], dw[2:])
    # the last columns of the first group, from all of its rows
    part = mm.grouped_backward_weight(dy[:65530], (codes[:65530, -128:].contiguous(), scales[:65530, -1:].contiguous()),
                                      torch.tensor([0, 65530], dtype=torch.int32, device="cuda"), dtype=FP32)
    value = ref.decode(codes[:65530, -128:], scales[:65530, -1:])
    check_weight(dy[:65530], value, [0, 65530], part)
    check_weight(dy[:65530], value, [0, 65530], dw[:1, :, -128:])
    del codes, scales
    torch.cuda.empty_cache()
