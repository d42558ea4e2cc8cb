"""Products grouped by expert and their gradients against plain products in 64 bits.

Tolerance.  Operands are exact in both; a 16-bit product is exact in fp32, and a sum of c terms in fp32 is off
by at most c * 2^-24 times the sum of the terms' magnitudes S, whatever the order (each of the at most c
additions rounds a partial sum of magnitude at most S by 2^-24).  Rounding the output adds half a step of its
type, eps / 2 relative, and for float16 at most half of its smallest subnormal.  S is computed in 64 bits from
the operands' magnitudes."""
import pytest
import torch

import dispatch_fp8_grouped_amd as mm

pytestmark = pytest.mark.gpu

KINDS = {"bf16": torch.bfloat16, "fp16": torch.float16}


def offsets_of(counts, first=0):
    o = [first]
    for c in counts:
        o.append(o[-1] + c)
    return o


def make(counts, n, k, dtype, seed=0, extra=0, first=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    off = offsets_of(counts, first)
    rows = off[-1] + extra
    x = torch.randn(rows, k, generator=g, device="cuda").to(dtype)
    dy = torch.randn(rows, n, generator=g, device="cuda").to(dtype)
    w = torch.randn(len(counts), n, k, generator=g, device="cuda").to(dtype)
    return x, dy, w, torch.tensor(off, dtype=torch.int32, device="cuda"), off


def close(got, want, magnitude, terms):
    eps = torch.finfo(got.dtype).eps
    tiny = torch.finfo(got.dtype).smallest_normal * eps
    bound = terms * 2.0 ** -24 * magnitude
    bound = bound + eps / 2 * (want.abs() + bound) + tiny / 2
    d = (got.double() - want).abs()
    assert torch.isfinite(got.double()).all()
    assert (d <= bound).all(), f"worst excess {(d - bound).max().item():.3g}, {(d > bound).sum().item()} values"


def check_forward(x, w, off_t, off, y):
    for e in range(len(off) - 1):
        s = slice(off[e], off[e + 1])
        a, b = x[s].double(), w[e].double().t().contiguous()
        close(y[s], a @ b, a.abs() @ b.abs(), x.shape[1])


def check_rows(dy, w, off_t, off, dx):
    for e in range(len(off) - 1):
        s = slice(off[e], off[e + 1])
        a, b = dy[s].double(), w[e].double()
        close(dx[s], a @ b, a.abs() @ b.abs(), dy.shape[1])


def check_weight(dy, x, off, dw, before=None):
    for e in range(len(off) - 1):
        s = slice(off[e], off[e + 1])
        a, b = dy[s].double().t().contiguous(), x[s].double()
        want, mag = a @ b, a.abs() @ b.abs()
        if before is not None:
            want, mag = want + before[e].double(), mag + before[e].double().abs()
        close(dw[e], want, mag, off[e + 1] - off[e] + 1)


# counts of the groups, n, k: one row, no rows, counts around the tile heights, odd columns, many groups
SHAPES = [
    ([1], 8, 8),
    ([0, 1, 0], 64, 72),
    ([5], 1000, 136),
    ([3, 0, 17, 16, 15, 1], 264, 520),
    ([33, 31, 64, 65, 0, 2], 136, 328),
    ([127, 128, 129, 1], 256, 192),
    ([255, 0, 257, 300], 520, 264),
    ([700, 0, 0, 900], 768, 1096),
    ([2048], 512, 64),
    ([1] * 100 + [0] * 50 + [7] * 50, 72, 128),
    ([40] * 8, 2056, 2048),
    # long enough for the large tiles, with groups that end just behind one, in its first and in its second half
    ([3000, 0, 2500, 1300, 257], 4104, 200),
    ([6000, 129, 128, 127, 1], 2056, 328),
    ([1, 300, 8000], 520, 3080),
    ([9000], 264, 4104),
    ([3000, 17, 0, 900], 4104, 2056),
    # the shapes with groups of waves along the contraction; weights whose rows are split into parts
    ([64], 2056, 7168),
    ([3], 520, 8200),
    ([700, 0, 520, 300], 2056, 4104),
    ([20000], 72, 64),
    ([9000, 0, 3, 4000], 136, 264),
    # few tiles with long contractions, in either direction; square tiles with a short last one
    ([250, 262], 2048, 8192),
    ([250, 262], 8192, 2048),
    ([260, 130, 0, 190, 300], 1032, 2056),
]


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("counts,n,k", SHAPES)
def test_forward_and_gradients(counts, n, k, kind):
    print(f"[case] {counts} n {n} k {k} {kind}", flush=True)
    x, dy, w, off_t, off = make(counts, n, k, KINDS[kind], seed=len(counts) + n)
    check_forward(x, w, off_t, off, mm.grouped_forward(x, w, off_t))
    check_rows(dy, w, off_t, off, mm.grouped_backward_rows(dy, w, off_t))
    check_weight(dy, x, off, mm.grouped_backward_weight(dy, x, off_t))
    check_weight(dy, x, off, mm.grouped_backward_weight(dy, x, off_t, dtype=torch.float32))


def test_many_groups_of_one_row():
    """More groups than one batch of the tile search holds (64), up to the limit of 1024."""
    x, dy, w, off_t, off = make([1, 0, 2, 0] * 256, 40, 48, torch.bfloat16, seed=3)
    check_forward(x, w, off_t, off, mm.grouped_forward(x, w, off_t))
    check_rows(dy, w, off_t, off, mm.grouped_backward_rows(dy, w, off_t))
    check_weight(dy, x, off, mm.grouped_backward_weight(dy, x, off_t, dtype=torch.float32))


@pytest.mark.parametrize("counts", [[7, 0, 20], [150, 3, 90], [600, 300]])
def test_rows_outside_the_groups_are_left_alone(counts):
    """Rows before the first group and behind the last one are not written, and NaN in them reaches nothing."""
    x, dy, w, off_t, off = make(counts, 136, 200, torch.bfloat16, seed=5, extra=37, first=9)
    inside = slice(off[0], off[-1])
    for t in (x, dy):
        t[:9] = float("nan")
        t[off[-1]:] = float("nan")
    y = torch.full((x.shape[0], 136), 7.0, dtype=torch.bfloat16, device="cuda")
    assert mm.grouped_forward(x, w, off_t, out=y) is y
    check_forward(x, w, off_t, off, y)
    dx = torch.full_like(x, 7.0)
    mm.grouped_backward_rows(dy, w, off_t, out=dx)
    check_rows(dy, w, off_t, off, dx)
    for t in (y, dx):
        assert (t[:9] == 7.0).all() and (t[inside.stop:] == 7.0).all()
    check_weight(dy, x, off, mm.grouped_backward_weight(dy, x, off_t, dtype=torch.float32))


def test_nan_stays_in_its_row_and_its_group():
    x, dy, w, off_t, off = make([20, 140, 9], 264, 136, torch.bfloat16, seed=6)
    clean_y, clean_dx = mm.grouped_forward(x, w, off_t), mm.grouped_backward_rows(dy, w, off_t)
    clean_dw = mm.grouped_backward_weight(dy, x, off_t)
    x[25], dy[25] = float("nan"), float("inf")
    y, dx = mm.grouped_forward(x, w, off_t), mm.grouped_backward_rows(dy, w, off_t)
    dw = mm.grouped_backward_weight(dy, x, off_t)
    keep = torch.arange(x.shape[0], device="cuda") != 25
    assert torch.isnan(y[25]).all() and not torch.isfinite(dx[25]).any()
    assert torch.equal(y[keep], clean_y[keep]) and torch.equal(dx[keep], clean_dx[keep])
    assert torch.equal(dw[0], clean_dw[0]) and torch.equal(dw[2], clean_dw[2])
    assert torch.isnan(dw[1]).all()


# one work-group per tile; parts of the rows; streams of tiles
@pytest.mark.parametrize("counts,n,k", [([30, 0, 200], 136, 264), ([3000, 0, 2500], 136, 264), ([700, 0, 90], 2056, 2312)])
def test_accumulate_into_fp32_gradient(counts, n, k):
    x, dy, w, off_t, off = make(counts, n, k, torch.bfloat16, seed=7)
    before = torch.randn(3, n, k, device="cuda")
    dw = before.clone()
    assert mm.grouped_backward_weight(dy, x, off_t, out=dw, accumulate=True) is dw
    check_weight(dy, x, off, dw, before)
    assert torch.equal(dw[1], before[1])


def test_gradients_against_differences():
    """d/dx and d/dw of sum(g * y) by central differences of the 64-bit product, and the kernels' gradients."""
    x, g, w, off_t, off = make([4, 0, 9], 24, 16, torch.float16, seed=8)
    dx, dw = mm.grouped_backward_rows(g, w, off_t), mm.grouped_backward_weight(g, x, off_t, dtype=torch.float32)

    def loss(xx, ww):
        return sum((g[off[e]:off[e + 1]].double() * (xx[off[e]:off[e + 1]] @ ww[e].t())).sum() for e in range(3))
    xd, wd, h = x.double(), w.double(), 2.0 ** -6
    for (r, c) in [(0, 0), (3, 15), (12, 7)]:
        d = torch.zeros_like(xd)
        d[r, c] = h
        diff = (loss(xd + d, wd) - loss(xd - d, wd)) / (2 * h)
        # the loss is linear in x: the difference is exact up to fp64 rounding; dx is rounded to fp16
        assert abs(diff - dx[r, c].double()) <= 2.0 ** -10 * (g[r].double().abs() @ wd[0 if r < 4 else 2][:, c].abs())
    for (e, i, c) in [(0, 0, 0), (2, 23, 15), (1, 3, 3)]:
        d = torch.zeros_like(wd)
        d[e, i, c] = h
        diff = (loss(xd, wd + d) - loss(xd, wd - d)) / (2 * h)
        assert abs(diff - dw[e, i, c].double()) <= 1e-5 * (1 + abs(diff))


def test_broken_offsets_latch_the_status_and_stay_in_bounds():
    x, dy, w, off_t, off = make([10, 20, 30], 72, 64, torch.bfloat16, seed=9)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    mm.grouped_forward(x, w, off_t, status=st)
    mm.grouped_backward_weight(dy, x, off_t, status=st)
    assert st.item() == 0
    for bad in ([0, 10, 5, 60], [-3, 10, 30, 60], [0, 10, 30, 61], [0, 10, 2 ** 31 - 1, 60], [2 ** 31 - 1, -2 ** 31, 0, 0]):
        b = torch.tensor(bad, dtype=torch.int32, device="cuda")
        for call in (lambda s: mm.grouped_forward(x, w, b, status=s), lambda s: mm.grouped_backward_rows(dy, w, b, status=s),
                     lambda s: mm.grouped_backward_weight(dy, x, b, status=s)):
            st.zero_()
            call(st)
            assert st.item() == mm.STATUS_BAD_LAYOUT, bad


def test_no_rows():
    x, dy, w, off_t, off = make([0, 0], 16, 24, torch.bfloat16)
    assert mm.grouped_forward(x, w, off_t).shape == (0, 16)
    assert mm.grouped_backward_rows(dy, w, off_t).shape == (0, 24)
    dw = mm.grouped_backward_weight(dy, x, off_t, out=torch.full((2, 16, 24), 3.0, dtype=torch.bfloat16, device="cuda"))
    assert (dw == 0).all()


def test_repeat_other_stream_and_graph_replay_give_the_same_bits():
    replay_all([90, 0, 300, 11], 264, 392)


@pytest.mark.parametrize("counts,n,k", [([5000, 0, 2000], 264, 136), ([900, 1, 0, 2500, 40], 2056, 2056)])
def test_split_sums_streams_and_large_tiles_replay_to_the_same_bits(counts, n, k):
    replay_all(counts, n, k)


def replay_all(counts, n, k):
    x, dy, w, off_t, off = make(counts, n, k, torch.bfloat16, seed=10)

    def all_three(stream=None):
        return (mm.grouped_forward(x, w, off_t, stream=stream), mm.grouped_backward_rows(dy, w, off_t, stream=stream),
                mm.grouped_backward_weight(dy, x, off_t, dtype=torch.float32, stream=stream))
    want = all_three()
    for a, b in zip(want, all_three()):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for how in (side, side.cuda_stream):
        got = all_three(how)
        side.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = all_three()
    for i in range(3):
        x.mul_(-1)
        for t in got:
            t.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        eager = all_three()
        for a, b in zip(eager, got):
            assert torch.equal(a, b), i


def test_row_tensors_past_32_bit_offsets():
    """Rows of more than 2^32 bytes and 2^31 values, in one group and at the edge of another."""
    rows, n, k = 600_000, 16, 4104
    g = torch.Generator(device="cuda").manual_seed(11)
    x = torch.randn(rows, k, generator=g, device="cuda", dtype=torch.bfloat16)
    dy = torch.randn(rows, n, generator=g, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(2, n, k, generator=g, device="cuda", dtype=torch.bfloat16)
    off = [0, 590_001, rows]
    off_t = torch.tensor(off, dtype=torch.int32, device="cuda")
    y = mm.grouped_forward(x, w, off_t)
    dx = mm.grouped_backward_rows(dy, w, off_t)
    for e, s in ((0, slice(0, 300)), (0, slice(523_000, 523_500)), (0, slice(589_800, 590_001)), (1, slice(590_001, 590_300)),
                 (1, slice(rows - 100, rows))):
        a, d, b = x[s].double(), dy[s].double(), w[e].double()
        bt = b.t().contiguous()
        close(y[s], a @ bt, a.abs() @ bt.abs(), k)
        close(dx[s], d @ b, d.abs() @ b.abs(), n)
    dw = mm.grouped_backward_weight(dy, x, off_t, dtype=torch.float32)
    for e in range(2):
        want, mag = torch.zeros(n, k, device="cuda", dtype=torch.float64), torch.zeros(n, k, device="cuda", dtype=torch.float64)
        for r in range(off[e], off[e + 1], 50_000):
            s = slice(r, min(r + 50_000, off[e + 1]))
            a, b = dy[s].double().t().contiguous(), x[s].double()
            want += a @ b
            mag += a.abs() @ b.abs()
        close(dw[e], want, mag, off[e + 1] - off[e])


def test_weights_past_32_bit_offsets():
    groups, n, k = 40, 8192, 8200
    counts = [3, 0, 1] + [0] * 35 + [2, 5]
    g = torch.Generator(device="cuda").manual_seed(12)
    off = offsets_of(counts)
    off_t = torch.tensor(off, dtype=torch.int32, device="cuda")
    x = torch.randn(off[-1], k, generator=g, device="cuda", dtype=torch.bfloat16)
    dy = torch.randn(off[-1], n, generator=g, device="cuda", dtype=torch.bfloat16)
    dw = mm.grouped_backward_weight(dy, x, off_t)
    assert dw.numel() > 2 ** 31
    for e in (0, 1, 2, 20, 38, 39):
        a, b = dy[off[e]:off[e + 1]].double().t().contiguous(), x[off[e]:off[e + 1]].double()
        close(dw[e], a @ b, a.abs() @ b.abs(), counts[e] + 1)
    y, dx = mm.grouped_forward(x, dw, off_t), mm.grouped_backward_rows(dy, dw, off_t)
    for e in (0, 2, 38, 39):
        s = slice(off[e], off[e + 1])
        a, d, b = x[s].double(), dy[s].double(), dw[e].double()
        bt = b.t().contiguous()
        close(y[s], a @ bt, a.abs() @ bt.abs(), k)
        close(dx[s], d @ b, d.abs() @ b.abs(), n)


def test_two_calls_at_once_on_two_streams():
    x, dy, w, off_t, off = make([900, 1, 0, 2500, 40], 2056, 2056, torch.bfloat16, seed=13)
    x2, dy2, w2, off2_t, off2 = make([5000, 0, 2000], 264, 136, torch.bfloat16, seed=14)
    want = (mm.grouped_forward(x, w, off_t), mm.grouped_backward_weight(dy, x, off_t, dtype=torch.float32))
    want2 = (mm.grouped_forward(x2, w2, off2_t), mm.grouped_backward_weight(dy2, x2, off2_t, dtype=torch.float32))
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        got = (mm.grouped_forward(x, w, off_t, stream=one), mm.grouped_backward_weight(dy, x, off_t, dtype=torch.float32, stream=one))
        got2 = (mm.grouped_forward(x2, w2, off2_t, stream=two),
                mm.grouped_backward_weight(dy2, x2, off2_t, dtype=torch.float32, stream=two))
        torch.cuda.synchronize()
        for a, b in zip(want + want2, got + got2):
            assert torch.equal(a, b)
