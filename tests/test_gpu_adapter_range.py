"""Adapters in float16 whose low-rank values v = scale * x a^T lie outside float16's range, against 64 bits.

Tolerance, beyond that of test_gpu_adapter.py: v enters the second product as two float16 numbers, times a power of two
that takes the largest of the row's 32 neighbouring values into 2^14 .. 2^15.  Two numbers leave h^2 |v| of a value
(h = 2^-11) or, where the second is subnormal, half of its spacing 2^-24, which relative to the largest is
2^-25 / 2^14 = 2^-39.  The sums of 32 ranks are added one after the other: rank / 32 additions more."""
import pytest
import torch

import dispatch_fp8_grouped_amd as mm
from test_gpu_adapter import check as check_in_type, make

pytestmark = pytest.mark.gpu


def check(s, y):
    x, w = s["x"].double(), s["w"].double()
    k, rank = w.shape[1], s["a"].shape[1]
    eps, tiny = torch.finfo(y.dtype).eps, torch.finfo(y.dtype).smallest_normal * torch.finfo(y.dtype).eps
    wt = w.t().contiguous()
    want, bound = x @ wt, k * 2.0 ** -24 * (x.abs() @ wt.abs())
    off = s["offsets"].tolist()
    for r, i in enumerate(s["adapter"].tolist()):
        if i < 0:
            continue
        m = slice(off[r], off[r + 1])
        at, bt, sc = s["a"][i].double().t().contiguous(), s["b"][i].double().t().contiguous(), s["scales"][i].double()
        v, sv = x[m] @ at * sc, x[m].abs() @ at.abs() * sc.abs()
        largest = (v.abs() + (k + 1) * 2.0 ** -24 * sv).max(dim=1, keepdim=True).values
        dv = (k + 1) * 2.0 ** -24 * sv + (eps / 2) ** 2 * v.abs() + 2.0 ** -39 * largest
        sums = (v.abs() + dv) @ bt.abs()
        want[m] += v @ bt
        bound[m] += dv @ bt.abs() + (2 * rank + rank / 32 + 1) * 2.0 ** -24 * 1.01 * sums
        bound[m] += (rank / 32 + 1) * 2.0 ** -24 * 1.01 * (x[m].abs() @ wt.abs() + sums)
    bound = bound + eps / 2 * (want.abs() + bound) + tiny / 2
    assert (want.abs() < 65000).all()                      # an ordinary result
    assert torch.isfinite(y).all(), f"{int((~torch.isfinite(y)).sum())} of {y.numel()} values"
    d = (y.double() - want).abs()
    assert (d <= bound).all(), f"worst excess {(d - bound).max().item():.3g}, {int((d > bound).sum())} values"


# bounds, adapters, rows, n, k, rank: a row, rows with an adapter each, many column blocks of few requests (the forms of
# few rows), and more rows than those take
SHAPES = [([0, 1], [0], 1, 136, 264, 24),
          ([0, 1, 2], [1, 0], 2, 520, 1544, 256),
          (list(range(65)), [i % 4 for i in range(64)], 64, 264, 200, 16),
          ([0, 90, 91, 200], [0, 1, 3], 256, 4104, 136, 72),
          ([5, 100, 101, 290, 300], [1, 2, 0, 3], 310, 264, 136, 40),
          ([0, 2000, 5000], [0, 1], 5000, 2056, 136, 64)]


@pytest.mark.parametrize("bounds,adapter,rows,n,k,rank", SHAPES)
def test_values_beyond_float16(bounds, adapter, rows, n, k, rank):
    print(f"[case] {rows} {n} {k} {rank}", flush=True)
    s = make(bounds, adapter, rows, n, k, rank, 4, torch.float16, seed=rank)
    s["w"].mul_(2.0 ** -6)
    # v of 1e6, 1e-7, 1e-30 and 1: b takes the results back to ordinary numbers where float16 has such a b
    s["scales"] = torch.tensor([1e6, -1e-7, 1e-30, 1.0], device="cuda")
    s["b"][0].mul_(2.0 ** -9)
    s["b"][1].mul_(2.0 ** 12)
    check(s, mm.adapter_forward(**s))


@pytest.mark.parametrize("rows", [3, 70, 300])
def test_large_and_small_values_in_one_row(rows):
    """Ranks whose values differ by ten orders of magnitude, with a b that evens them out."""
    s = make([0, rows], [0], rows, 136, 264, 64, 1, torch.float16, seed=rows)
    step = 2.0 ** torch.arange(-12, 12, 24 / 64, device="cuda").double()
    s["a"] = (s["a"].double() * step[None, :, None] * 2.0 ** -4).half()
    s["b"] = (s["b"].double() / step[None, None, :] * 2.0 ** -2).half()
    s["scales"][0] = 4e4
    check(s, mm.adapter_forward(**s))


def test_an_infinite_value_stays_in_its_row():
    s = make([0, 3, 9], [0, 1], 9, 136, 264, 16, 2, torch.float16, seed=3)
    clean = mm.adapter_forward(**s)
    s["x"][4] = 60000.0
    s["scales"][1] = 1e38
    y = mm.adapter_forward(**s)
    assert torch.equal(y[:3], clean[:3])
    assert not torch.isfinite(y[4]).any()


def test_large_scales_in_both_types():
    """The inputs of test_large_values_in_float16: v reaches 1.7e7.  float16 rounds what the definition gives, infinite or
    not; in bfloat16 everything is a number."""
    s = make([0, 2, 4], [0, -1], 4, 16, 16, 8, 1, torch.float16, seed=24)
    s["scales"][:] = 3e7
    x, w, a, b = (s[n].double() for n in "xwab")
    want = x @ w.t().contiguous()
    want[:2] += x[:2] @ a[0].t().contiguous() * 3e7 @ b[0].t().contiguous()
    y = mm.adapter_forward(**s)
    beyond = want.abs() >= 65520
    assert torch.equal(torch.isinf(y), beyond) and torch.equal(y[beyond].double().sign(), want[beyond].sign())
    t = {k: (v.bfloat16() if v.dtype == torch.float16 else v) for k, v in s.items()}
    check_in_type(t, mm.adapter_forward(**t))
