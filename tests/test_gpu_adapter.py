"""Adapter projections against the plain computation in 64 bits.

Tolerance.  S1, Sv, S2 are the sums of the magnitudes of the terms of x w^T, of x a^T and of v b^T, in 64 bits.
fp32 sums are off by at most (terms) * 2^-24 of them.  v enters the second product as two 16-bit numbers: after
the first, at most h |v| is left over (h = eps / 2, half a step); the second leaves h of that, so h^2 |v|, and in
float16 at most half of the smallest subnormal.  The output adds one rounding, h."""
import pytest
import torch

import dispatch_fp8_grouped_amd as mm

pytestmark = pytest.mark.gpu

KINDS = {"bf16": torch.bfloat16, "fp16": torch.float16}


def make(bounds, adapter, rows, n, k, rank, adapters, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)
    return dict(x=normal(rows, k), w=normal(n, k, std=0.05), a=normal(adapters, rank, k, std=0.05),
                b=normal(adapters, n, rank, std=0.3), scales=torch.rand(adapters, generator=g, device="cuda") * 3 - 1,
                offsets=torch.tensor(bounds, dtype=torch.int32, device="cuda"),
                adapter=torch.tensor(adapter, dtype=torch.int32, device="cuda"))


def check(s, y, rows=None):
    x, w = s["x"].double(), s["w"].double()
    n, k, rank, dt = w.shape[0], w.shape[1], s["a"].shape[1], y.dtype
    eps, tiny = torch.finfo(dt).eps, torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
    wt = w.t().contiguous()
    want, bound = x @ wt, k * 2.0 ** -24 * (x.abs() @ wt.abs())
    off, ad = s["offsets"].tolist(), s["adapter"].tolist()
    for r, i in enumerate(ad):
        if not 0 <= i < s["a"].shape[0]:
            continue
        m = slice(off[r], off[r + 1])
        at, bt, sc = s["a"][i].double().t().contiguous(), s["b"][i].double().t().contiguous(), s["scales"][i].double()
        v, sv = x[m] @ at * sc, x[m].abs() @ at.abs() * sc.abs()
        dv = (k + 1) * 2.0 ** -24 * sv + (eps / 2) ** 2 * v.abs() + tiny / 2
        want[m] += v @ bt
        bound[m] += dv @ bt.abs() + 2 * rank * 2.0 ** -24 * ((v.abs() + dv) @ bt.abs()) * 1.01
        # the adapter's 2 rank terms are added onto the shared sum, each addition rounding a partial sum of at most S1 + S2
        bound[m] += 2 * rank * 2.0 ** -24 * (x[m].abs() @ wt.abs()) * 1.01
        bound[m] += 2.0 ** -24 * (want[m].abs() + bound[m])       # or, with few rows, its own sum added to it
    bound = bound + eps / 2 * (want.abs() + bound) + tiny / 2
    sel = slice(None) if rows is None else rows
    d = (y.double() - want)[sel].abs()
    assert (d <= bound[sel]).all(), f"worst excess {(d - bound[sel]).max().item():.3g}"


# bounds of the requests, their adapters, rows, n, k, rank, adapters
CASES = [
    ([0, 1], [0], 1, 8, 8, 8, 1),
    ([0, 1], [2], 1, 1000, 520, 32, 4),
    ([0, 5, 5, 9, 20], [1, 0, -1, 1], 20, 136, 264, 16, 3),
    (list(range(65)), [i % 7 - 1 for i in range(64)], 64, 520, 200, 24, 6),
    (list(range(0, 300, 3)), [(i * 5) % 11 - 1 for i in range(99)], 300, 264, 136, 40, 10),
    ([3, 40, 140, 140, 300], [0, 1, 0, 2], 333, 328, 328, 64, 3),       # rows of no request before and behind
    ([0, 700, 1500], [1, 1], 1500, 264, 192, 128, 2),
    ([0, 130, 131, 400], [0, 1, 2], 400, 72, 1032, 256, 3),
    ([0], [], 50, 136, 72, 8, 1),                                        # no request at all
    ([0, 17, 34, 51], [-1, -1, -1], 51, 136, 72, 8, 1),
    ([0, 1], [1], 1, 2056, 2048, 48, 2),                                 # long contractions, split between work-groups
    ([0, 3, 60, 61], [0, 1, 1], 61, 1032, 4104, 128, 2),
    ([0, 255], [0], 256, 392, 1544, 16, 1),
    ([0, 250, 257], [0, 1], 257, 392, 1544, 16, 2),                      # just too many rows for that
    ([0, 1000, 1001, 5000, 5100], [0, 1, 2, 0], 5131, 2056, 520, 24, 3),  # the large tiles
    ([0, 4000, 9000], [1, 0], 9000, 4104, 136, 72, 2),
    # few rows: many column blocks of few requests, many requests of high rank, more than four adapters to 16 rows
    ([0, 256], [1], 256, 1032, 2056, 256, 2),
    ([0, 90, 91, 200], [0, -1, 1], 200, 2056, 1032, 72, 2),
    (list(range(0, 257, 2)), [i % 33 - 1 for i in range(128)], 256, 264, 1544, 136, 32),
    ([0, 2, 4, 6, 8, 10, 12, 14, 16, 40], [0, 1, 2, 3, 4, 5, 6, 7, 0], 40, 4104, 520, 32, 8),
]


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_64_bits(case, kind):
    print(f"[case] {case} {kind}", flush=True)
    s = make(*CASES[case], KINDS[kind], seed=case)
    check(s, mm.adapter_forward(**s))


def test_more_requests_than_one_batch_of_the_search_holds():
    n = 1000
    s = make(list(range(n + 1)), [(i * 37) % 60 - 1 for i in range(n)], n, 72, 136, 16, 59, torch.bfloat16, seed=20)
    check(s, mm.adapter_forward(**s))
    s = make([min(i // 2, 1500) for i in range(4097)], [i % 5 for i in range(4096)], 1600, 40, 48, 8, 5, torch.bfloat16,
             seed=21)
    check(s, mm.adapter_forward(**s))


def test_one_requests_infinities_reach_no_other_row():
    s = make([0, 3, 10, 40, 41, 200], [0, 1, 2, 1, 0], 200, 136, 264, 16, 3, torch.bfloat16, seed=22)
    clean = mm.adapter_forward(**s)
    s["b"][1], s["a"][2, 0, 0] = float("inf"), float("nan")
    s["x"][41] = float("nan")
    y = mm.adapter_forward(**s)
    same = torch.ones(200, dtype=torch.bool, device="cuda")
    same[3:41] = False                                     # requests 1, 2 and 3
    same[41] = False
    assert torch.equal(y[same], clean[same])
    assert not torch.isfinite(y[3:41]).any() and torch.isnan(y[41]).all()


def test_workspace_contents_do_not_matter_and_out_is_used():
    s = make([0, 9, 30, 64], [1, -1, 0], 70, 136, 136, 24, 2, torch.float16, seed=23)
    want = mm.adapter_forward(**s)
    ws = torch.full((mm.mega_moe_adapter_workspace_bytes(70, 136, 136, 24, 3),), 0xFF, dtype=torch.uint8, device="cuda")
    y = torch.full_like(want, float("nan"))
    assert mm.adapter_forward(**s, out=y, workspace=ws) is y
    assert torch.equal(y, want)
    with pytest.raises(mm.MegaMoEError) as e:
        mm.adapter_forward(**s, workspace=ws[:-16])
    assert e.value.code == mm.ERR_WORKSPACE_TOO_SMALL
    with pytest.raises(ValueError):
        mm.adapter_forward(**{**s, "scales": s["scales"].double()})
    with pytest.raises(ValueError):
        mm.adapter_forward(**{**s, "x": s["x"].t()})


def test_large_values_in_float16():
    """Beyond 65504 the low-rank value is infinite in float16, and stays so; in bfloat16 it is a number."""
    s = make([0, 2, 4], [0, -1], 4, 16, 16, 8, 1, torch.float16, seed=24)
    s["scales"][:] = 3e7
    y = mm.adapter_forward(**s)
    assert not torch.isfinite(y[:2]).any() and torch.isfinite(y[2:]).all()
    t = {k: (v.bfloat16() if v.dtype == torch.float16 else v) for k, v in s.items()}
    check(t, mm.adapter_forward(**t))


def test_broken_ids_and_offsets_latch_the_status():
    s = make([0, 5, 9, 20], [0, 1, 2], 20, 72, 64, 8, 3, torch.bfloat16, seed=25)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    check(s, mm.adapter_forward(**s, status=st))
    assert st.item() == 0
    s["adapter"] = torch.tensor([-2, 3, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    check(s, mm.adapter_forward(**s, status=st))            # as if none had an adapter
    assert st.item() == mm.STATUS_BAD_EXPERT_ID
    s["adapter"] = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    for bad in ([0, 9, 5, 20], [-1, 5, 9, 20], [0, 5, 9, 21]):
        st.zero_()
        s["offsets"] = torch.tensor(bad, dtype=torch.int32, device="cuda")
        mm.adapter_forward(**s, status=st)
        assert st.item() == mm.STATUS_BAD_LAYOUT, bad


def test_repeat_other_stream_and_graph_replay_give_the_same_bits():
    s = make([0, 30, 31, 200, 290], [0, 1, -1, 1], 300, 264, 392, 32, 2, torch.bfloat16, seed=26)
    want = mm.adapter_forward(**s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mm.adapter_forward(**s, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    # two graphs, each with the workspace of its own call
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for g in graphs:
        with torch.cuda.graph(g):
            outs.append(mm.adapter_forward(**s))
    for i in range(3):
        s["x"].mul_(-1.5)
        s["adapter"].copy_(torch.tensor([i % 2, -1, 1, 0], dtype=torch.int32, device="cuda"))
        for g, o in zip(graphs, outs):
            o.fill_(5.0)
            g.replay()
        torch.cuda.synchronize()
        eager = mm.adapter_forward(**s)
        for o in outs:
            assert torch.equal(o, eager), i


def test_rows_past_32_bit_offsets():
    rows, n, k, rank = 540_000, 4104, 16, 8
    g = torch.Generator(device="cuda").manual_seed(31)
    x = torch.randn(rows, k, generator=g, device="cuda").bfloat16()
    w = torch.randn(n, k, generator=g, device="cuda").bfloat16()
    a = torch.randn(2, rank, k, generator=g, device="cuda").bfloat16()
    b = torch.randn(2, n, rank, generator=g, device="cuda").bfloat16()
    scales = torch.tensor([0.5, -2.0], device="cuda")
    off = torch.tensor([0, 300_001, 530_000, rows], dtype=torch.int32, device="cuda")
    which = torch.tensor([1, -1, 0], dtype=torch.int32, device="cuda")
    y = mm.adapter_forward(x, w, a, b, scales, off, which)
    assert y.numel() > 2 ** 31
    for i, m in ((1, slice(0, 200)), (1, slice(299_900, 300_001)), (-1, slice(300_001, 300_200)), (-1, slice(529_900, 530_000)),
                 (0, slice(530_000, 530_200)), (0, slice(rows - 100, rows))):
        check(dict(x=x[m], w=w, a=a, b=b, scales=scales, offsets=torch.tensor([0, m.stop - m.start]), adapter=torch.tensor([i])),
              y[m])
