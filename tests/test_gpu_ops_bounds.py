"""The operators write their outputs and the workspace of the size that they ask for, and not a byte beside them:
every buffer lies between guard bytes, at exactly the queried size, and goes to the C-named entry points."""
import pytest
import torch

import dispatch_fp8_grouped_amd as mm

pytestmark = pytest.mark.gpu

GUARD, MARK = 65536, 0xA5


class Guarded:
    """A buffer of `nbytes` bytes inside a larger one whose other bytes hold a mark."""

    def __init__(self, nbytes, fill=0x5C):
        self.all = torch.full((GUARD + nbytes + GUARD,), MARK, dtype=torch.uint8, device="cuda")
        self.nbytes = nbytes
        self.all[GUARD:GUARD + nbytes] = fill

    @classmethod
    def of(cls, shape, dtype, **kw):
        n = 1
        for d in shape:
            n *= d
        g = cls(n * torch.empty(0, dtype=dtype).element_size(), **kw)
        g.shape, g.dtype = shape, dtype
        return g

    def bytes(self):
        return self.all[GUARD:GUARD + self.nbytes]

    def tensor(self):
        return self.bytes().view(self.dtype).view(self.shape)

    def ptr(self):
        return self.all.data_ptr() + GUARD

    def check(self, name):
        before, behind = self.all[:GUARD], self.all[GUARD + self.nbytes:]
        assert (before == MARK).all(), f"{name}: {int((before != MARK).sum())} bytes written before it"
        assert (behind == MARK).all(), f"{name}: {int((behind != MARK).sum())} bytes written behind it"


def check_all(**buffers):
    torch.cuda.synchronize()
    for name, g in buffers.items():
        g.check(name)


@pytest.mark.parametrize("pairs", [0, 1, 1000, 8193, 40000])
@pytest.mark.parametrize("experts", [1, 512, 513, 4096])
def test_ordering(pairs, experts):
    print(f"[case] {pairs} {experts}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(pairs + experts)
    idx = torch.randint(-1, experts + 3, (pairs,), device="cuda", generator=gen)
    need = mm.mega_moe_group_workspace_bytes(pairs, experts)
    ws = Guarded(need)
    offsets, order, slot = (Guarded.of((n,), torch.int32) for n in (experts + 1, pairs, pairs))
    mm.mega_moe_group_by_expert(idx, pairs, 0, experts, offsets.ptr(), order.ptr(), slot.ptr(), ws.ptr(), need)
    check_all(workspace=ws, offsets=offsets, order=order, slot=slot)
    local = (idx >= 0) & (idx < experts)
    count = torch.bincount(idx[local], minlength=experts)
    want = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), count.cumsum(0)]).int()
    assert torch.equal(offsets.tensor(), want)
    assert torch.equal(slot.tensor() >= 0, local)


BF16 = torch.bfloat16
# counts of the groups, n, k: the shapes of few and of many rows, split sums, streams of tiles, odd edges
GROUPED = [([1], 8, 8), ([3, 0, 17, 16, 15, 1], 264, 520), ([255, 0, 257, 300], 520, 264), ([9000, 0, 3, 4000], 136, 264),
           ([700, 0, 0, 900], 2056, 2312), ([3000, 17, 0, 900], 4104, 136), ([3], 520, 8200)]


def rows_of(rows, cols, seed):
    return torch.randn(rows, cols, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(BF16)


def grouped_calls(offsets, rows, n, k, groups):
    """The three products into guarded buffers, which are returned; `offsets` may be broken."""
    x, dy = rows_of(rows, k, 1), rows_of(rows, n, 2)
    w = rows_of(groups * n, k, 3)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    status = Guarded.of((1,), torch.int32, fill=0)
    y, dx = Guarded.of((rows, n), BF16), Guarded.of((rows, k), BF16)
    mm.mega_moe_grouped_forward(x, w, off, y.ptr(), rows, n, k, groups, mm.BF16, status.ptr())
    mm.mega_moe_grouped_backward_rows(dy, w, off, dx.ptr(), rows, n, k, groups, mm.BF16, status.ptr())
    check_all(y=y, dx=dx, status=status)
    need = mm.mega_moe_grouped_weight_workspace_bytes(rows, n, k, groups)
    for kind, code, add in ((BF16, mm.BF16, False), (torch.float32, mm.FP32, False), (torch.float32, mm.FP32, True)):
        dw, ws = Guarded.of((groups, n, k), kind, fill=0), Guarded(need)
        mm.mega_moe_grouped_backward_weight(dy, x, off, dw.ptr(), rows, n, k, groups, mm.BF16, code, add,
                                            ws.ptr() if need else None, need, status.ptr())
        check_all(dw=dw, workspace=ws, status=status)
        assert torch.isfinite(dw.tensor()).all()
    return y, dx, status


@pytest.mark.parametrize("counts,n,k", GROUPED)
def test_grouped_products(counts, n, k):
    print(f"[case] {counts} {n} {k}", flush=True)
    before, behind, total = 5, 7, sum(counts)
    offsets = [before]
    for c in counts:
        offsets.append(offsets[-1] + c)
    y, dx, status = grouped_calls(offsets, before + total + behind, n, k, len(counts))
    assert status.tensor().item() == 0
    for g in (y, dx):                                  # rows of no group stay as they were
        rows = g.tensor().view(torch.uint8)
        assert (rows[:before] == 0x5C).all() and (rows[before + total:] == 0x5C).all()
        assert torch.isfinite(g.tensor()[before:before + total]).all()


# decreasing pairs, entries below 0 and above the rows, every group with all rows
BROKEN = [[0, 10, 5, 60], [-3, 10, 30, 60], [0, 10, 30, 61], [0, 10, 2 ** 31 - 1, 60], [2 ** 31 - 1, -2 ** 31, 0, 0],
          [0, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1], [0, 60, 0, 60], [-2 ** 31] * 4, [2 ** 31 - 1] * 4]


@pytest.mark.parametrize("offsets", BROKEN)
@pytest.mark.parametrize("n,k", [(72, 64), (1032, 264)])
def test_grouped_products_with_broken_offsets(offsets, n, k):
    print(f"[case] {offsets} {n} {k}", flush=True)
    _, _, status = grouped_calls(offsets, 60, n, k, 3)
    assert status.tensor().item() == mm.STATUS_BAD_LAYOUT


def adapter_call(offsets, adapter, rows, n, k, rank, adapters, kind=BF16):
    def normal(*shape):
        return (torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(sum(shape)), device="cuda") * 0.1).to(kind)
    x, w, a, b = normal(rows, k), normal(n, k), normal(adapters, rank, k), normal(adapters, n, rank)
    scales = torch.ones(adapters, device="cuda")
    requests = len(adapter)
    need = mm.mega_moe_adapter_workspace_bytes(rows, n, k, rank, requests)
    y, ws, status = Guarded.of((rows, n), kind), Guarded(need, fill=0xFF), Guarded.of((1,), torch.int32, fill=0)
    mm.mega_moe_adapter_forward(x, w, a, b, scales, torch.tensor(offsets, dtype=torch.int32, device="cuda"),
                                torch.tensor(adapter, dtype=torch.int32, device="cuda"), y.ptr(), rows, n, k, rank, requests,
                                adapters, mm.BF16 if kind == BF16 else mm.FP16, ws.ptr(), need, status.ptr())
    check_all(y=y, workspace=ws, status=status)
    return y, status


@pytest.mark.parametrize("kind", [BF16, torch.float16])
@pytest.mark.parametrize("rows,requests,n,k,rank", [(1, 1, 8, 8, 8), (1, 1, 1000, 2056, 256), (64, 64, 520, 1544, 24),
                                                    (256, 3, 1032, 520, 72), (256, 128, 264, 136, 40), (257, 3, 264, 136, 16),
                                                    (1500, 700, 136, 264, 128), (5003, 5, 2056, 520, 24), (70, 0, 136, 72, 8)])
def test_adapters(rows, requests, n, k, rank, kind):
    print(f"[case] {rows} {requests} {n} {k} {rank} {kind}", flush=True)
    offsets = [rows * i // max(requests, 1) for i in range(requests + 1)]
    y, status = adapter_call(offsets, [i % 4 - 1 for i in range(requests)], rows, n, k, rank, 3, kind)
    assert status.tensor().item() == 0 and torch.isfinite(y.tensor()).all()


@pytest.mark.parametrize("offsets", BROKEN)
@pytest.mark.parametrize("rows", [60, 300])
def test_adapters_with_broken_offsets_and_ids(offsets, rows):
    print(f"[case] {offsets} {rows}", flush=True)
    offsets = [o if abs(o) > 100 else o * rows // 60 for o in offsets]
    _, status = adapter_call(offsets, [0, 1, 2], rows, 136, 264, 24, 3)
    assert status.tensor().item() == mm.STATUS_BAD_LAYOUT
    _, status = adapter_call(offsets, [-2, 2 ** 31 - 1, -2 ** 31], rows, 136, 264, 24, 3)
    assert status.tensor().item() == mm.STATUS_BAD_LAYOUT | mm.STATUS_BAD_EXPERT_ID


@pytest.mark.parametrize("kind,code", [(torch.float32, mm.FP32), (BF16, mm.BF16), (torch.float16, mm.FP16)])
@pytest.mark.parametrize("t,e,k,groups", [(1, 1, 1, 1), (3, 7, 7, 1), (33, 60, 6, 5), (4099, 60, 6, 5), (4097, 256, 8, 8),
                                          (5, 510, 16, 6), (2, 1001, 10, 7), (2, 3001, 5, 1), (3, 4096, 8, 64)])
def test_router(t, e, k, groups, kind, code):
    print(f"[case] {t} {e} {k} {groups} {kind}", flush=True)
    logits = rows_of(t, e, 4).to(kind)
    bias = rows_of(1, e, 5).float().reshape(-1)
    for score in (mm.SCORE_SOFTMAX, mm.SCORE_SIGMOID):
        for b, renorm in ((None, 1), (bias, 0)):
            cfg = mm.mega_moe_router_config(t, e, k, score, groups, max(1, groups // 2 + 1), 2, renorm, 1.5, code)
            idx, weights = Guarded.of((t, k), torch.int64), Guarded.of((t, k), torch.float32)
            mm.mega_moe_router_topk(cfg, logits, b, idx.ptr(), weights.ptr())
            dlogits = Guarded.of((t, e), kind)
            mm.mega_moe_router_backward(cfg, weights.tensor(), logits, idx.tensor(), dlogits.ptr())
            check_all(idx=idx, weights=weights, dlogits=dlogits)
            ids = idx.tensor()
            assert ((ids >= -1) & (ids < e)).all() and torch.isfinite(weights.tensor()).all()
            assert torch.isfinite(dlogits.tensor()).all()
