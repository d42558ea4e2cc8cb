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
