"""The norm, SwiGLU and 8-bit rows as a program uses them: on streams, in graphs, beside autograd, with guarded buffers,
and one after the other around the layer and through the experts' gradients."""
import pytest
import torch

import dispatch_fp8_grouped_amd as mm
import row_refs as ref
from test_gpu_ops_bounds import Guarded, check_all

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
CODE = {BF16: mm.BF16, FP16: mm.FP16, FP32: mm.FP32}


def case(rows=300, hidden=264, inter=136, seed=0):
    """Arguments of every call, made anew."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=BF16):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)
    off = torch.tensor([0, rows // 3, rows], dtype=torch.int32, device="cuda")
    return {
        "rms_norm": lambda: dict(x=normal(rows, hidden), weight=normal(hidden), residual=normal(rows, hidden, dtype=FP32), quantize="both"),
        "rms_norm_backward": lambda: dict(dy=normal(rows, hidden), h=normal(rows, hidden), weight=normal(hidden), dresidual=normal(rows, hidden)),
        "rms_norm_backward (8 bits)": lambda: dict(dy=normal(rows, hidden), h=mm.quantize_rows(normal(rows, hidden)), weight=normal(hidden)),
        "quantize_rows": lambda: dict(x=normal(rows, hidden)),
        "dequantize_rows": lambda: dict(zip(("codes", "scales"), mm.quantize_rows(normal(rows, hidden)))),
        "swiglu": lambda: dict(gate_up=normal(rows, 2 * inter), checkpoint=True, offsets=off.clone()),
        "swiglu_backward": lambda: dict(dact=normal(rows, inter), gate_up=mm.swiglu(normal(rows, 2 * inter), checkpoint=True)[1],
                                        recompute=True, offsets=off.clone()),
        "grouped_backward_weight": lambda: dict(dy=normal(rows, hidden), x=mm.quantize_rows(normal(rows, inter)), offsets=off.clone()),
        # rows that are restored first
        "grouped_backward_weight (restored)": lambda: dict(dy=normal(rows, hidden), x=mm.quantize_rows(normal(rows, 8)), offsets=off.clone()),
    }


CALLS = ("rms_norm", "rms_norm_backward", "rms_norm_backward (8 bits)", "quantize_rows", "dequantize_rows", "swiglu", "swiglu_backward",
         "grouped_backward_weight", "grouped_backward_weight (restored)")


def call(name):
    return getattr(mm, name.split()[0])


def flat(y):
    if isinstance(y, torch.Tensor):
        return [y]
    return [t for v in (y or ()) if v is not None for t in flat(v)]


def tensors(args):
    return [t for v in args.values() for t in (v if isinstance(v, tuple) else (v,)) if isinstance(t, torch.Tensor)]


@pytest.mark.parametrize("name", CALLS)
def test_repeated_calls_give_the_same_bits(name):
    args = case(rows=3000)[name]()
    want = [t.clone() for t in flat(call(name)(**args))]
    for _ in range(3):
        for a, b in zip(want, flat(call(name)(**args))):
            assert torch.equal(a, b)


@pytest.mark.parametrize("name", CALLS)
def test_tensors_dropped_after_a_call_on_another_stream_stay_until_it_has_read_them(name):
    """The call waits behind other work of its stream while its inputs are dropped and their sizes asked for again."""
    side = torch.cuda.Stream()
    want = [t.clone() for t in flat(call(name)(**case()[name]()))]
    args = case()[name]()
    sizes = [(v.shape, v.dtype) for v in tensors(args)]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    got = flat(call(name)(**args, stream=side))
    del args
    again = [torch.zeros(s, dtype=d, device="cuda") for s, d in sizes for _ in range(4)]
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    del again


@pytest.mark.parametrize("name", CALLS)
def test_two_calls_at_once(name):
    """On two streams, different inputs: each has its own outputs and workspace."""
    one, two = case(rows=2000, seed=1)[name](), case(rows=2000, seed=2)[name]()
    want = [[t.clone() for t in flat(call(name)(**a))] for a in (one, two)]
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    got = [[], []]
    for _ in range(4):
        got[0].append(flat(call(name)(**one, stream=s)))
        got[1].append(flat(call(name)(**two, stream=t)))
    torch.cuda.synchronize()
    for w, rounds in zip(want, got):
        for outs in rounds:
            for a, b in zip(w, outs):
                assert torch.equal(a, b)


@pytest.mark.parametrize("name", CALLS)
def test_a_captured_call(name):
    """Replayed with new inputs in the same places, eager work in between."""
    args = case(rows=700)[name]()
    want = [t.clone() for t in flat(call(name)(**args))]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = flat(call(name)(**args, stream=torch.cuda.current_stream()))
    for seed in (0, 5, 6):
        for old, new in zip(tensors(args), tensors(case(rows=700, seed=seed)[name]())):
            old.copy_(new)
        want = [t.clone() for t in flat(call(name)(**args))]
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)


@pytest.mark.parametrize("name,inputs", [("rms_norm", ("x", "weight", "residual")), ("swiglu", ("gate_up",)), ("dequantize_rows", ("scales",))])
def test_a_gradient_is_not_lost_silently(name, inputs):
    args = case()[name]()
    want = flat(call(name)(**args))
    for key in inputs:
        with_grad = {**args, key: args[key].clone().requires_grad_()}
        got = flat(call(name)(**with_grad))
        for a, b in zip(want, got):
            assert torch.equal(a, b)
        with pytest.raises(RuntimeError, match=f"{name} records no autograd graph"):
            got[0].float().sum().backward()
        with torch.no_grad():
            assert not any(t.requires_grad for t in flat(call(name)(**with_grad)))
    if name == "rms_norm":                             # h is the weight's no more than the sum is
        y, h, _ = mm.rms_norm(**{**args, "weight": args["weight"].clone().requires_grad_()})
        assert y.requires_grad and not h.requires_grad


@pytest.mark.parametrize("name,key", [("rms_norm_backward", "dy"), ("rms_norm_backward", "weight"), ("swiglu_backward", "dact"),
                                      ("quantize_rows", "x"), ("grouped_backward_weight", "dy")])
def test_gradients_and_8_bit_rows_are_plain_tensors(name, key):
    args = case()[name]()
    args[key].requires_grad_()
    assert not any(t.requires_grad for t in flat(call(name)(**args)))


def test_refusals():
    x, w = torch.randn(4, 64, device="cuda"), torch.randn(64, device="cuda")
    half, codes = x.to(BF16), mm.quantize_rows(x)
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    for bad in (lambda: mm.rms_norm(half, w.to(FP16)), lambda: mm.rms_norm(half, w, residual=x.to(FP16)), lambda: mm.rms_norm(half, w[:32]),
                lambda: mm.rms_norm(half, w, residual=half[:2]), lambda: mm.rms_norm(half, w, dtype=FP32), lambda: mm.rms_norm(x, w, residual=x, dtype=BF16),
                lambda: mm.rms_norm(x.t(), w), lambda: mm.rms_norm(x, w, dtype=torch.float64), lambda: mm.rms_norm(half, w, quantize=2),
                lambda: mm.rms_norm_backward(half, x.to(FP16), w), lambda: mm.rms_norm_backward(half, half, w, dresidual=x),
                lambda: mm.rms_norm_backward(half, codes, w, dresidual=x.to(FP16)), lambda: mm.rms_norm_backward(half[:2], codes, w),
                lambda: mm.rms_norm_backward(half, (codes[0], codes[1][:2]), w), lambda: mm.quantize_rows(x.double()), lambda: mm.quantize_rows(x[:, ::2]),
                lambda: mm.dequantize_rows(codes[0], codes[1].double()), lambda: mm.dequantize_rows(codes[0].view(torch.int8), codes[1]),
                lambda: mm.swiglu(x), lambda: mm.swiglu(half[:, :63].contiguous()), lambda: mm.swiglu(half, offsets=off.long()),
                lambda: mm.swiglu(half, offsets=off[:1]), lambda: mm.swiglu(half[0]), lambda: mm.swiglu_backward(half, half),
                lambda: mm.swiglu_backward(half[:, :32].contiguous(), half.to(FP16)), lambda: mm.swiglu_backward(half[:, :32].contiguous(), codes),
                lambda: mm.grouped_backward_weight(x, codes, off), lambda: mm.grouped_backward_weight(half[:2], codes, off),
                lambda: mm.grouped_backward_weight(half, (codes[0], codes[1][:2]), off),
                lambda: mm.grouped_backward_weight(half, codes, off, out=torch.empty(1, 64, 64, device="cuda", dtype=FP16))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: mm.rms_norm(half, w, eps=-1.0), lambda: mm.rms_norm(half, w, eps=float("nan")),
                lambda: mm.rms_norm(torch.zeros(2, 16385, device="cuda"), torch.zeros(16385, device="cuda")),
                lambda: mm.quantize_rows(torch.zeros(2, 65537, device="cuda"))):
        with pytest.raises(mm.MegaMoEError):
            bad()
    # what is added to lies beside its inputs
    pool = torch.zeros(1 << 16, device="cuda")
    out, scales = pool[:64 * 64].view(1, 64, 64), pool[64 * 64 - 4:64 * 64].view(4, 1)
    with pytest.raises(ValueError, match="out overlaps"):
        mm.grouped_backward_weight(half, (codes[0], scales), off, out=out, accumulate=True)


# ------------------------------------------------------------------ outputs between guard bytes
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("rows,hidden", [(1, 1), (3, 7), (17, 128), (5, 129), (9, 1000), (6, 2049), (4, 7168), (3, 12289), (2, 16384), (700, 24)])
def test_norm_writes_its_outputs_alone(rows, hidden, dtype):
    print(f"[case] {rows} {hidden} {dtype}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(hidden)
    x, res, dy = ((torch.randn(rows, hidden, generator=g, device="cuda")).to(dtype) for _ in range(3))
    w = torch.randn(hidden, generator=g, device="cuda")
    nb = -(-hidden // 128)
    h, y, codes = Guarded.of((rows, hidden), dtype), Guarded.of((rows, hidden), dtype), Guarded(rows * hidden)
    scales = Guarded.of((rows, nb), FP32)
    mm.mega_moe_rms_norm(x, res, w, h.ptr(), y.ptr(), codes.ptr(), scales.ptr(), rows, hidden, 1e-6, CODE[dtype], CODE[dtype], mm.FP32)
    check_all(h=h, y=y, codes=codes, scales=scales)
    want = mm.rms_norm(x, w, residual=res, quantize="both")
    assert torch.equal(y.tensor(), want[0]) and torch.equal(h.tensor(), want[1])
    assert torch.equal(codes.bytes().view(rows, hidden), want[2][0]) and torch.equal(scales.tensor(), want[2][1])
    need = mm.mega_moe_norm_workspace_bytes(rows, hidden)
    for scale in (None, scales.ptr()):
        dx, dw, ws = Guarded.of((rows, hidden), dtype), Guarded.of((hidden,), FP32), Guarded(need, fill=0xFF)
        mm.mega_moe_rms_norm_backward(dy, codes.ptr() if scale else h.ptr(), scale, w, res, dx.ptr(), dw.ptr(), rows, hidden, 1e-6, CODE[dtype],
                                      CODE[dtype], mm.FP32, ws.ptr(), need)
        check_all(dx=dx, dw=dw, workspace=ws)
        given = (codes.bytes().view(rows, hidden), scales.tensor()) if scale else h.tensor()
        want = mm.rms_norm_backward(dy, given, w, dresidual=res)
        assert torch.equal(dx.tensor(), want[0]) and torch.equal(dw.tensor(), want[1])


@pytest.mark.parametrize("rows,inter", [(1, 1), (3, 7), (5, 127), (4, 136), (9, 1000), (3, 8192), (1000, 3)])
def test_swiglu_and_8_bit_rows_write_their_outputs_alone(rows, inter):
    print(f"[case] {rows} {inter}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(inter)
    nb = -(-inter // 128)
    for dtype in (BF16, FP16):
        gate_up, dact = (torch.randn(rows, c * inter, generator=g, device="cuda").to(dtype) for c in (2, 1))
        act, codes, scales = Guarded.of((rows, inter), dtype), Guarded(rows * 2 * inter), Guarded.of((rows, 2 * nb), FP32)
        mm.mega_moe_swiglu(gate_up, act.ptr(), codes.ptr(), scales.ptr(), None, 0, rows, inter, CODE[dtype])
        again, d = Guarded.of((rows, inter), dtype), Guarded.of((rows, 2 * inter), dtype)
        mm.mega_moe_swiglu_backward(dact, codes.ptr(), scales.ptr(), d.ptr(), again.ptr(), None, 0, rows, inter, CODE[dtype])
        check_all(act=act, codes=codes, scales=scales, again=again, d=d)
        want, kept = mm.swiglu(gate_up, checkpoint=True)
        assert torch.equal(act.tensor(), want) and torch.equal(codes.bytes().view(rows, 2 * inter), kept[0])
        assert torch.equal(d.tensor(), mm.swiglu_backward(dact, kept)[0])
        for out in (BF16, FP16, FP32):
            y = Guarded.of((rows, inter), out)
            mm.mega_moe_quantize_rows(dact, codes.ptr(), scales.ptr(), rows, inter, CODE[dtype])
            mm.mega_moe_dequantize_rows(codes.ptr(), scales.ptr(), y.ptr(), rows, inter, CODE[out])
            check_all(y=y, codes=codes, scales=scales)
            assert torch.equal(y.tensor(), mm.dequantize_rows(*mm.quantize_rows(dact), dtype=out))


# counts of the groups, n, k; the offsets leave rows before and behind
@pytest.mark.parametrize("counts,n,k", [([1], 8, 8), ([1], 8, 16), ([3, 0, 17, 16, 15, 1], 264, 520), ([255, 0, 257, 300], 520, 264),
                                        ([9000, 0, 3, 4000], 136, 264), ([700, 0, 0, 900], 2056, 2312), ([33, 31], 8200, 8200)])
def test_weight_gradient_writes_its_outputs_alone(counts, n, k):
    print(f"[case] {counts} {n} {k}", flush=True)
    offsets = [5]
    for c in counts:
        offsets.append(offsets[-1] + c)
    rows, groups = offsets[-1] + 7, len(counts)
    g = torch.Generator(device="cuda").manual_seed(n)
    x, dy = (torch.randn(rows, c, generator=g, device="cuda").to(BF16) for c in (k, n))
    # the inputs end where their allocations' guard bytes begin
    codes, scales = Guarded(rows * k), Guarded.of((rows, -(-k // 128)), FP32)
    mm.mega_moe_quantize_rows(x, codes.ptr(), scales.ptr(), rows, k, mm.BF16)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    status = Guarded.of((1,), torch.int32, fill=0)
    need = mm.mega_moe_grouped_codes_workspace_bytes(rows, n, k, groups)
    for kind, code, add in ((BF16, mm.BF16, False), (FP32, mm.FP32, False), (FP32, mm.FP32, True)):
        dw, ws = Guarded.of((groups, n, k), kind, fill=0), Guarded(need)
        mm.mega_moe_grouped_backward_weight_codes(dy, codes.ptr(), scales.ptr(), off, dw.ptr(), rows, n, k, groups, mm.BF16, code, add,
                                                  ws.ptr() if need else None, need, status.ptr())
        check_all(dw=dw, workspace=ws, status=status, codes=codes, scales=scales)
        assert torch.isfinite(dw.tensor()).all() and status.tensor().item() == 0


@pytest.mark.parametrize("offsets", [[0, 10, 5, 60], [-3, 10, 30, 60], [0, 10, 30, 61], [0, 10, 2 ** 31 - 1, 60], [2 ** 31 - 1, -2 ** 31, 0, 0],
                                     [0, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1], [-2 ** 31] * 4, [2 ** 31 - 1] * 4])
@pytest.mark.parametrize("n,k", [(72, 8), (72, 64), (1032, 264)])
def test_weight_gradient_with_broken_offsets(offsets, n, k):
    print(f"[case] {offsets} {n} {k}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(n)
    dy = torch.randn(60, n, generator=g, device="cuda").to(BF16)
    codes, scales = mm.quantize_rows(torch.randn(60, k, generator=g, device="cuda"))
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    status, dw = Guarded.of((1,), torch.int32, fill=0), Guarded.of((3, n, k), FP32, fill=0)
    need = mm.mega_moe_grouped_codes_workspace_bytes(60, n, k, 3)
    ws = Guarded(need)
    mm.mega_moe_grouped_backward_weight_codes(dy, codes, scales, off, dw.ptr(), 60, n, k, 3, mm.BF16, mm.FP32, False, ws.ptr() if need else None, need,
                                              status.ptr())
    check_all(dw=dw, status=status, workspace=ws)
    assert status.tensor().item() == mm.STATUS_BAD_LAYOUT and torch.isfinite(dw.tensor()).all()


# ------------------------------------------------------------------ runs of them together
def test_the_norm_feeds_the_router_and_the_layer():
    """A decode-sized step: residual and norm, router on its 16-bit rows, the fused layer on its 8-bit rows, against the
    layer's oracle on the same codes, with the layer's own bound."""
    import numpy as np

    import oracle
    from inputs import MoEShape, make_inputs, to_numpy
    shape = MoEShape("normed", 2, 48, 512, 256, 16, 8, 4, 64, seed=71)
    inp = make_inputs(shape, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    dims = (shape.num_shards, shape.max_tokens_per_shard, shape.hidden)
    x, residual = (torch.randn(dims, generator=g, device="cuda").to(BF16) for _ in range(2))
    w = 1 + 0.1 * torch.randn(shape.hidden, generator=g, device="cuda")
    router = torch.randn(shape.num_experts, shape.hidden, generator=g, device="cuda").to(BF16) * 0.05
    y, h, (codes, scales) = mm.rms_norm(x, w, residual=residual, quantize="both")
    idx, weights = mm.router_topk((y @ router.t()).contiguous(), shape.topk)
    inp.update(x=codes, x_sf=scales, topk_idx=idx, topk_weights=weights)
    moe = mm.MegaMoE.from_shape(shape)
    out = moe(inp)
    torch.cuda.synchronize()
    assert moe.status() == 0
    want = oracle.forward(to_numpy(inp), shape.num_experts, shape.num_local_experts, shape.local_rank, shape.block_m)["y"]
    assert np.abs(out.double().cpu().numpy() - want).max() <= 2e-2 * np.abs(want).max() + 1e-3
    moe.close()
    assert torch.equal(h, (x.float() + residual.float()).to(BF16))


def test_a_trained_layer_from_its_norm_to_its_gradients():
    """Norm, router, ordering, grouped products and SwiGLU, with gate_up and the rows kept in 8 bits, and every gradient back,
    against the same in 64 bits from the same kept values.

    Tolerance: the steps round to bf16, each half a step of 2^-8 relative to values that enter the next sum; over the
    dozen roundings on any path errors stay below 12 * 2^-8 of the largest magnitude in the tensor."""
    T, H, I, E, K = 96, 256, 136, 8, 2
    g = torch.Generator(device="cuda").manual_seed(31)
    x, res, dout = (torch.randn(T, H, generator=g, device="cuda").bfloat16() for _ in range(3))
    wn = 1 + 0.1 * torch.randn(H, generator=g, device="cuda")
    w1 = (torch.randn(E, 2 * I, H, generator=g, device="cuda") * 0.1).bfloat16()
    w2 = (torch.randn(E, H, I, generator=g, device="cuda") * 0.1).bfloat16()
    logits = torch.randn(T, E, generator=g, device="cuda")

    y, h, rows8 = mm.rms_norm(x, wn, residual=res, quantize="both")
    h8 = mm.quantize_rows(h)
    idx, wt = mm.router_topk(logits, K)
    offsets, order, slot = mm.group_by_expert(idx, E)
    token = (order // K).long()
    rows, kept_rows = y[token], (rows8[0][token], rows8[1][token])
    gate_up = mm.grouped_forward(rows, w1, offsets)
    act, kept = mm.swiglu(gate_up, checkpoint=True, offsets=offsets)
    o = mm.grouped_forward(act, w2, offsets)
    out = h.float() + (o[slot.long()].float() * wt.unsqueeze(-1)).sum(1)
    do = (dout[token].float() * wt.reshape(-1)[order.long()].unsqueeze(-1)).bfloat16()
    dact = mm.grouped_backward_rows(do, w2, offsets)
    dgate_up, act_again = mm.swiglu_backward(dact, kept, recompute=True, offsets=offsets)
    dw2 = mm.grouped_backward_weight(do, act_again, offsets, dtype=FP32)
    dw1 = mm.grouped_backward_weight(dgate_up, kept_rows, offsets, dtype=FP32)
    drows = mm.grouped_backward_rows(dgate_up, w1, offsets)
    dy = drows[slot.long()].float().sum(1).bfloat16()
    dx, dwn = mm.rms_norm_backward(dy, h8, wn, dresidual=dout)

    def near(name, got, want):
        d = (got.double() - want).abs().max().item()
        assert d <= 12 * 2.0 ** -8 * want.abs().max().item(), (name, d, want.abs().max().item())
    d64 = lambda t: t.double()      # noqa: E731
    Y, V, _ = ref.norm(x, res, wn, 1e-6)
    R, place = Y[token], slot.long()
    bounds = offsets.tolist()
    spans = [slice(a, b) for a, b in zip(bounds, bounds[1:])]
    G = torch.cat([R[s] @ d64(w1[e]).t().contiguous() for e, s in enumerate(spans)])
    A = ref.swiglu(*G.chunk(2, 1))
    O = torch.cat([A[s] @ d64(w2[e]).t().contiguous() for e, s in enumerate(spans)])
    near("out", out, V + (O[place] * d64(wt).unsqueeze(-1)).sum(1))
    DO = d64(dout)[token] * d64(wt).reshape(-1)[order.long()].unsqueeze(-1)
    DA = torch.cat([DO[s] @ d64(w2[e]) for e, s in enumerate(spans)])
    gate, up = ref.decode(kept[0].view(-1, 2, I), kept[1].view(-1, 2, 2)).unbind(1)
    DG = torch.cat(ref.swiglu_backward(DA, gate, up), 1)
    A8, X8 = ref.swiglu(gate, up), ref.decode(*kept_rows)
    near("dw2", dw2, torch.stack([DO[s].t().contiguous() @ A8[s].contiguous() for s in spans]))
    near("dw1", dw1, torch.stack([DG[s].t().contiguous() @ X8[s].contiguous() for s in spans]))
    DR = torch.cat([DG[s] @ d64(w1[e]) for e, s in enumerate(spans)])
    DX, DWN, _, _ = ref.norm_backward(DR[place].sum(1), ref.decode(*h8), wn, dout, 1e-6)
    near("dx", dx, DX)
    near("dweight", dwn, DWN)


def test_kept_values_cost_a_sixteenth():
    """What keeping 8 bits means: every kept value is within 2^-4 of itself, or 2^-10 of its block's scale, and a weight
    gradient from kept rows is that close to the one from the rows themselves, term by term."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x, dy = (torch.randn(500, c, generator=g, device="cuda").to(BF16) for c in (256, 264))
    off = torch.tensor([0, 200, 500], dtype=torch.int32, device="cuda")
    kept = mm.quantize_rows(x)
    half = torch.maximum(2.0 ** -4 * x.double().abs(), 2.0 ** -10 * kept[1].double().repeat_interleave(128, 1))
    assert ((ref.decode(*kept) - x.double()).abs() <= half).all()
    a, b = mm.grouped_backward_weight(dy, kept, off, dtype=FP32), mm.grouped_backward_weight(dy, x, off, dtype=FP32)
    for e, s in enumerate((slice(0, 200), slice(200, 500))):
        d = dy[s].double().abs().t().contiguous()
        bound = d @ half[s] + 2 * 301 * ref.U * (d @ (x[s].double().abs() + half[s]))
        assert ((a[e].double() - b[e].double()).abs() <= bound).all()


def test_quantize_is_read_as_a_truth_value():
    x, w = torch.randn(3, 128, device="cuda"), torch.ones(128, device="cuda")
    for alone in (True, 1):
        y, _, rows8 = mm.rms_norm(x, w, quantize=alone)
        assert y is None and rows8 is not None
    for none in (False, 0):
        y, _, rows8 = mm.rms_norm(x, w, quantize=none)
        assert y is not None and rows8 is None
