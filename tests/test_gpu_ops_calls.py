"""How the operators' Python calls treat the tensors and streams of their caller."""
import pytest
import torch

import dispatch_fp8_grouped_amd as mm

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def case(rows=300, n=264, k=136, groups=3, seed=0):
    """Arguments of every operator, made anew."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=BF16):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)
    off = torch.tensor([rows * i // groups for i in range(groups + 1)], dtype=torch.int32, device="cuda")
    idx = torch.randint(0, 32, (rows, 4), generator=g, device="cuda")
    return {
        "grouped_forward": lambda: dict(x=normal(rows, k), w=normal(groups, n, k), offsets=off.clone()),
        "grouped_backward_rows": lambda: dict(dy=normal(rows, n), w=normal(groups, n, k), offsets=off.clone()),
        "grouped_backward_weight": lambda: dict(dy=normal(rows, n), x=normal(rows, k), offsets=off.clone()),
        "router_topk": lambda: dict(logits=normal(rows, 32, dtype=torch.float32), topk=4,
                                    bias=normal(32, dtype=torch.float32)),
        "router_backward": lambda: dict(dweights=normal(rows, 4, dtype=torch.float32),
                                        logits=normal(rows, 32, dtype=torch.float32), topk_idx=idx.clone()),
        "group_by_expert": lambda: dict(topk_idx=idx.clone(), num_local_experts=32),
        "adapter_forward": lambda: dict(x=normal(rows, k), w=normal(n, k), a=normal(2, 16, k), b=normal(2, n, 16),
                                        scales=normal(2, dtype=torch.float32), offsets=off.clone(),
                                        adapter=torch.tensor([0, 1, -1], dtype=torch.int32, device="cuda")),
    }


OPERATORS = ("grouped_forward", "grouped_backward_rows", "grouped_backward_weight", "router_topk", "router_backward",
             "group_by_expert", "adapter_forward")


def outputs(y):
    return list(y) if isinstance(y, tuple) else [y]


@pytest.mark.parametrize("name", OPERATORS)
def test_tensors_dropped_after_a_call_on_another_stream_stay_until_it_has_read_them(name):
    """The call waits behind other work of its stream while its inputs are dropped and their sizes asked for again."""
    call, side = getattr(mm, name), torch.cuda.Stream()
    want = [t.clone() for t in outputs(call(**case()[name]()))]
    args = case()[name]()
    tensors = {k: v for k, v in args.items() if isinstance(v, torch.Tensor)}
    sizes = [(v.shape, v.dtype) for v in tensors.values()]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    got = outputs(call(**args, stream=side))
    del args, tensors
    again = [torch.zeros(s, dtype=d, device="cuda") for s, d in sizes for _ in range(4)]
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    del again


@pytest.mark.parametrize("name", OPERATORS)
def test_a_captured_call_with_its_stream_given(name):
    call, args = getattr(mm, name), case()[name]()
    want = [t.clone() for t in outputs(call(**args))]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = outputs(call(**args, stream=torch.cuda.current_stream()))
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)
    del args                                           # recorded on the capture's stream
    more = torch.zeros(1 << 20, device="cuda")
    torch.cuda.synchronize()
    del more, graph


@pytest.mark.parametrize("kind", [torch.float32, BF16, torch.float16])
@pytest.mark.parametrize("experts,topk", [(60, 3), (7, 5), (256, 8), (1001, 1)])
def test_slices_of_tokens_that_start_anywhere(experts, topk, kind):
    """Slices whose rows are no multiple of 16 bytes, bias and ids from the middle of a tensor."""
    g = torch.Generator(device="cuda").manual_seed(experts)
    logits = torch.randn(40, experts, generator=g, device="cuda").to(kind)
    bias = torch.randn(experts + 1, generator=g, device="cuda")[1:]
    dweights = torch.randn(40, topk, generator=g, device="cuda")
    side = torch.cuda.Stream()
    for score in ("softmax", "sigmoid"):
        whole = mm.router_topk(logits, topk, bias=bias.clone(), score=score)
        grads = mm.router_backward(dweights, logits, whole[0], score=score)
        torch.cuda.synchronize()
        for lo, hi, stream in ((1, 40, None), (3, 17, side), (39, 40, None), (40, 40, None)):
            idx, weights = mm.router_topk(logits[lo:hi], topk, bias=bias, score=score, stream=stream)
            torch.cuda.synchronize()
            assert torch.equal(idx, whole[0][lo:hi]) and torch.equal(weights, whole[1][lo:hi])
            d = mm.router_backward(dweights[lo:hi], logits[lo:hi], whole[0][lo:hi], score=score, stream=stream)
            some = mm.group_by_expert(whole[0][lo:hi], experts, stream=stream)
            torch.cuda.synchronize()
            assert torch.equal(d, grads[lo:hi])
            for a, b in zip(some, mm.group_by_expert(whole[0][lo:hi].clone(), experts)):
                assert torch.equal(a, b)


@pytest.mark.parametrize("name,inputs", [("grouped_forward", ("x", "w")), ("router_topk", ("logits",)),
                                         ("adapter_forward", ("x", "w", "a", "b", "scales"))])
def test_a_gradient_is_not_lost_silently(name, inputs):
    call, args = getattr(mm, name), case()[name]()
    want = outputs(call(**args))
    for key in inputs:
        with_grad = {**args, key: args[key].clone().requires_grad_()}
        got = outputs(call(**with_grad))
        for a, b in zip(want, got):
            assert torch.equal(a, b)
            assert b.requires_grad == b.is_floating_point()
        with pytest.raises(RuntimeError, match=f"{name} records no autograd graph"):
            got[-1].float().sum().backward()
        with torch.no_grad():
            assert not any(t.requires_grad for t in outputs(call(**with_grad)))
        if name != "router_topk":                      # into a buffer of the caller's: as it was
            out = torch.empty_like(want[0])
            assert call(**with_grad, out=out) is out and not out.requires_grad


@pytest.mark.parametrize("name,inputs", [("grouped_backward_rows", ("dy", "w")), ("grouped_backward_weight", ("dy", "x")),
                                         ("router_backward", ("dweights", "logits"))])
def test_gradients_are_plain_tensors(name, inputs):
    args = case()[name]()
    for key in inputs:
        args[key].requires_grad_()
    assert not getattr(mm, name)(**args).requires_grad


def test_numbers_beyond_32_bits_are_refused():
    logits = torch.randn(3, 32, device="cuda")
    idx = torch.randint(0, 32, (3, 4), device="cuda")
    wide = torch.empty(0, (1 << 32) + 16, dtype=BF16, device="cuda")
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    for call in (lambda: mm.router_topk(logits, (1 << 32) + 2), lambda: mm.router_topk(logits, 2, num_groups=(1 << 32) + 2),
                 lambda: mm.router_topk(logits, 2, num_groups=2, topk_groups=(1 << 32) + 1),
                 lambda: mm.router_topk(logits, 2, num_groups=2, group_top=(1 << 32) + 1),
                 lambda: mm.group_by_expert(idx, (1 << 32) + 8), lambda: mm.group_by_expert(idx, 8, first_expert=1 << 32),
                 lambda: mm.group_by_expert(idx, 8, first_expert=-(1 << 32)),
                 lambda: mm.grouped_backward_weight(torch.empty(0, 8, dtype=BF16, device="cuda"), wide, off)):
        with pytest.raises(ValueError, match="32-bit"):
            call()
    with pytest.raises(mm.MegaMoEError):               # within 32 bits the library refuses
        mm.group_by_expert(idx, 8, first_expert=-1)


def test_outputs_and_workspaces_apart_from_the_inputs():
    args = {n: f() for n, f in case(n=136).items()}
    pool = torch.zeros(1 << 20, dtype=BF16, device="cuda")

    def place(first, shape):
        return pool[first:first + shape[0] * shape[1]].view(shape)
    forward, rows, adapter = args["grouped_forward"], args["grouped_backward_rows"], args["adapter_forward"]
    with pytest.raises(ValueError, match="out overlaps"):
        mm.grouped_forward(**forward, out=forward["x"])
    with pytest.raises(ValueError, match="out overlaps"):
        mm.grouped_backward_rows(**rows, out=rows["dy"])
    with pytest.raises(ValueError, match="out overlaps"):
        mm.adapter_forward(**adapter, out=adapter["x"])
    # neighbours in one allocation are taken
    x, out = place(0, (300, 136)), place(300 * 136, (300, 136))
    x.copy_(forward["x"])
    want = mm.grouped_forward(**forward)
    assert torch.equal(mm.grouped_forward(x, forward["w"], forward["offsets"], out=out), want)
    with pytest.raises(ValueError, match="out overlaps"):
        mm.grouped_forward(x, forward["w"], forward["offsets"], out=place(299 * 136, (300, 136)))
    dy = place(0, (300, 136))
    with pytest.raises(ValueError, match="out overlaps"):
        mm.grouped_backward_weight(dy, forward["x"], forward["offsets"], accumulate=True,
                                   out=pool[136 * 299:136 * 299 + 2 * 3 * 136 * 136].view(torch.float32).view(3, 136, 136))
    need = mm.mega_moe_adapter_workspace_bytes(300, 136, 136, 16, 3)
    space = torch.empty(need + 300 * 136 * 2, dtype=torch.uint8, device="cuda")
    out = space[need:].view(BF16).view(300, 136)
    want = mm.adapter_forward(**adapter)
    assert torch.equal(mm.adapter_forward(**adapter, out=out, workspace=space[:need]), want)
    with pytest.raises(ValueError, match="overlaps"):
        mm.adapter_forward(**adapter, out=out, workspace=space)
    inside = space[:300 * 136 * 2].view(BF16).view(300, 136)
    with pytest.raises(ValueError, match="workspace overlaps"):
        mm.adapter_forward(**{**adapter, "x": inside}, workspace=space)
