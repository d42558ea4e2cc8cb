"""The router against a plain implementation in 64 bits, row by row: choices equal, weights and gradients within
the rounding of their type.

Tolerance.  Kernel and reference compute in fp64: each value carries at most a few fp64 roundings per operation,
and exp's argument is off by 2^-53 of at most some hundreds, together below 1e-12 of the terms' magnitude.  What
is stored is rounded to fp32 (2^-24 relative) and, for 16-bit gradients, once more (eps / 2)."""
import math

import numpy as np
import pytest
import torch

import dispatch_fp8_grouped_amd as mm

pytestmark = pytest.mark.gpu

KINDS = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
LARGEST = float(np.finfo(np.float32).max)


def scores_of(row, score):
    """Scores of one token's logits (floats), 0 where masked, and the mask."""
    live = [not (math.isnan(v) or v == -math.inf) for v in row]
    x = [min(v, LARGEST) if ok else -math.inf for v, ok in zip(row, live)]
    if score == "sigmoid":
        return [0.0 if not ok else (1.0 / (1.0 + math.exp(-v)) if v > -700 else 0.0) for v, ok in zip(x, live)], live, x
    if not any(live):
        return [0.0] * len(row), live, x
    top = max(x)
    e = [math.exp(v - top) if ok else 0.0 for v, ok in zip(x, live)]
    total = math.fsum(e)
    return [v / total for v in e], live, x


def route_row(row, k, bias, score, groups, kept, group_top, renorm, scale):
    s, live, x = scores_of(row, score)
    n = len(row)
    rank = list(x)
    if bias is not None:
        rank = [a + b for a, b in zip(s, bias)]
        live = [ok and r > -math.inf for ok, r in zip(live, rank)]
    ok = list(live)
    if groups > 1:
        worth_of = rank if bias is not None or group_top == 1 else s
        size = n // groups
        worth = []
        for g in range(groups):
            best = sorted((worth_of[e] for e in range(g * size, (g + 1) * size) if live[e]), reverse=True)[:group_top]
            worth.append(sum(best) if best else -math.inf)
        keep = sorted((g for g in range(groups) if worth[g] > -math.inf or
                       any(live[g * size:(g + 1) * size])), key=lambda g: (-worth[g], g))[:kept]
        ok = [o and e // size in keep for e, o in enumerate(ok)]
    idx = sorted((e for e in range(n) if ok[e]), key=lambda e: (-rank[e], e))[:k]
    w = [s[e] for e in idx]
    if renorm and score == "softmax" and idx:          # the softmax's own sum cancels
        w, _, _ = scores_of([row[e] for e in idx], score)
    elif renorm:
        total = math.fsum(w)
        w = [v / total if total > 0 else 0.0 for v in w]
    pad = k - len(idx)
    return idx + [-1] * pad, [v * scale for v in w] + [0.0] * pad


def check_forward(logits, k, bias=None, score="softmax", groups=1, kept=1, group_top=1, renorm=True, scale=1.0,
                  rows=slice(None)):
    idx, w = mm.router_topk(logits, k, bias=bias, score=score, num_groups=groups, topk_groups=kept, group_top=group_top,
                            renormalize=renorm, scale=scale)
    assert idx.dtype == torch.int64 and w.dtype == torch.float32
    sample, i_s, w_s = logits[rows].double().cpu().tolist(), idx[rows], w[rows]
    b = None if bias is None else bias.double().cpu().tolist()
    want = [route_row(r, k, b, score, groups, kept, group_top, renorm, scale) for r in sample]
    got_i, got_w = i_s.cpu().tolist(), w_s.double().cpu().numpy()
    for t, (wi, ww) in enumerate(want):
        assert got_i[t] == wi, (t, got_i[t], wi)
    ww = np.array([x[1] for x in want], dtype=np.float64).reshape(got_w.shape)
    assert (np.abs(got_w - ww) <= np.abs(ww) * (2.0 ** -24 + 1e-12) + 2.0 ** -149).all()
    return idx, w


def logits_of(t, e, kind="fp32", seed=0, std=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(t, e, generator=g, device="cuda") * std).to(KINDS[kind])


# tokens, experts, k, groups, kept: one expert, one token, odd counts, groups that share no power of two, the
# limits of each lane width (64, 128, 256, 512, 1024, 4096)
SIZES = [(1, 1, 1, 1, 1), (3, 7, 7, 1, 1), (5, 64, 8, 8, 3), (6, 60, 6, 5, 2), (9, 65, 4, 1, 1), (4, 128, 8, 4, 4),
         (7, 129, 3, 3, 1), (33, 256, 8, 8, 4), (2, 384, 12, 64, 20), (5, 510, 16, 6, 2), (3, 1000, 10, 8, 5),
         (2, 1024, 64, 16, 2), (2, 4096, 8, 64, 8), (2, 3001, 5, 1, 1)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("t,e,k,groups,kept", SIZES)
def test_choice_and_weights(t, e, k, groups, kept, kind, score):
    print(f"[case] {t} {e} {k} {groups} {kept} {kind} {score}", flush=True)
    x = logits_of(t, e, kind, seed=e)
    bias = torch.randn(e, device="cuda", generator=torch.Generator(device="cuda").manual_seed(e)) * 0.1
    for renorm in (True, False):
        check_forward(x, k, None, score, 1, 1, 1, renorm)
        check_forward(x, k, bias, score, groups, kept, 2, renorm, 2.5)
        check_forward(x, k, None, score, groups, kept, 2, renorm)
        check_forward(x, k, bias, score, groups, kept, 1, renorm)
        check_forward(x, k, None, score, groups, kept, 1, renorm, 0.5)


# many tokens: a quarter wave each.  The last tokens of a wave and of a work-group are missing
MANY = [(4097, 7, 7, 1, 1), (4099, 60, 6, 5, 2), (5000, 64, 16, 16, 3), (4110, 100, 4, 4, 2), (6001, 128, 8, 8, 3),
        (4096, 200, 12, 1, 1), (9001, 256, 8, 8, 4)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("t,e,k,groups,kept", MANY)
def test_many_tokens(t, e, k, groups, kept, kind, score):
    print(f"[case] {t} {e} {k} {groups} {kept} {kind} {score}", flush=True)
    x = logits_of(t, e, kind, seed=e + 5)
    x[3] = float("-inf")
    x[t - 2, ::2] = float("nan")
    x[t - 1] = 0.5
    rows = torch.tensor([*range(12), *range(t // 2, t // 2 + 9), *range(t - 25, t)], device="cuda")
    bias = torch.randn(e, device="cuda", generator=torch.Generator(device="cuda").manual_seed(e)) * 0.1
    g = torch.randn(t, k, device="cuda", generator=torch.Generator(device="cuda").manual_seed(9))
    for renorm in (True, False):
        check_forward(x, k, None, score, 1, 1, 1, renorm, rows=rows)
        check_forward(x, k, bias, score, groups, kept, 2, renorm, 2.5, rows=rows)
        check_forward(x, k, bias, score, 1, 1, 1, renorm, rows=rows)
        idx, _ = check_forward(x, k, None, score, groups, kept, 2, renorm, rows=rows)
        idx[4, 0] = -1
        idx[5, k - 1] = idx[5, 0]
        check_backward(x, idx, g, score, renorm, 2.5, sel=rows)


def test_ties_go_to_the_lowest_expert():
    x = torch.randint(-2, 3, (200, 96), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).float()
    for kind in KINDS.values():
        for groups, kept, top in ((1, 1, 1), (8, 3, 1), (8, 3, 2), (6, 2, 2)):
            check_forward(x.to(kind), 10, None, "softmax", groups, kept, top)
            check_forward(x.to(kind), 10, torch.zeros(96, device="cuda"), "sigmoid", groups, kept, top)
    zeros = torch.zeros(2, 300, device="cuda")
    zeros[1, ::2] = -0.0                               # a negative zero ranks with zero
    idx, w = check_forward(zeros, 8)
    assert idx.tolist() == [list(range(8))] * 2


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masks_infinities_and_lowest_values(score):
    x = logits_of(12, 80, seed=3)
    lowest = torch.finfo(torch.float32).min
    x[0] = float("-inf")                               # nothing to choose
    x[1] = float("nan")
    x[2] = float("-inf")
    x[2, 41] = 0.3                                     # fewer than k
    x[3, :79] = float("nan")
    x[4] = lowest                                      # masked by the type's lowest value: still numbers
    x[5, 3:] = lowest
    x[6, 7] = float("inf")
    x[7, 70:] = float("inf")
    x[8] = float("inf")
    x[9, ::2] = float("-inf")
    x[10, :40] = float("-inf")                         # whole groups without an expert
    x[11] = LARGEST
    bias = torch.randn(80, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4)) * 0.2
    for groups, kept, top in ((1, 1, 1), (8, 2, 2), (8, 8, 1), (5, 3, 2)):
        for renorm in (True, False):
            check_forward(x, 6, None, score, groups, kept, top, renorm)
            check_forward(x, 6, bias, score, groups, kept, top, renorm)
    odd = bias.clone()
    odd[5], odd[20], odd[33], odd[60:] = float("nan"), float("inf"), float("-inf"), float("-inf")
    check_forward(x[9:], 6, odd, score, 8, 3, 1)
    check_forward(x[9:], 6, odd, score)


def test_padded_tokens_and_more_tokens_than_one_pass_of_the_grid_row():
    x = logits_of(700, 40, "bf16", seed=5)
    x[650:] = float("-inf")
    idx, w = check_forward(x, 4)
    assert (idx[650:] == -1).all() and (w[650:] == 0).all()


def reference_backward(g, row, idx, score, renorm, scale):
    """dlogits of one token and the magnitude of its terms, from the Jacobian of the scores."""
    s, live, x = scores_of(row, score)
    n = len(row)
    G, cnt = [0.0] * n, [0] * n
    for gv, e in zip(g, idx):
        if 0 <= e < n:
            G[e] += gv
            cnt[e] += 1
    if renorm and score == "softmax":                  # the softmax's own sum cancels: over the named experts alone
        s, _, _ = scores_of([v if c else -math.inf for v, c in zip(row, cnt)], score)
    if renorm:
        S = math.fsum(cnt[i] * s[i] for i in range(n))
        gs = math.fsum(G[i] * s[i] for i in range(n) if cnt[i])
        ds = [(G[i] - cnt[i] * gs / S) / S * scale if S > 0 and cnt[i] else 0.0 for i in range(n)]
        mag = [(abs(G[i]) + cnt[i] * math.fsum(abs(G[j]) * s[j] for j in range(n) if cnt[j]) / S) / S * abs(scale)
               if S > 0 and cnt[i] else 0.0 for i in range(n)]
    else:
        ds = [v * scale for v in G]
        mag = [abs(v) for v in ds]
    if score == "sigmoid":
        return [d * v * (1 - v) if ok else 0.0 for d, v, ok in zip(ds, s, live)], \
               [m * v for m, v in zip(mag, s)]
    dot = math.fsum(d * v for d, v in zip(ds, s) if v)
    amp = math.fsum(m * v for m, v in zip(mag, s) if v)
    return [v * (d - dot) if v else 0.0 for d, v in zip(ds, s)], [v * (m + amp) for m, v in zip(mag, s)]


def check_backward(logits, idx, g, score, renorm, scale=1.0, sel=slice(None)):
    d = mm.router_backward(g, logits, idx, score=score, renormalize=renorm, scale=scale)
    assert d.dtype == logits.dtype and d.shape == logits.shape
    rows, ids, gs = (v[sel].double().cpu().tolist() for v in (logits, idx, g))
    ids = [[int(e) for e in r] for r in ids]
    got, eps = d[sel].double().cpu().numpy(), torch.finfo(logits.dtype).eps
    tiny = torch.finfo(logits.dtype).smallest_normal * eps
    for t in range(len(rows)):
        want, mag = map(np.array, reference_backward(gs[t], rows[t], ids[t], score, renorm, scale))
        bound = np.abs(want) * (eps / 2 + 2.0 ** -23) + mag * 1e-12 + tiny
        assert (np.abs(got[t] - want) <= bound).all(), (t, np.abs(got[t] - want).max())


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("t,e,k,groups,kept", SIZES)
def test_gradient(t, e, k, groups, kept, kind):
    print(f"[case] {t} {e} {k} {kind}", flush=True)
    x = logits_of(t, e, kind, seed=e + 1)
    g = torch.randn(t, k, device="cuda", generator=torch.Generator(device="cuda").manual_seed(9))
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            idx, _ = mm.router_topk(x, k, score=score, num_groups=groups, topk_groups=kept)
            check_backward(x, idx, g, score, renorm, 2.5)


def test_gradient_with_masks_repeated_and_absent_experts():
    x = logits_of(8, 50, seed=6)
    x[0] = float("-inf")
    x[1, 10:] = float("nan")
    x[2, 4] = float("inf")
    x[3] = torch.finfo(torch.float32).min
    idx = torch.randint(0, 50, (8, 6), device="cuda", generator=torch.Generator(device="cuda").manual_seed(7))
    idx[4] = torch.tensor([3, 3, 3, 9, 3, 9])
    idx[5] = torch.tensor([-1, 8, -1, 50, 2 ** 40, -2 ** 40])
    idx[6] = -1
    g = torch.randn(8, 6, device="cuda", generator=torch.Generator(device="cuda").manual_seed(8))
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            check_backward(x, idx, g, score, renorm)


def test_gradient_against_differences():
    """Central differences of sum(g * weights) in 64 bits; their own error is h^2 times the third derivative."""
    x = logits_of(3, 20, seed=10)
    g = torch.randn(3, 5, device="cuda", generator=torch.Generator(device="cuda").manual_seed(11))
    h = 2.0 ** -10
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            idx, _ = mm.router_topk(x, 5, score=score)
            d = mm.router_backward(g, x, idx, score=score, renormalize=renorm).cpu()
            for t in range(3):
                def loss(row):
                    s, _, _ = scores_of(row, score)
                    w = [s[e] for e in idx[t].tolist()]
                    total = sum(w) if renorm else 1.0
                    return sum(a * b / total for a, b in zip(g[t].tolist(), w))
                row = x[t].double().tolist()
                for e in range(20):
                    up, dn = list(row), list(row)
                    up[e] += h
                    dn[e] -= h
                    diff = (loss(up) - loss(dn)) / (2 * h)
                    assert abs(diff - d[t, e].item()) <= 1e-5, (score, renorm, t, e)


# ------------------------------------------------------------------------------------------- ordering
def check_order(idx, experts, first=0):
    offsets, order, slot = mm.group_by_expert(idx, experts, first_expert=first)
    flat = idx.reshape(-1).cpu()
    local = torch.where((flat >= first) & (flat < first + experts), flat - first, torch.full_like(flat, experts))
    key, by = local.sort(stable=True)
    total = int((local < experts).sum())
    count = torch.bincount(local, minlength=experts + 1)[:experts]
    want_off = torch.cat([torch.zeros(1, dtype=torch.int64), count.cumsum(0)]).int()
    assert torch.equal(offsets.cpu(), want_off)
    want_order = torch.where(torch.arange(flat.numel()) < total, by, torch.full_like(by, -1)).int()
    assert torch.equal(order.cpu(), want_order)
    want_slot = torch.full_like(flat, -1)
    want_slot[by[:total]] = torch.arange(total)
    assert slot.shape == idx.shape and torch.equal(slot.cpu().reshape(-1), want_slot.int())


@pytest.mark.parametrize("pairs", [0, 1, 63, 64, 65, 1000, 8192, 8193, 40000, 300007])
@pytest.mark.parametrize("experts", [1, 2, 32, 257, 512, 513, 4096])
def test_ordering(pairs, experts):
    g = torch.Generator(device="cuda").manual_seed(pairs + experts)
    print(f"[case] {pairs} {experts}", flush=True)
    check_order(torch.randint(0, experts, (pairs,), device="cuda", generator=g), experts)
    # a rank's share of more experts, with absent ones and ids far outside
    far = torch.randint(-2, 3 * experts, (pairs,), device="cuda", generator=g)
    far[:pairs // 7] = 2 ** 40
    far[pairs // 7:pairs // 5] = -2 ** 63
    check_order(far, experts, first=experts)


def test_ordering_with_one_expert_taking_everything_and_none():
    idx = torch.full((5000, 4), 6, dtype=torch.int64, device="cuda")
    check_order(idx, 16)
    check_order(idx, 4)
    check_order(idx, 4, first=3)


def test_repeat_other_stream_and_graph_replay_give_the_same_bits():
    x = logits_of(3000, 256, seed=12)
    bias = torch.randn(256, device="cuda") * 0.1
    g = torch.randn(3000, 8, device="cuda")

    def run(stream=None):
        idx, w = mm.router_topk(x, 8, bias=bias, score="sigmoid", num_groups=8, topk_groups=4, group_top=2, stream=stream)
        return (idx, w, *mm.group_by_expert(idx, 256, stream=stream),
                mm.router_backward(g, x, idx, score="sigmoid", stream=stream),
                mm.router_backward(g, x, idx, renormalize=False, stream=stream))
    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(side)
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for i in range(3):
        x.mul_(-1.25)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(run(), got):
            assert torch.equal(a, b), i


def test_a_layer_from_its_router_to_its_gradients():
    """Router, ordering, grouped products and their gradients as one expert layer: outputs and every gradient
    against the same layer in 64 bits with torch's autograd.

    Tolerance: the steps between the products round to bf16 (rows, activations, outputs, their gradients), each
    half a step of 2^-8 relative to values that enter the next sum; over the handful of roundings on any path,
    errors stay below 8 * 2^-8 of the largest magnitude in the tensor."""
    T, H, I, E, K = 96, 128, 64, 8, 2
    gen = torch.Generator(device="cuda").manual_seed(21)
    x = torch.randn(T, H, generator=gen, device="cuda").bfloat16()
    w1 = (torch.randn(E, I, H, generator=gen, device="cuda") * 0.1).bfloat16()
    w2 = (torch.randn(E, H, I, generator=gen, device="cuda") * 0.1).bfloat16()
    logits = torch.randn(T, E, generator=gen, device="cuda")
    dy = torch.randn(T, H, generator=gen, device="cuda").bfloat16()

    idx, wt = mm.router_topk(logits, K)
    offsets, order, slot = mm.group_by_expert(idx, E)
    token = (order // K).long()
    rows = x[token]
    h = mm.grouped_forward(rows, w1, offsets)
    a = torch.relu(h)
    o = mm.grouped_forward(a, w2, offsets)
    y = (o[slot.long()].float() * wt.unsqueeze(-1)).sum(1)
    # backward
    do = (dy[token].float() * wt.reshape(-1)[order.long()].unsqueeze(-1)).bfloat16()
    dwt = (o[slot.long()].float() * dy.float().unsqueeze(1)).sum(-1)
    dw2 = mm.grouped_backward_weight(do, a, offsets, dtype=torch.float32)
    dh = torch.where(h > 0, mm.grouped_backward_rows(do, w2, offsets), torch.zeros_like(h))
    dw1 = mm.grouped_backward_weight(dh, rows, offsets, dtype=torch.float32)
    drows = mm.grouped_backward_rows(dh, w1, offsets)
    dx = drows[slot.long()].float().sum(1)
    dlogits = mm.router_backward(dwt, logits, idx)

    X, W1, W2, L = (t.double().cpu().requires_grad_() for t in (x, w1, w2, logits))
    keep = (h.cpu() > 0)                     # the same branches of relu as the rounded path took
    place = slot.cpu().long()
    probs = torch.softmax(L, -1).gather(1, idx.cpu())
    probs = probs / probs.sum(-1, keepdim=True)
    want = torch.zeros(T, H, dtype=torch.float64)
    for k in range(K):
        e = idx.cpu()[:, k]
        hk = (W1[e] @ X.unsqueeze(-1)).squeeze(-1) * keep[place[:, k]]
        want = want + probs[:, k:k + 1] * (W2[e] @ hk.unsqueeze(-1)).squeeze(-1)
    want.backward(dy.double().cpu())
    for name, got, ref in (("y", y, want.detach()), ("dx", dx, X.grad), ("dw1", dw1, W1.grad), ("dw2", dw2, W2.grad),
                           ("dlogits", dlogits, L.grad)):
        d = (got.double().cpu() - ref).abs().max().item()
        assert d <= 8 * 2.0 ** -8 * ref.abs().max().item(), (name, d, ref.abs().max().item())


def test_sixteen_bit_ranks():
    """bf16 and fp16 ranks: every sign, infinities beside the largest finite numbers, subnormal numbers, both
    zeros and NaN of both signs; 16 lanes and 64 lanes per token."""
    for kind in (torch.bfloat16, torch.float16):
        bits = torch.arange(65536, device="cuda", dtype=torch.int32).to(torch.int16)
        values = bits.view(kind)
        order = torch.randperm(65536, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
        mixed = values[order].view(256, 256)
        for t in (256, 4096):
            x = mixed.repeat(t // 256, 1).contiguous()
            print(f"[case] {kind} {t}", flush=True)
            idx, _ = mm.router_topk(x, 16, score="sigmoid", renormalize=False)
            wide = x.double()
            wide = torch.where(torch.isnan(wide), torch.full_like(wide, -float("inf")), wide)
            want = torch.sort(wide, dim=1, descending=True, stable=True)[1][:, :16]
            assert torch.equal(idx.cpu(), want.cpu())


def test_ordering_of_many_pairs_for_a_wave():
    """More pairs than the ordering's waves hold in registers."""
    g = torch.Generator(device="cuda").manual_seed(4)
    check_order(torch.randint(-1, 300, ((1 << 20) + 777,), device="cuda", generator=g), 257)


@pytest.mark.parametrize("pairs", [1023, 1024, 1025, 9 * 1024 + 1, 32767, 32768, 32769])
def test_ordering_at_the_edges_of_its_work_groups(pairs):
    g = torch.Generator(device="cuda").manual_seed(pairs)
    for experts in (3, 512, 513):
        check_order(torch.randint(-1, experts + 2, (pairs,), device="cuda", generator=g), experts)


def test_logits_past_32_bit_offsets():
    """More than 2^31 logits: the last tokens as a call for them alone gives them."""
    t, e = 8_500_000, 256
    x = torch.empty(t, e, device="cuda", dtype=torch.bfloat16)
    g = torch.Generator(device="cuda").manual_seed(21)
    for r in range(0, t, 500_000):
        x[r:r + 500_000] = torch.randn(min(500_000, t - r), e, generator=g, device="cuda").bfloat16()
    idx, w = mm.router_topk(x, 4)
    for s in (slice(0, 5000), slice(t - 5000, t)):
        some = x[s].contiguous()
        i, v = mm.router_topk(some, 4)
        assert torch.equal(i, idx[s]) and torch.equal(v, w[s])
    dw = torch.randn(t, 4, generator=g, device="cuda")
    d = mm.router_backward(dw, x, idx)
    for s in (slice(0, 5000), slice(t - 5000, t)):
        assert torch.equal(d[s], mm.router_backward(dw[s].contiguous(), x[s].contiguous(), idx[s].contiguous()))
