"""The operators around the fused MoE layer, as measured workloads: products grouped by expert with ragged
rows (forward, and both gradients), the router that chooses and weighs the experts (forward, with the
ordering of the pairs by expert, and its gradient), and a projection shared by many requests that each
bring a low-rank adapter.

`run` computes a case with elementary torch operations in 32 bits (choices between near-equal scores in 64),
or, with `own` set, through dispatch_fp8_grouped_amd.  `exact` computes the same from the definition in 64
bits.  Row counts per expert and per request come from the case itself, so that `work` is exact; the values
come from the seed.
"""
import random

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_DEV = "cuda"


# ------------------------------------------------------------------------------------------- cases
def listed():
    def experts(name, direction, rows, n, k, e, split, rows_by="uniform", dtype="bf16", out="same"):
        return dict(name=name, op="experts", direction=direction, rows=rows, n=n, k=k, experts=e, split=split,
                    rows_by=rows_by, dtype=dtype, out=out)

    def router(name, direction, tokens, e, topk, score, dtype, bias=False, groups=1, kept=1, group_top=1,
               renormalize=True, scale=1.0, padded=0):
        return dict(name=name, op="router", direction=direction, tokens=tokens, experts=e, topk=topk, score=score,
                    dtype=dtype, bias=bias, groups=groups, kept=kept, group_top=group_top,
                    renormalize=renormalize, scale=scale, padded=padded)

    def adapter(name, rows, requests, n, k, rank, adapters, split, dtype="bf16"):
        return dict(name=name, op="adapter", rows=rows, requests=requests, n=n, k=k, rank=rank, adapters=adapters,
                    split=split, dtype=dtype)

    return [
        # the gate_up product of the prefill-shaped share: 32 experts, about 1024 rows each (matrix-bound)
        experts("experts_forward_prefill", "forward", 32768, 4096, 7168, 32, 11),
        # the down product of the decode-shaped share: about 32 rows an expert (the weights are streamed)
        experts("experts_forward_decode", "forward", 1024, 7168, 2048, 32, 12),
        # one token's eight rows, each for another expert: latency and weight streaming
        experts("experts_forward_token", "forward", 8, 4096, 7168, 32, 13, rows_by="distinct"),
        # fp16, sizes that fill no tile, few experts
        experts("experts_forward_odd", "forward", 1999, 1000, 2056, 10, 14, dtype="fp16"),
        # gradient of the rows through the mid-sized share's down weights
        experts("experts_backward_rows_mid", "backward_rows", 8192, 4096, 1536, 32, 15),
        # gradient of the gate_up weights under skewed routing, some experts without a row, fp32 out
        experts("experts_backward_weight_skewed", "backward_weight", 16384, 4096, 7168, 32, 16, rows_by="zipf",
                out="fp32"),
        # routing of a decode step: 1024 tokens, sigmoid scores, a balancing bias, 4 of 8 groups kept, padding rows
        router("router_decode", "forward", 1024, 256, 8, "sigmoid", "fp32", bias=True, groups=8, kept=4, group_top=2,
               scale=2.5, padded=24),
        # routing of a prefill step from bf16 logits (many equal ones), softmax
        router("router_prefill", "forward", 32768, 256, 8, "softmax", "bf16"),
        # the router's gradient in training, probabilities over all experts
        router("router_backward", "backward", 32768, 128, 8, "softmax", "fp32", renormalize=False),
        # one decode step of 64 requests, a row each, 24 adapters between them, through a shared gate_up weight
        adapter("adapter_decode", 64, 64, 4096, 7168, 16, 24, 17),
        # prompts of 12 requests at once
        adapter("adapter_prefill", 8192, 12, 4096, 7168, 64, 8, 18),
        # a single request's next token
        adapter("adapter_token", 1, 1, 7168, 2048, 32, 4, 19),
    ]


def _log_int(rng, lo, hi):
    """An integer spread over the logarithm of lo..hi."""
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    """A case of the listed ranges: 1 to 32768 rows, 8 to 8192 columns in steps of 8 (16-byte rows), 1 to 64
    experts; 1 to 32768 tokens over 8 to 512 routed experts; 1 to 8192 rows of 1 to 128 requests."""
    while True:
        op = rng.choice(["experts", "experts", "router", "adapter"])
        if op == "experts":
            direction = rng.choice(["forward", "backward_rows", "backward_weight"])
            case = dict(op=op, direction=direction, rows=_log_int(rng, 1, 32768), n=8 * _log_int(rng, 8, 1024),
                        k=8 * _log_int(rng, 8, 1024), experts=_log_int(rng, 1, 64), split=rng.randrange(1 << 30),
                        rows_by=rng.choice(["uniform", "zipf"]), dtype=rng.choice(["bf16", "bf16", "fp16"]),
                        out=rng.choice(["same", "fp32"]) if direction == "backward_weight" else "same")
        elif op == "router":
            groups = rng.choice([1, 1, 2, 4, 8])
            experts = groups * _log_int(rng, max(2, 8 // groups), 512 // groups)
            kept = rng.randint(1, groups)
            direction = rng.choice(["forward", "forward", "backward"])
            tokens = _log_int(rng, 1, 32768)
            case = dict(op=op, direction=direction, tokens=tokens, experts=experts,
                        topk=rng.randint(1, min(16, experts // groups * kept)),
                        score=rng.choice(["softmax", "sigmoid"]), dtype=rng.choice(["fp32", "bf16", "fp16"]),
                        bias=rng.random() < 0.5, groups=groups, kept=kept, group_top=rng.choice([1, 2]),
                        renormalize=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]),
                        padded=tokens // 8 if direction == "forward" and rng.random() < 0.5 else 0)
        else:
            rows = _log_int(rng, 1, 8192)
            case = dict(op=op, rows=rows, requests=_log_int(rng, 1, min(rows, 128)), n=8 * _log_int(rng, 8, 1024),
                        k=8 * _log_int(rng, 8, 1024), rank=rng.choice([8, 16, 24, 32, 64, 128]),
                        adapters=_log_int(rng, 1, 32), split=rng.randrange(1 << 30),
                        dtype=rng.choice(["bf16", "fp16"]))
        if work(case)["flops"] <= 1.9e12 and work(case)["bytes"] <= 4.0e9:
            return case


def _bounds(case):
    """First row of every expert (or request), and the row count at the end."""
    rng = np.random.default_rng(case["split"])
    m = case["rows"]
    if case["op"] == "adapter":
        # every request has at least one row; prompts differ in length by a few times
        r = case["requests"]
        share = rng.gamma(1.5, size=r)
        count = 1 + rng.multinomial(m - r, share / share.sum())
    else:
        e = case["experts"]
        if case["rows_by"] == "distinct":
            count = np.zeros(e, dtype=np.int64)
            count[rng.choice(e, m, replace=False)] = 1
        else:
            p = np.ones(e) if case["rows_by"] == "uniform" else (1.0 + rng.permutation(e)) ** -1.2
            if case["rows_by"] == "zipf" and e >= 4:
                p[rng.choice(e, e // 4, replace=False)] = 0.0       # experts that no token chose
            count = rng.multinomial(m, p / p.sum())
    return [0] + [int(v) for v in np.cumsum(count)]


def _request_adapters(case):
    """The adapter of every request; about one request in eight has none (-1) where there are several."""
    rng = random.Random(case["split"] + 1)
    n = case["requests"]
    return [-1 if n >= 8 and rng.random() < 0.125 else rng.randrange(case["adapters"]) for _ in range(n)]


# ------------------------------------------------------------------------------------------- inputs
def _inputs(case, seed):
    gen = torch.Generator(device=_DEV).manual_seed(seed)
    dt = _DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, dtype=None):
        t = torch.randn(*shape, generator=gen, device=_DEV, dtype=dtype or dt)
        return t.mul_(std) if std != 1.0 else t

    s = {}
    if case["op"] == "experts":
        m, n, k, e = case["rows"], case["n"], case["k"], case["experts"]
        if case["direction"] != "backward_rows":
            s["x"] = normal(m, k)
        if case["direction"] != "forward":
            s["dy"] = normal(m, n)
        if case["direction"] != "backward_weight":
            s["w"] = normal(e, n, k, std=0.02)
    elif case["op"] == "router":
        t, e, k = case["tokens"], case["experts"], case["topk"]
        s["logits"] = normal(t, e, std=1.5)
        if case["padded"]:
            s["logits"][t - case["padded"]:] = float("-inf")     # padding tokens: no expert at all
        if case["bias"]:
            s["bias"] = normal(e, std=0.1, dtype=torch.float32)
        if case["direction"] == "backward":
            # distinct experts per token, as a forward pass returned them
            s["idx"] = torch.rand(t, e, generator=gen, device=_DEV).argsort(dim=1)[:, :k].contiguous()
            s["dweights"] = normal(t, k, dtype=torch.float32)
    else:
        m, n, k, r = case["rows"], case["n"], case["k"], case["rank"]
        s["x"] = normal(m, k)
        s["w"] = normal(n, k, std=0.02)
        s["a"] = normal(case["adapters"], r, k, std=0.02)
        s["b"] = normal(case["adapters"], n, r, std=0.02)
        s["scales"] = torch.rand(case["adapters"], generator=gen, device=_DEV) * 2 + 0.25
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] != "router":
        # a user's program knows the row counts on the host and keeps the offsets on the GPU
        s["bounds"] = _bounds(case)
        s["offsets"] = torch.tensor(s["bounds"], dtype=torch.int32, device=_DEV)
    if case["op"] == "adapter":
        s["request_adapters"] = _request_adapters(case)
        s["adapter"] = torch.tensor(s["request_adapters"], dtype=torch.int32, device=_DEV)
    return s


# ------------------------------------------------------------------------------------------- passes
def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    return {"experts": _plain_experts, "router": _plain_router, "adapter": _plain_adapter}[case["op"]](state, case)


def _run_own(s, c):
    import dispatch_fp8_grouped_amd as mm
    if c["op"] == "experts":
        if c["direction"] == "forward":
            return mm.grouped_forward(s["x"], s["w"], s["offsets"])
        if c["direction"] == "backward_rows":
            return mm.grouped_backward_rows(s["dy"], s["w"], s["offsets"])
        return mm.grouped_backward_weight(s["dy"], s["x"], s["offsets"],
                                          dtype=torch.float32 if c["out"] == "fp32" else None)
    if c["op"] == "router":
        if c["direction"] == "backward":
            return mm.router_backward(s["dweights"], s["logits"], s["idx"], score=c["score"],
                                      renormalize=c["renormalize"], scale=c["scale"])
        idx, weights = mm.router_topk(s["logits"], c["topk"], bias=s.get("bias"), score=c["score"],
                                      num_groups=c["groups"], topk_groups=c["kept"], group_top=c["group_top"],
                                      renormalize=c["renormalize"], scale=c["scale"])
        offsets, order, slot = mm.group_by_expert(idx, c["experts"])
        return idx, weights, offsets, order, slot
    return mm.adapter_forward(s["x"], s["w"], s["a"], s["b"], s["scales"], s["offsets"], s["adapter"])


def _plain_experts(s, c):
    bounds = s["bounds"]
    spans = [(e, bounds[e], bounds[e + 1]) for e in range(c["experts"])]
    dt = _DTYPES[c["dtype"]]
    if c["direction"] == "backward_weight":
        dw = torch.empty(c["experts"], c["n"], c["k"], device=_DEV,
                         dtype=torch.float32 if c["out"] == "fp32" else dt)
        for e, lo, hi in spans:
            dw[e] = s["dy"][lo:hi].float().t() @ s["x"][lo:hi].float()
        return dw
    forward = c["direction"] == "forward"
    rows = s["x"] if forward else s["dy"]
    out = torch.empty(c["rows"], c["n"] if forward else c["k"], device=_DEV, dtype=dt)
    for e, lo, hi in spans:
        if hi > lo:
            w = s["w"][e].float()
            out[lo:hi] = rows[lo:hi].float() @ (w.t() if forward else w)
    return out


def _plain_scores(logits, c):
    """Scores in 64 bits; a masked logit (-inf or NaN) scores 0, and +inf counts as the largest fp32."""
    x = logits.double()
    masked = torch.isnan(x) | (x == float("-inf"))
    x = torch.where(masked, torch.full_like(x, -torch.finfo(torch.float32).max), x)
    x = x.clamp(max=torch.finfo(torch.float32).max)
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-x))
    else:
        top = torch.where(masked, torch.full_like(x, float("-inf")), x).max(dim=1, keepdim=True).values
        top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
        ex = torch.where(masked, torch.zeros_like(x), torch.exp(x - top))
        score = ex / ex.sum(dim=1, keepdim=True).clamp_min(1e-300)
    return torch.where(masked, torch.zeros_like(score), score), masked


def _plain_router(s, c):
    e, k = c["experts"], c["topk"]
    score, masked = _plain_scores(s["logits"], c)
    if c["direction"] == "backward":
        idx, g = s["idx"], s["dweights"].double()
        picked = score.gather(1, idx)
        if c["renormalize"]:
            total = picked.sum(dim=1, keepdim=True)
            share = picked / total
            dpicked = c["scale"] / total * (g - (g * share).sum(dim=1, keepdim=True))
        else:
            dpicked = c["scale"] * g
        dscore = torch.zeros_like(score).scatter_add_(1, idx, dpicked)
        if c["score"] == "sigmoid":
            d = dscore * score * (1.0 - score)
        else:
            d = score * (dscore - (dscore * score).sum(dim=1, keepdim=True))
        return d.to(s["logits"].dtype)

    # the order of the scores is the order of the logits, which no rounding ties
    choice = score + s["bias"].double() if c["bias"] else s["logits"].double()
    none = torch.full_like(choice, float("-inf"))
    choice = torch.where(masked, none, choice)
    if c["groups"] > 1:
        value = choice if c["bias"] or c["group_top"] == 1 else torch.where(masked, none, score)
        best = value.view(-1, c["groups"], e // c["groups"]).sort(dim=2, descending=True).values
        best = best[:, :, :c["group_top"]]
        empty = torch.isinf(best[:, :, 0])
        group = torch.where(torch.isinf(best), torch.zeros_like(best), best).sum(dim=2)
        group = torch.where(empty, torch.full_like(group, float("-inf")), group)
        keep = group.sort(dim=1, descending=True, stable=True).indices[:, :c["kept"]]
        kept = torch.zeros_like(group, dtype=torch.bool).scatter_(1, keep, True)
        choice = torch.where(kept.repeat_interleave(e // c["groups"], dim=1), choice, none)
    top = choice.sort(dim=1, descending=True, stable=True)
    idx = top.indices[:, :k]
    gone = torch.isinf(top.values[:, :k])
    picked = torch.where(gone, torch.zeros((), dtype=torch.float64, device=_DEV), score.gather(1, idx))
    if c["renormalize"]:
        picked = picked / picked.sum(dim=1, keepdim=True).clamp_min(1e-300)
    idx = torch.where(gone, torch.full_like(idx, -1), idx)

    flat = idx.reshape(-1)
    key = torch.where(flat < 0, torch.full_like(flat, e), flat)
    order = key.sort(stable=True).indices
    count = torch.zeros(e + 1, dtype=torch.int64, device=_DEV).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(e + 1, dtype=torch.int64, device=_DEV)
    offsets[1:] = count[:e].cumsum(0)
    place = torch.arange(flat.numel(), device=_DEV)
    slot = torch.empty_like(flat).scatter_(0, order, place)
    slot = torch.where(flat < 0, torch.full_like(slot, -1), slot)
    order = torch.where(place < offsets[e], order, torch.full_like(order, -1))
    return (idx, (picked * c["scale"]).float(), offsets.int(), order.int(), slot.int().view(-1, k))


def _plain_adapter(s, c):
    x = s["x"].float()
    y = x @ s["w"].float().t()
    scales = s["scales"]
    for r, ad in enumerate(s["request_adapters"]):
        if ad < 0:
            continue
        lo, hi = s["bounds"][r], s["bounds"][r + 1]
        low = x[lo:hi] @ s["a"][ad].float().t()
        y[lo:hi] += (low * scales[ad]) @ s["b"][ad].float().t()
    return y.to(_DTYPES[c["dtype"]])


# ------------------------------------------------------------------------------------------- definition
def exact(case, seed):
    """The outputs from the operators' definitions in 64 bits."""
    s = _inputs(case, seed)
    if case["op"] == "experts":
        return _exact_experts(s, case, _bounds(case))
    if case["op"] == "adapter":
        return _exact_adapter(s, case, _bounds(case), _request_adapters(case))
    return _exact_router(s, case)


def _exact_experts(s, case, bounds):
    parts = []
    for e in range(case["experts"]):
        span = slice(bounds[e], bounds[e + 1])
        if case["direction"] == "forward":          # y[m, n] = sum_k x[m, k] w[e, n, k]
            parts.append(torch.mm(s["x"][span].double(), s["w"][e].double().t().contiguous()))
        elif case["direction"] == "backward_rows":  # dx[m, k] = sum_n dy[m, n] w[e, n, k]
            parts.append(torch.mm(s["dy"][span].double(), s["w"][e].double()))
        else:                                       # dw[e, n, k] = sum_m dy[m, n] x[m, k]
            parts.append(torch.mm(s["dy"][span].double().t().contiguous(), s["x"][span].double()))
    return torch.stack(parts) if case["direction"] == "backward_weight" else torch.cat(parts)


def _exact_adapter(s, case, bounds, adapters):
    y = torch.mm(s["x"].double(), s["w"].double().t().contiguous())
    for (lo, hi), ad in zip(zip(bounds, bounds[1:]), adapters):
        if ad >= 0:                                 # the adapter's own weight, W + scale * B A
            delta = torch.mm(s["b"][ad].double(), s["a"][ad].double()) * s["scales"][ad].double()
            y[lo:hi] += torch.mm(s["x"][lo:hi].double(), delta.t().contiguous())
    return y


def _exact_router(s, case):
    """Row by row with numpy on the host, in 64 bits."""
    x = s["logits"].double().cpu().numpy()
    t, e, k = case["tokens"], case["experts"], case["topk"]
    live = x > -np.inf
    with np.errstate(all="ignore"):
        if case["score"] == "softmax":
            shifted = np.exp(x - np.where(live.any(1), x.max(1), 0.0)[:, None])
            p = shifted / shifted.sum(1, keepdims=True)
            p[~live.any(1)] = 0.0
        else:
            p = np.where(live, np.exp(-np.logaddexp(0.0, -x)), 0.0)
    if case["direction"] == "backward":
        # differentiate w_i = scale * p_i (/ sum of the chosen p) through p's own Jacobian
        idx = s["idx"].cpu().numpy()
        g = s["dweights"].double().cpu().numpy()
        chosen = np.take_along_axis(p, idx, 1)
        if case["renormalize"]:
            total = chosen.sum(1, keepdims=True)
            g = (g * total - (g * chosen).sum(1, keepdims=True)) / total ** 2
        dp = np.zeros_like(p)
        np.put_along_axis(dp, idx, g * case["scale"], 1)
        d = p * (1 - p) * dp if case["score"] == "sigmoid" else p * dp - p * (p * dp).sum(1, keepdims=True)
        return torch.from_numpy(d)

    rank = p + s["bias"].double().cpu().numpy() if case["bias"] else x
    rank = np.where(live, rank, -np.inf)
    if case["groups"] > 1:
        # a group is worth the sum of its best one or two; the best groups stay
        value = rank if case["bias"] or case["group_top"] == 1 else np.where(live, p, -np.inf)
        value = -np.sort(-value.reshape(t, case["groups"], -1), axis=2)[:, :, :case["group_top"]]
        worth = np.where(value[:, :, 0] > -np.inf, np.where(value > -np.inf, value, 0.0).sum(2), -np.inf)
        place = np.argsort(np.argsort(-worth, axis=1, kind="stable"), axis=1, kind="stable")
        rank = np.where(np.repeat(place < case["kept"], e // case["groups"], axis=1), rank, -np.inf)
    idx = np.argsort(-rank, axis=1, kind="stable")[:, :k]
    taken = np.take_along_axis(rank, idx, 1) > -np.inf
    w = np.where(taken, np.take_along_axis(p, idx, 1), 0.0)
    if case["renormalize"]:
        total = w.sum(1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    idx = np.where(taken, idx, -1)

    flat = idx.reshape(-1)
    where = [np.flatnonzero(flat == j) for j in range(e)]
    offsets = np.concatenate([[0], np.cumsum([len(v) for v in where])])
    order = np.full(flat.size, -1)
    order[:offsets[-1]] = np.concatenate(where)
    slot = np.full(flat.size, -1)
    slot[order[:offsets[-1]]] = np.arange(offsets[-1])
    return tuple(torch.from_numpy(np.ascontiguousarray(v)) for v in
                 (idx.astype(np.int64), w * case["scale"], offsets.astype(np.int32), order.astype(np.int32),
                  slot.reshape(t, k).astype(np.int32)))


# ------------------------------------------------------------------------------------------- work
def work(case):
    """Bytes and operations of one pass: every input read once (of the weights those that some row meets),
    every output written once."""
    size = torch.finfo(_DTYPES[case["dtype"]]).bits // 8
    if case["op"] == "experts":
        m, n, k = case["rows"], case["n"], case["k"]
        b = _bounds(case)
        used = sum(hi > lo for lo, hi in zip(b, b[1:]))
        if case["direction"] == "backward_weight":
            out = case["experts"] * n * k * (4 if case["out"] == "fp32" else size)
            moved = m * (n + k) * size + out
        else:
            moved = (m * (n + k) + used * n * k) * size
        return {"bytes": moved + 4 * len(b), "flops": 2 * m * n * k}
    if case["op"] == "router":
        t, e, k = case["tokens"], case["experts"], case["topk"]
        if case["direction"] == "backward":
            return {"bytes": t * (2 * e * size + k * 12), "flops": 12 * t * e}
        # ids and weights out; the ordering reads the ids back and writes order and slot
        return {"bytes": t * (e * size + k * (12 + 8 + 8)) + 4 * (e + 1) + (4 * e if case["bias"] else 0),
                "flops": 12 * t * e}
    m, n, k, r = case["rows"], case["n"], case["k"], case["rank"]
    b, ads = _bounds(case), _request_adapters(case)
    used = len({a for a in ads if a >= 0})
    adapted = sum(hi - lo for lo, hi, a in zip(b, b[1:], ads) if a >= 0)
    return {"bytes": (m * (n + k) + n * k + used * r * (n + k)) * size + 4 * (2 * len(b) + case["adapters"]),
            "flops": 2 * m * n * k + 2 * adapted * r * (n + k)}
