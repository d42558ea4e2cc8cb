"""What surrounds the experts' products in training and serving, as measured workloads: the root-mean-square norm
with the residual's addition, in 16 bits and in 8 bits with scales, and its gradient; SwiGLU between the two products,
and its gradient; activation checkpoints in 8 bits, stored, restored and multiplied into the gradient of the experts'
weights.

An 8-bit row holds e4m3 codes and one scale per 128 columns, the power of two 2^ceil(log2(largest / 448)); outputs in 8
bits are returned as the values that they stand for.  `run` computes a case with elementary torch operations in 32 bits,
or, with `own` set, through dispatch_fp8_grouped_amd.  `exact` computes the same from the definition in 64 bits.
"""
import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
_DEV = "cuda"
_EPS = 1e-6


# ------------------------------------------------------------------------------------------- cases
def listed():
    def norm(name, direction, rows, hidden, dtype="bf16", stream="same", residual=True, weight="same", out="y",
             checkpoint=False):
        return dict(name=name, op="norm", direction=direction, rows=rows, hidden=hidden, dtype=dtype, stream=stream,
                    residual=residual, weight=weight, out=out, checkpoint=checkpoint)

    def swiglu(name, direction, rows, inter, dtype="bf16", checkpoint=True, recompute=False):
        return dict(name=name, op="swiglu", direction=direction, rows=rows, inter=inter, dtype=dtype,
                    checkpoint=checkpoint, recompute=recompute)

    def weight(name, rows, n, k, experts, split, rows_by="uniform", dtype="bf16", out="same"):
        return dict(name=name, op="checkpoint", direction="weight", rows=rows, n=n, k=k, experts=experts, split=split,
                    rows_by=rows_by, dtype=dtype, out=out)

    return [
        # the norm in front of one decoded token's layer: latency
        norm("norm_token", "forward", 1, 7168),
        # a decode step: 8 shards of 128 tokens, a residual stream in fp32, rows for the layer in 8 bits
        norm("norm_decode", "forward", 1024, 7168, stream="fp32", weight="fp32", out="8bit"),
        # a prefill step: rows for the router in 16 bits and for the layer in 8
        norm("norm_prefill", "forward", 32768, 7168, out="both"),
        # the norm's gradient in training, with the residual's gradient added
        norm("norm_backward_prefill", "backward", 32768, 7168),
        # fp16 rows that fill no tile, the norm's input kept in 8 bits
        norm("norm_backward_odd", "backward", 1999, 1000, dtype="fp16", residual=False, checkpoint=True),
        # between the two products of a decode step
        swiglu("swiglu_decode", "forward", 1024, 2048, checkpoint=False),
        # between the two products in training, its input kept in 8 bits
        swiglu("swiglu_prefill", "forward", 32768, 2048),
        # its gradient from the 8 bits, with the activation again for the down weights' gradient
        swiglu("swiglu_backward_prefill", "backward", 32768, 2048, recompute=True),
        # rows kept in 8 bits and restored
        dict(name="checkpoint_store", op="checkpoint", direction="store", rows=8192, cols=4096, dtype="bf16"),
        # gradient of the gate_up weights from rows kept in 8 bits
        weight("checkpoint_weight_prefill", 32768, 4096, 7168, 32, 21),
        # gradient of the down weights under skewed routing, some experts without a row, fp32 out
        weight("checkpoint_weight_skewed", 16384, 7168, 2048, 32, 22, rows_by="zipf", out="fp32"),
        # fp16, sizes that fill no tile, few experts
        weight("checkpoint_weight_odd", 1999, 1000, 2056, 10, 23, dtype="fp16"),
    ]


def _log_int(rng, lo, hi):
    """An integer spread over the logarithm of lo..hi."""
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    """A case of the listed ranges: 1 to 32768 rows of 16 to 16384 columns for the norm; 1 to 65536 rows of 1 to 8192
    columns for SwiGLU and the stored rows; weights of 8 to 8192 columns in steps of 8 and 1 to 64 experts."""
    while True:
        op = rng.choice(["norm", "norm", "swiglu", "checkpoint"])
        if op == "norm":
            direction = rng.choice(["forward", "backward"])
            dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
            case = dict(op=op, direction=direction, rows=_log_int(rng, 1, 32768), hidden=_log_int(rng, 16, 16384),
                        dtype=dtype, stream=rng.choice(["same", "fp32"]), residual=rng.random() < 0.7,
                        weight=rng.choice(["same", "fp32"]),
                        out=rng.choice(["y", "8bit", "both"]) if direction == "forward" else "y",
                        checkpoint=direction == "backward" and rng.random() < 0.5)
        elif op == "swiglu":
            direction = rng.choice(["forward", "backward"])
            case = dict(op=op, direction=direction, rows=_log_int(rng, 1, 65536), inter=_log_int(rng, 1, 8192),
                        dtype=rng.choice(["bf16", "fp16"]), checkpoint=rng.random() < 0.6,
                        recompute=direction == "backward" and rng.random() < 0.5)
        elif rng.random() < 0.4:
            case = dict(op=op, direction="store", rows=_log_int(rng, 1, 65536), cols=_log_int(rng, 1, 8192),
                        dtype=rng.choice(["bf16", "fp16", "fp32"]))
        else:
            case = dict(op=op, direction="weight", rows=_log_int(rng, 1, 32768), n=8 * _log_int(rng, 1, 1024),
                        k=8 * _log_int(rng, 1, 1024), experts=_log_int(rng, 1, 64), split=rng.randrange(1 << 30),
                        rows_by=rng.choice(["uniform", "zipf"]), dtype=rng.choice(["bf16", "bf16", "fp16"]),
                        out=rng.choice(["same", "fp32"]))
        if work(case)["flops"] <= 1.9e12 and work(case)["bytes"] <= 2.1e9:
            return case


def _bounds(case):
    """First row of every expert, and the row count at the end."""
    rng = np.random.default_rng(case["split"])
    e = case["experts"]
    p = np.ones(e) if case["rows_by"] == "uniform" else (1.0 + rng.permutation(e)) ** -1.2
    if case["rows_by"] == "zipf" and e >= 4:
        p[rng.choice(e, e // 4, replace=False)] = 0.0       # experts that no token chose
    return [0] + [int(v) for v in np.cumsum(rng.multinomial(case["rows"], p / p.sum()))]


# ------------------------------------------------------------------------------------------- 8 bits
def _blocks(x):
    """x [..., cols] in 32 bits as [..., blocks, 128], zeros behind the last column."""
    x = x.float()
    return torch.nn.functional.pad(x, (0, -x.shape[-1] % 128)).unflatten(-1, (-1, 128))


def _encode(x):
    """(codes uint8 [..., cols], scales fp32 [..., blocks])"""
    b = _blocks(x)
    m, e = torch.frexp(b.abs().amax(dim=-1))                # largest = m 2^e with m in [1/2, 1), 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9).clamp_min(-126)
    scales = torch.ldexp(torch.ones_like(m), e)
    codes = (b / scales.unsqueeze(-1)).to(torch.float8_e4m3fn).flatten(-2)
    return codes[..., :x.shape[-1]].contiguous().view(torch.uint8), scales


def _decode(codes, scales):
    """The values in 32 bits."""
    v = codes.view(torch.float8_e4m3fn).float()
    return v * scales.repeat_interleave(128, dim=-1)[..., :v.shape[-1]]


# ------------------------------------------------------------------------------------------- inputs
def _inputs(case, seed):
    gen = torch.Generator(device=_DEV).manual_seed(seed)
    dt = _DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, dtype=None):
        t = torch.randn(*shape, generator=gen, device=_DEV, dtype=dtype or dt)
        return t.mul_(std) if std != 1.0 else t

    s = {}
    if case["op"] == "norm":
        r, c = case["rows"], case["hidden"]
        stream = dt if case["stream"] == "same" else torch.float32
        s["weight"] = 1.0 + normal(c, std=0.1, dtype=dt if case["weight"] == "same" else torch.float32)
        if case["direction"] == "forward":
            s["x"] = normal(r, c)
            if case["residual"]:
                s["residual"] = normal(r, c, std=2.0, dtype=stream)
        else:
            s["dy"] = normal(r, c)
            s["h"] = normal(r, c, std=2.0, dtype=stream)
            if case["residual"]:
                s["dresidual"] = normal(r, c, dtype=stream)
            if case["checkpoint"]:
                s["h"] = _encode(s["h"])
    elif case["op"] == "swiglu":
        r, c = case["rows"], case["inter"]
        s["gate_up"] = normal(r, 2 * c, std=1.5)
        if case["direction"] == "backward":
            s["dact"] = normal(r, c)
            if case["checkpoint"]:          # gate and up are rows of their own
                codes, scales = _encode(s["gate_up"].view(r, 2, c))
                s["gate_up"] = codes.view(r, 2 * c), scales.view(r, -1)
    elif case["direction"] == "store":
        s["x"] = normal(case["rows"], case["cols"])
    else:
        s["dy"] = normal(case["rows"], case["n"])
        s["x"] = _encode(normal(case["rows"], case["k"]))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["direction"] == "weight":
        # a user's program knows the row counts on the host and keeps the offsets on the GPU
        s["bounds"] = _bounds(case)
        s["offsets"] = torch.tensor(s["bounds"], dtype=torch.int32, device=_DEV)
    return s


# ------------------------------------------------------------------------------------------- passes
def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    return {"norm": _plain_norm, "swiglu": _plain_swiglu, "checkpoint": _plain_checkpoint}[case["op"]](state, case)


def _run_own(s, c):
    import dispatch_fp8_grouped_amd as mm
    if c["op"] == "norm":
        if c["direction"] == "backward":
            return mm.rms_norm_backward(s["dy"], s["h"], s["weight"], eps=_EPS, dresidual=s.get("dresidual"))
        y, h, kept = mm.rms_norm(s["x"], s["weight"], residual=s.get("residual"), eps=_EPS,
                                 quantize={"y": False, "8bit": True, "both": "both"}[c["out"]])
        return y, h, None if kept is None else mm.dequantize_rows(*kept)
    if c["op"] == "swiglu":
        if c["direction"] == "backward":
            return mm.swiglu_backward(s["dact"], s["gate_up"], recompute=c["recompute"])
        act, kept = mm.swiglu(s["gate_up"], checkpoint=c["checkpoint"])
        if kept is None:
            return act, None
        return act, mm.dequantize_rows(kept[0].view(2 * c["rows"], -1), kept[1].view(2 * c["rows"], -1))
    if c["direction"] == "store":
        return mm.dequantize_rows(*mm.quantize_rows(s["x"]))
    return mm.grouped_backward_weight(s["dy"], s["x"], s["offsets"], dtype=torch.float32 if c["out"] == "fp32" else None)


def _plain_norm(s, c):
    dt, w = _DTYPES[c["dtype"]], s["weight"].float()
    stream = dt if c["stream"] == "same" else torch.float32
    if c["direction"] == "backward":
        kept = c["checkpoint"]
        h = _decode(*s["h"]) if kept else s["h"].float()
        dy = s["dy"].float()
        r = torch.rsqrt((h * h).mean(dim=1, keepdim=True) + _EPS)
        n, g = h * r, dy * w
        dx = r * (g - n * (g * n).mean(dim=1, keepdim=True))
        if c["residual"]:
            dx += s["dresidual"].float()
        # of the residual stream's type; with a kept h and no gradient beside it, of dy's
        return dx.to(stream if c["residual"] or not kept else dt), (dy * n).sum(dim=0)
    v = s["x"].float()
    if c["residual"]:
        v = v + s["residual"].float()
    y = v * torch.rsqrt((v * v).mean(dim=1, keepdim=True) + _EPS) * w
    return (y.to(dt) if c["out"] != "8bit" else None, v.to(stream) if c["residual"] else None,
            _decode(*_encode(y)).to(torch.bfloat16) if c["out"] != "y" else None)


def _plain_swiglu(s, c):
    dt, kept = _DTYPES[c["dtype"]], None
    if c["direction"] == "forward":
        gate, up = s["gate_up"].float().chunk(2, dim=1)
        if c["checkpoint"]:
            kept = _decode(*_encode(s["gate_up"].view(2 * c["rows"], -1))).to(torch.bfloat16)
        return (gate / (1.0 + torch.exp(-gate)) * up).to(dt), kept
    if c["checkpoint"]:
        codes, scales = s["gate_up"]
        gate, up = _decode(codes.view(c["rows"], 2, -1), scales.view(c["rows"], 2, -1)).unbind(1)
    else:
        gate, up = s["gate_up"].float().chunk(2, dim=1)
    dact, sig = s["dact"].float(), 1.0 / (1.0 + torch.exp(-gate))
    dgate = dact * up * sig * (1.0 + gate * (1.0 - sig))
    return (torch.cat([dgate, dact * gate * sig], dim=1).to(dt),
            (gate * sig * up).to(dt) if c["recompute"] else None)


def _plain_checkpoint(s, c):
    if c["direction"] == "store":
        return _decode(*_encode(s["x"])).to(torch.bfloat16)
    x, bounds = _decode(*s["x"]), s["bounds"]
    dw = torch.empty(c["experts"], c["n"], c["k"], device=_DEV,
                     dtype=torch.float32 if c["out"] == "fp32" else _DTYPES[c["dtype"]])
    for e in range(c["experts"]):
        lo, hi = bounds[e], bounds[e + 1]
        dw[e] = s["dy"][lo:hi].float().t() @ x[lo:hi]
    return dw


# ------------------------------------------------------------------------------------------- definition
def exact(case, seed):
    """The outputs from the operators' definitions in 64 bits."""
    s = _inputs(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s, case)
    if case["op"] == "swiglu":
        return _exact_swiglu(s, case)
    if case["direction"] == "store":
        return _rounded(s["x"].double())
    x, parts = _value(*s["x"]), []
    for lo, hi in zip(_bounds(case), _bounds(case)[1:]):    # dw[e, n, k] = sum_m dy[m, n] x[m, k]
        parts.append(torch.mm(s["dy"][lo:hi].double().t().contiguous(), x[lo:hi].contiguous()))
    return torch.stack(parts)


def _value(codes, scales):
    """What the codes stand for: sign, four bits of exponent, three of mantissa, times the scale of their 128."""
    c = codes.to(torch.int64)
    e, m = c >> 3 & 15, (c & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e.double() - 10))
    v = torch.where(c > 127, -v, v)
    col = torch.arange(v.shape[-1], device=v.device) // 128
    return v * scales.double()[..., col]


def _rounded(v):
    """Values of v [rows, cols] in 64 bits on the grid of their block: four significant bits, no finer than 2^-9 scales."""
    out = torch.empty_like(v)
    for at in range(0, v.shape[1], 128):
        b = v[:, at:at + 128]
        scale = torch.exp2(torch.ceil(torch.log2(b.abs().amax(dim=1, keepdim=True) / 448)).clamp_min(-126))
        step = torch.exp2(torch.floor(torch.log2((b / scale).abs())).clamp_min(-6) - 3) * scale
        out[:, at:at + 128] = torch.round(b / step) * step  # to nearest, ties to even
    return out


def _exact_norm(s, case):
    w = s["weight"].double()
    if case["direction"] == "backward":
        h = _value(*s["h"]) if case["checkpoint"] else s["h"].double()
        g = s["dy"].double() * w
        r = (h.square().mean(1, keepdim=True) + _EPS) ** -0.5
        # d(h r)/dh = r (1 - h h^T r^2 / columns)
        dx = r * g - h * r ** 3 * (g * h).mean(1, keepdim=True)
        if case["residual"]:
            dx += s["dresidual"].double()
        return dx, (s["dy"].double() * h * r).sum(0)
    v = s["x"].double()
    if case["residual"]:
        v = v + s["residual"].double()
    y = v / torch.sqrt(v.square().mean(1, keepdim=True) + _EPS) * w
    return (y if case["out"] != "8bit" else None, v if case["residual"] else None,
            _rounded(y) if case["out"] != "y" else None)


def _exact_swiglu(s, case):
    r, c = case["rows"], case["inter"]
    if case["direction"] == "backward" and case["checkpoint"]:
        both = _value(s["gate_up"][0].view(r, 2, c), s["gate_up"][1].view(r, 2, -1))
    else:
        both = s["gate_up"].double().view(r, 2, c)
    gate, up = both[:, 0], both[:, 1]
    sig = torch.sigmoid(gate)
    if case["direction"] == "forward":
        return gate * sig * up, _rounded(both.reshape(2 * r, c)) if case["checkpoint"] else None
    dact = s["dact"].double()
    d = torch.cat([dact * up * (sig + gate * sig * torch.sigmoid(-gate)), dact * gate * sig], dim=1)
    return d, gate * sig * up if case["recompute"] else None


# ------------------------------------------------------------------------------------------- work
def work(case):
    """Bytes and operations of one pass: every input read once, every output written once (8 bits as such, with their
    scales)."""
    t = _BYTES[case["dtype"]]
    if case["op"] == "norm":
        r, c = case["rows"], case["hidden"]
        stream = t if case["stream"] == "same" else 4
        kept = c + 4 * (-(-c // 128))
        w = c * (t if case["weight"] == "same" else 4)
        if case["direction"] == "backward":
            dx = stream if case["residual"] or not case["checkpoint"] else t
            row = c * (t + dx + (stream if case["residual"] else 0)) + (kept if case["checkpoint"] else c * stream)
            return {"bytes": r * row + w + 4 * c, "flops": 10 * r * c}
        row = c * (t + (2 * stream if case["residual"] else 0) + (t if case["out"] != "8bit" else 0))
        return {"bytes": r * (row + (kept if case["out"] != "y" else 0)) + w, "flops": 5 * r * c}
    if case["op"] == "swiglu":
        r, c = case["rows"], case["inter"]
        kept = 2 * (c + 4 * (-(-c // 128)))
        if case["direction"] == "forward":
            return {"bytes": r * (3 * c * t + (kept if case["checkpoint"] else 0)), "flops": 6 * r * c}
        row = 3 * c * t + (kept if case["checkpoint"] else 2 * c * t) + (c * t if case["recompute"] else 0)
        return {"bytes": r * row, "flops": 12 * r * c}
    if case["direction"] == "store":    # stored and restored (in bf16): the 8 bits are written and read
        r, c = case["rows"], case["cols"]
        return {"bytes": r * (c * (t + 2) + 2 * (c + 4 * (-(-c // 128)))), "flops": 3 * r * c}
    m, n, k, e = case["rows"], case["n"], case["k"], case["experts"]
    out = e * n * k * (4 if case["out"] == "fp32" else t)
    return {"bytes": m * (n * t + k + 4 * (-(-k // 128))) + out + 4 * (e + 1), "flops": 2 * m * n * k}
