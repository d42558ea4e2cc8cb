"""Operators around the fused MoE layer (include/mega_moe_ops.h): products grouped by expert and their
gradients, the router with its gradient and the ordering of its pairs, and adapter projections.

The functions with the C names marshal arguments only; the short names below them check shapes, types and
devices, allocate what they return, and call them.  Everything runs in the HIP kernels of libmegamoe.so.

    idx, weights = mm.router_topk(logits, 8, bias=bias, score="sigmoid", num_groups=8, topk_groups=4, group_top=2)
    offsets, order, slot = mm.group_by_expert(idx, num_experts)      # rows sorted by expert
    y = mm.grouped_forward(x_sorted, w, offsets)                     # y[m] = x[m] @ w[e].T
    dx = mm.grouped_backward_rows(dy, w, offsets)
    dw = mm.grouped_backward_weight(dy, x_sorted, offsets)
    y = mm.adapter_forward(x, w, a, b, scales, offsets, adapter)     # one low-rank adapter per request

Tensors must be dense, on one GPU; a slice of tokens that the router or the ordering is given may start anywhere,
and the other tensors start at a multiple of 16 bytes, as slices of their rows do; `out` and `workspace` share no
memory with the other tensors.  Calls run on the current
stream of that GPU, or on `stream` (a torch stream or a stream handle); a tensor that a call returns belongs to the
stream of the call.  The tensors given with `stream` are recorded on it, so that their memory is not handed out
again before the call has read it; that they are ready by then is up to the caller, as for any stream.

The functions compute values and gradients; autograd does not derive the one from the other.  Where it records and
an input requires a gradient, what grouped_forward, router_topk (its weights) and adapter_forward return carries a node
that raises in backward(), so that no parameter goes without its gradient unnoticed; what the gradient calls return,
and what is written into `out`, is recorded nowhere.
"""
from __future__ import annotations

import ctypes
import functools

import dispatch_fp8_grouped_amd as _mm       # the package imports this module last

BF16 = 0
FP16 = 1
FP32 = 2
SCORE_SOFTMAX = 0
SCORE_SIGMOID = 1
_SCORES = {"softmax": SCORE_SOFTMAX, "sigmoid": SCORE_SIGMOID}

# Exported symbols of include/mega_moe_ops.h
OPS_EXPORTS = ("mega_moe_grouped_forward", "mega_moe_grouped_backward_rows", "mega_moe_grouped_backward_weight",
               "mega_moe_grouped_weight_workspace_bytes",
               "mega_moe_router_topk", "mega_moe_router_backward", "mega_moe_group_workspace_bytes",
               "mega_moe_group_by_expert", "mega_moe_adapter_workspace_bytes", "mega_moe_adapter_forward")


__all__ = ["BF16", "FP16", "FP32", "SCORE_SOFTMAX", "SCORE_SIGMOID", "OPS_EXPORTS", *OPS_EXPORTS,
           "grouped_forward", "grouped_backward_rows", "grouped_backward_weight", "mega_moe_router_config",
           "router_topk", "router_backward", "group_by_expert", "adapter_forward"]


class mega_moe_router_config(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("num_experts", ctypes.c_int32), ("topk", ctypes.c_int32),
                ("score", ctypes.c_int32), ("num_groups", ctypes.c_int32), ("topk_groups", ctypes.c_int32),
                ("group_top", ctypes.c_int32), ("renormalize", ctypes.c_int32), ("scale", ctypes.c_float),
                ("dtype", ctypes.c_int32)]


def _bind(L):
    """Argument types of the operators' symbols (called once, by lib())."""
    vp, i32, i64, u64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64
    rows = [vp, vp, vp, vp, i64, i32, i32, i32, i32]
    L.mega_moe_grouped_forward.argtypes = rows + [vp, vp]
    L.mega_moe_grouped_backward_rows.argtypes = rows + [vp, vp]
    L.mega_moe_grouped_backward_weight.argtypes = rows + [i32, i32, vp, u64, vp, vp]
    L.mega_moe_grouped_weight_workspace_bytes.argtypes = [i64, i32, i32, i32, ctypes.POINTER(u64)]
    cfg = ctypes.POINTER(mega_moe_router_config)
    L.mega_moe_router_topk.argtypes = [cfg, vp, vp, vp, vp, vp]
    L.mega_moe_router_backward.argtypes = [cfg, vp, vp, vp, vp, vp]
    L.mega_moe_group_workspace_bytes.argtypes = [i64, i32, ctypes.POINTER(u64)]
    L.mega_moe_group_by_expert.argtypes = [vp, i64, i32, i32, vp, vp, vp, vp, u64, vp]
    L.mega_moe_adapter_workspace_bytes.argtypes = [i64, i32, i32, i32, i32, ctypes.POINTER(u64)]
    L.mega_moe_adapter_forward.argtypes = [vp] * 8 + [i64] + [i32] * 6 + [vp, u64, vp, vp]
    for name in OPS_EXPORTS:
        getattr(L, name).restype = i32


# --------------------------------------------------------------- the C entry points, same names
def mega_moe_grouped_forward(x, w, offsets, y, rows, n, k, groups, dtype, device_status=None, stream=None):
    _mm._check(_mm.lib().mega_moe_grouped_forward(_mm._ptr(x), _mm._ptr(w), _mm._ptr(offsets), _mm._ptr(y), rows, n, k, groups,
                                                dtype, _mm._ptr(device_status), _mm._stream(stream)),
              "mega_moe_grouped_forward")


def mega_moe_grouped_backward_rows(dy, w, offsets, dx, rows, n, k, groups, dtype, device_status=None, stream=None):
    _mm._check(_mm.lib().mega_moe_grouped_backward_rows(_mm._ptr(dy), _mm._ptr(w), _mm._ptr(offsets), _mm._ptr(dx), rows, n, k,
                                                      groups, dtype, _mm._ptr(device_status), _mm._stream(stream)),
              "mega_moe_grouped_backward_rows")


def mega_moe_grouped_weight_workspace_bytes(rows: int, n: int, k: int, groups: int) -> int:
    out = ctypes.c_uint64(0)
    _mm._check(_mm.lib().mega_moe_grouped_weight_workspace_bytes(rows, n, k, groups, ctypes.byref(out)),
               "mega_moe_grouped_weight_workspace_bytes")
    return out.value


def mega_moe_grouped_backward_weight(dy, x, offsets, dw, rows, n, k, groups, dtype, out_dtype, accumulate=False,
                                     workspace=None, workspace_bytes=None, device_status=None, stream=None):
    nbytes = workspace_bytes
    if nbytes is None:
        nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _mm._check(_mm.lib().mega_moe_grouped_backward_weight(_mm._ptr(dy), _mm._ptr(x), _mm._ptr(offsets), _mm._ptr(dw), rows, n,
                                                        k, groups, dtype, out_dtype, 1 if accumulate else 0,
                                                        _mm._ptr(workspace), nbytes,
                                                        _mm._ptr(device_status), _mm._stream(stream)),
              "mega_moe_grouped_backward_weight")


def mega_moe_router_topk(cfg: mega_moe_router_config, logits, bias, topk_idx, topk_weights, stream=None):
    _mm._check(_mm.lib().mega_moe_router_topk(ctypes.byref(cfg), _mm._ptr(logits), _mm._ptr(bias), _mm._ptr(topk_idx),
                                            _mm._ptr(topk_weights), _mm._stream(stream)), "mega_moe_router_topk")


def mega_moe_router_backward(cfg: mega_moe_router_config, dweights, logits, topk_idx, dlogits, stream=None):
    _mm._check(_mm.lib().mega_moe_router_backward(ctypes.byref(cfg), _mm._ptr(dweights), _mm._ptr(logits), _mm._ptr(topk_idx),
                                                _mm._ptr(dlogits), _mm._stream(stream)), "mega_moe_router_backward")


def mega_moe_group_workspace_bytes(pairs: int, num_local_experts: int) -> int:
    out = ctypes.c_uint64(0)
    _mm._check(_mm.lib().mega_moe_group_workspace_bytes(pairs, num_local_experts, ctypes.byref(out)),
              "mega_moe_group_workspace_bytes")
    return out.value


def mega_moe_group_by_expert(topk_idx, pairs, first_expert, num_local_experts, offsets, order, slot, workspace,
                             workspace_bytes=None, stream=None):
    nbytes = workspace_bytes if workspace_bytes is not None else workspace.numel() * workspace.element_size()
    _mm._check(_mm.lib().mega_moe_group_by_expert(_mm._ptr(topk_idx), pairs, first_expert, num_local_experts,
                                                _mm._ptr(offsets), _mm._ptr(order), _mm._ptr(slot), _mm._ptr(workspace),
                                                nbytes, _mm._stream(stream)), "mega_moe_group_by_expert")


def mega_moe_adapter_workspace_bytes(rows: int, n: int, k: int, rank: int, requests: int) -> int:
    out = ctypes.c_uint64(0)
    _mm._check(_mm.lib().mega_moe_adapter_workspace_bytes(rows, n, k, rank, requests, ctypes.byref(out)),
               "mega_moe_adapter_workspace_bytes")
    return out.value


def mega_moe_adapter_forward(x, w, a, b, scales, offsets, adapter, y, rows, n, k, rank, requests, adapters, dtype,
                             workspace, workspace_bytes=None, device_status=None, stream=None):
    nbytes = workspace_bytes if workspace_bytes is not None else workspace.numel() * workspace.element_size()
    _mm._check(_mm.lib().mega_moe_adapter_forward(_mm._ptr(x), _mm._ptr(w), _mm._ptr(a), _mm._ptr(b), _mm._ptr(scales),
                                                _mm._ptr(offsets), _mm._ptr(adapter), _mm._ptr(y), rows, n, k, rank,
                                                requests, adapters, dtype, _mm._ptr(workspace), nbytes,
                                                _mm._ptr(device_status), _mm._stream(stream)), "mega_moe_adapter_forward")


# --------------------------------------------------------------- checks
def _int32(**sizes):
    """Each of them fits the library's int32: ctypes would pass its low 32 bits without a word."""
    for name, v in sizes.items():
        if not -1 << 31 <= v < 1 << 31:
            raise ValueError(f"{name}: want a 32-bit integer, got {v}")


# Sizes ask for the same workspace every time; the queries' ctypes calls would be a fifth of a small call's host time.
@functools.lru_cache(1024)
def _weight_bytes(rows, n, k, groups):
    _int32(n=n, k=k, groups=groups)
    return mega_moe_grouped_weight_workspace_bytes(rows, n, k, groups)


@functools.lru_cache(1024)
def _group_bytes(pairs, num_local_experts):
    _int32(num_local_experts=num_local_experts)
    return mega_moe_group_workspace_bytes(pairs, num_local_experts)


@functools.lru_cache(1024)
def _adapter_bytes(rows, n, k, rank, requests, adapters):
    _int32(n=n, k=k, rank=rank, requests=requests, adapters=adapters)
    return mega_moe_adapter_workspace_bytes(rows, n, k, rank, requests)


def _want(name, t, shape, dtypes, device=None):
    """t is a dense GPU tensor of this shape and one of these types (shape None: any)."""
    if (t is not None and t.is_cuda and t.is_contiguous() and t.dtype in dtypes
            and (shape is None or t.shape == shape) and (device is None or t.device == device)):
        return
    got = "None" if t is None else f"{t.dtype} {tuple(t.shape)} on {t.device}" + (
        "" if t.is_contiguous() else ", not contiguous")
    types = " or ".join(str(d) for d in dtypes)
    raise ValueError(f"{name}: want contiguous cuda {types}{'' if shape is None else ' ' + str(tuple(shape))}"
                     f"{'' if device is None else ' on ' + str(device)}, got {got}")


@functools.lru_cache(None)
def _current():
    import torch
    return torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


class _Call:
    """Makes `device` and the call's stream current, so that allocations belong to that stream, and records the
    call's tensors on a stream that was given; `raw` is the stream's handle."""

    def __init__(self, device, stream, *tensors):
        self.ctx = None
        if stream is None:
            # the handle of torch.cuda.current_stream(device), without making the object: the host time
            # of a call went from 12.4 to 8.6 us with it, and small calls are bound by that
            current_device, current_stream = _current()
            if current_device() != device.index:
                import torch
                self.ctx = torch.cuda.device(device)
            self.raw = current_stream(device.index)
        else:
            import torch
            if isinstance(stream, int):
                stream = torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)
            if stream.device != device:
                raise ValueError(f"stream of {stream.device} for tensors on {device}")
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
            self.ctx = torch.cuda.stream(stream)
            self.raw = stream.cuda_stream

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
        return self.raw

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


_KINDS = {}


def _halves():
    if not _KINDS:
        import torch
        _KINDS.update({torch.bfloat16: BF16, torch.float16: FP16})
    return _KINDS


@functools.lru_cache(None)
def _logit_kinds():
    import torch
    return {**_halves(), torch.float32: FP32}


def _at(t):
    return None if t is None else t.data_ptr()


def _apart(name, out, *others):
    """`out` shares no memory with the other tensors of the call: work-groups read them until the last one ends."""
    first = out.data_ptr()
    end = first + out.numel() * out.element_size()
    for t in others:
        if t is not None and t.data_ptr() < end and first < t.data_ptr() + t.numel() * t.element_size():
            raise ValueError(f"{name} overlaps another tensor of the call")


@functools.lru_cache(None)
def _stop():
    import torch

    class NoGraph(torch.autograd.Function):
        @staticmethod
        def forward(ctx, what, how, out, *inputs):
            ctx.message = f"{what} records no autograd graph: {how}, or call it under torch.no_grad()"
            return out.detach()

        @staticmethod
        def backward(ctx, *grads):
            raise RuntimeError(ctx.message)
    return NoGraph.apply


def _unrecorded(what, how, out, *inputs):
    """`out`, with a node that raises where autograd would pass through it to inputs that require a gradient."""
    for t in inputs:
        if t.requires_grad:
            import torch
            return _stop()(what, how, out, *inputs) if torch.is_grad_enabled() else out
    return out


def _from16(t):
    """t, or a copy of it where it does not start at a multiple of 16 bytes, which the library asks for: a slice of
    tokens whose rows are no such multiple (bfloat16 logits of 60 experts, ids of an odd topk)."""
    return t if t is None or not t.data_ptr() & 15 else t.clone()


def _grouped(what, rows_in, w, offsets, contract_k, out, status, stream):
    import torch
    kinds = _halves()
    _want("w", w, None, kinds)
    if w.dim() != 3 or rows_in is None or rows_in.dim() != 2:
        raise ValueError(f"{what}: want w [groups, n, k] and rows of two dimensions")
    groups, n, k = w.shape
    if (groups | n | k) >> 31:
        _int32(groups=groups, n=n, k=k)
    inner, outer = (k, n) if contract_k else (n, k)
    rows = rows_in.shape[0]
    _want("x" if contract_k else "dy", rows_in, (rows, inner), (w.dtype,), w.device)
    _want("offsets", offsets, (groups + 1,), (torch.int32,), w.device)
    if status is not None:
        _want("status", status, (1,), (torch.int32,), w.device)
    lib = _mm.lib()
    call = lib.mega_moe_grouped_forward if contract_k else lib.mega_moe_grouped_backward_rows
    with _Call(w.device, stream, rows_in, w, offsets, out, status) as raw:
        if out is None:
            out = torch.empty((rows, outer), dtype=w.dtype, device=w.device)
        else:
            _want("out", out, (rows, outer), (w.dtype,), w.device)
            _apart("out", out, rows_in, w, offsets, status)
        _mm._check(call(rows_in.data_ptr(), w.data_ptr(), offsets.data_ptr(), out.data_ptr(), rows, n, k, groups,
                        kinds[w.dtype], _at(status), raw), what)
    return out


def grouped_forward(x, w, offsets, out=None, status=None, stream=None):
    """y[m] = x[m] @ w[e].T for the rows m of group e, offsets[e] .. offsets[e+1]-1.

    x [rows, k], w [groups, n, k], both bfloat16 or float16; offsets int32 [groups + 1].  Rows that belong
    to no group are not written (in a new `out` they hold what the allocation held).  status: int32 [1], or
    None; see mega_moe_ops.h."""
    y = _grouped("grouped_forward", x, w, offsets, True, out, status, stream)
    return y if out is not None else _unrecorded(
        "grouped_forward", "compute its gradients with grouped_backward_rows and grouped_backward_weight", y, x, w)


def grouped_backward_rows(dy, w, offsets, out=None, status=None, stream=None):
    """dx[m] = dy[m] @ w[e]: the gradient of grouped_forward's rows.  dy [rows, n] -> dx [rows, k]."""
    return _grouped("grouped_backward_rows", dy, w, offsets, False, out, status, stream)


def grouped_backward_weight(dy, x, offsets, dtype=None, out=None, accumulate=False, status=None, stream=None):
    """dw[e] = dy_e.T @ x_e: the gradient of grouped_forward's weights, [groups, n, k] in `dtype` (the
    operands', or float32).  A group without rows gets zeros.  With accumulate, `out` (float32) is added to."""
    import torch
    kinds = _halves()
    _want("x", x, None, kinds)
    if x.dim() != 2 or dy is None or dy.dim() != 2 or offsets is None or offsets.dim() != 1 or offsets.numel() < 2:
        raise ValueError("grouped_backward_weight: want dy [rows, n], x [rows, k] and offsets [groups + 1]")
    rows, k = x.shape
    n, groups = dy.shape[1], offsets.numel() - 1
    _want("dy", dy, (rows, n), (x.dtype,), x.device)
    _want("offsets", offsets, (groups + 1,), (torch.int32,), x.device)
    if dtype is None:
        dtype = out.dtype if out is not None else x.dtype
    if dtype not in (x.dtype, torch.float32):
        raise ValueError(f"dtype: want {x.dtype} or torch.float32, got {dtype}")
    if accumulate and (out is None or dtype != torch.float32):
        raise ValueError("accumulate needs a float32 `out`")
    if status is not None:
        _want("status", status, (1,), (torch.int32,), x.device)
    nbytes = _weight_bytes(rows, n, k, groups)
    with _Call(x.device, stream, dy, x, offsets, out, status) as raw:
        if out is None:
            out = torch.empty((groups, n, k), dtype=dtype, device=x.device)
        else:
            _want("out", out, (groups, n, k), (dtype,), x.device)
            _apart("out", out, dy, x, offsets, status)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=x.device) if nbytes else None
        _mm._check(_mm.lib().mega_moe_grouped_backward_weight(
            dy.data_ptr(), x.data_ptr(), offsets.data_ptr(), out.data_ptr(), rows, n, k, groups, kinds[x.dtype],
            FP32 if dtype == torch.float32 else kinds[dtype], 1 if accumulate else 0, _at(workspace), nbytes, _at(status),
            raw), "grouped_backward_weight")
    return out


@functools.lru_cache(1024)
def _config(tokens, num_experts, topk, score, num_groups, topk_groups, group_top, renormalize, scale, dtype):
    _int32(num_experts=num_experts, topk=topk, num_groups=num_groups, topk_groups=topk_groups, group_top=group_top)
    return mega_moe_router_config(tokens, num_experts, topk, score, num_groups, topk_groups, group_top, renormalize,
                                  scale, dtype)


def _router_config(logits, topk, score, num_groups, topk_groups, group_top, renormalize, scale):
    kinds = _logit_kinds()
    _want("logits", logits, None, kinds)
    if logits.dim() < 2 or logits.shape[-1] < 1:
        raise ValueError(f"logits: want [..., num_experts], got {tuple(logits.shape)}")
    if score not in _SCORES:
        raise ValueError(f"score: want one of {sorted(_SCORES)}, got {score!r}")
    experts = logits.shape[-1]
    return _config(logits.numel() // experts, experts, topk, _SCORES[score], num_groups, topk_groups, group_top,
                   1 if renormalize else 0, scale, kinds[logits.dtype])


def router_topk(logits, topk, bias=None, score="softmax", num_groups=1, topk_groups=1, group_top=1, renormalize=True,
                scale=1.0, stream=None):
    """The `topk` experts of every token and their weights, (topk_idx int64, topk_weights float32) of shape
    [..., topk], as MegaMoE.forward takes them.

    logits [..., num_experts] (float32, bfloat16 or float16); -inf or NaN masks an expert.  bias: float32
    [num_experts], added to the scores for the choice only.  Only experts of the topk_groups best of num_groups
    equal groups are eligible; a group is worth the sum of its group_top (1 or 2) best.  See mega_moe_ops.h."""
    import torch
    given = logits
    cfg = _router_config(logits, topk, score, num_groups, topk_groups, group_top, renormalize, scale)
    if bias is not None:
        _want("bias", bias, (cfg.num_experts,), (torch.float32,), logits.device)
    shape = (*logits.shape[:-1], max(topk, 0))
    with _Call(logits.device, stream, logits, bias) as raw:
        logits, bias = _from16(logits), _from16(bias)
        idx = torch.empty(shape, dtype=torch.int64, device=logits.device)
        weights = torch.empty(shape, dtype=torch.float32, device=logits.device)
        _mm._check(_mm.lib().mega_moe_router_topk(cfg, logits.data_ptr(), _at(bias), idx.data_ptr(), weights.data_ptr(),
                                                  raw), "router_topk")
    return idx, _unrecorded("router_topk", "compute the gradient of its weights with router_backward", weights, given)


def router_backward(dweights, logits, topk_idx, score="softmax", renormalize=True, scale=1.0, stream=None):
    """dlogits (of the logits' type) from the gradient of router_topk's weights, the choice held fixed."""
    import torch
    if topk_idx is None or topk_idx.dim() < 2:
        raise ValueError("topk_idx: want [..., topk]")
    topk = topk_idx.shape[-1]
    cfg = _router_config(logits, topk, score, 1, 1, 1, renormalize, scale)
    _want("topk_idx", topk_idx, (*logits.shape[:-1], topk), (torch.int64,), logits.device)
    _want("dweights", dweights, (*logits.shape[:-1], topk), (torch.float32,), logits.device)
    with _Call(logits.device, stream, dweights, logits, topk_idx) as raw:
        dweights, logits, topk_idx = _from16(dweights), _from16(logits), _from16(topk_idx)
        dlogits = torch.empty_like(logits)
        _mm._check(_mm.lib().mega_moe_router_backward(cfg, dweights.data_ptr(), logits.data_ptr(), topk_idx.data_ptr(),
                                                      dlogits.data_ptr(), raw), "router_backward")
    return dlogits


def group_by_expert(topk_idx, num_local_experts, first_expert=0, stream=None):
    """Sort the chosen pairs by expert: (offsets int32 [num_local_experts + 1], order int32 [pairs], slot int32 of
    topk_idx's shape).  order[i] is the flat pair t*topk + k at place i (-1 behind the last), slot its inverse
    (-1 for a pair of no local expert).  Row i of the grouped products is then token order[i] // topk."""
    import torch
    _want("topk_idx", topk_idx, None, (torch.int64,))
    pairs, device = topk_idx.numel(), topk_idx.device
    nbytes = _group_bytes(pairs, num_local_experts)
    if first_expert >> 31:
        _int32(first_expert=first_expert)
    with _Call(device, stream, topk_idx) as raw:
        topk_idx = _from16(topk_idx)
        offsets = torch.empty(num_local_experts + 1, dtype=torch.int32, device=device)
        order = torch.empty(pairs, dtype=torch.int32, device=device)
        slot = torch.empty(topk_idx.shape, dtype=torch.int32, device=device)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None
        _mm._check(_mm.lib().mega_moe_group_by_expert(topk_idx.data_ptr(), pairs, first_expert, num_local_experts,
                                                      offsets.data_ptr(), order.data_ptr(), slot.data_ptr(),
                                                      _at(workspace), nbytes, raw), "group_by_expert")
    return offsets, order, slot


def adapter_forward(x, w, a, b, scales, offsets, adapter, out=None, workspace=None, status=None, stream=None):
    """y[m] = x[m] @ w.T + scales[i] * (x[m] @ a[i].T) @ b[i].T with i = adapter[r] of the request r that owns row m.

    x [rows, k], w [n, k], a [adapters, rank, k], b [adapters, n, rank], all bfloat16 or float16; scales float32
    [adapters]; offsets int32 [requests + 1] (request r owns rows offsets[r] .. offsets[r+1]-1), adapter int32
    [requests], -1 for a request without one.  workspace: uint8 of mega_moe_adapter_workspace_bytes(), or None."""
    import torch
    kinds = _halves()
    _want("w", w, None, kinds)
    if w.dim() != 2 or x is None or x.dim() != 2 or a is None or a.dim() != 3 or adapter is None or adapter.dim() != 1:
        raise ValueError("adapter_forward: want x [rows, k], w [n, k], a [adapters, rank, k], adapter [requests]")
    n, k = w.shape
    rows, adapters, rank, requests = x.shape[0], a.shape[0], a.shape[1], adapter.shape[0]
    device, same = w.device, (w.dtype,)
    _want("x", x, (rows, k), same, device)
    _want("a", a, (adapters, rank, k), same, device)
    _want("b", b, (adapters, n, rank), same, device)
    _want("scales", scales, (adapters,), (torch.float32,), device)
    _want("offsets", offsets, (requests + 1,), (torch.int32,), device)
    _want("adapter", adapter, (requests,), (torch.int32,), device)
    if status is not None:
        _want("status", status, (1,), (torch.int32,), w.device)
    nbytes = _adapter_bytes(rows, n, k, rank, requests, adapters)
    fresh = out is None
    with _Call(w.device, stream, x, w, a, b, scales, offsets, adapter, out, workspace, status) as raw:
        if out is None:
            out = torch.empty((rows, n), dtype=w.dtype, device=w.device)
        else:
            _want("out", out, (rows, n), (w.dtype,), w.device)
            _apart("out", out, x, w, a, b, scales, offsets, adapter, workspace, status)
        if workspace is None:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=w.device)
        else:
            _want("workspace", workspace, None, (torch.uint8,), w.device)
            _apart("workspace", workspace, x, w, a, b, scales, offsets, adapter, status)
        _mm._check(_mm.lib().mega_moe_adapter_forward(
            x.data_ptr(), w.data_ptr(), a.data_ptr(), b.data_ptr(), scales.data_ptr(), offsets.data_ptr(), adapter.data_ptr(),
            out.data_ptr(), rows, n, k, rank, requests, adapters, kinds[w.dtype], workspace.data_ptr(), workspace.numel(),
            _at(status), raw), "adapter_forward")
    return _unrecorded("adapter_forward", "it serves adapters and has no gradient", out, x, w, a, b, scales) if fresh else out
