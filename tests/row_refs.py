"""The row operators' definitions in 64 bits, shared by their tests (no code of the package)."""
import torch

U = 2.0 ** -24      # half a step of fp32, relative


def half_step(want, dtype):
    """Largest error of one rounding to dtype: half a step, half a smallest subnormal at least."""
    info = torch.finfo(dtype)
    return info.eps / 2 * want.abs() + info.smallest_normal * info.eps / 2


def close(got, want, before, what=""):
    """got is want up to `before` (an absolute bound) and one rounding to got's type; NaN and infinities where want has them."""
    g, bound = got.double(), before + half_step(want.abs() + before, got.dtype)
    top = torch.finfo(got.dtype).max
    fine = torch.isfinite(want) & (want.abs() + bound < top)        # beyond: may round to infinity
    assert torch.equal(torch.isnan(g), torch.isnan(want)), f"{what}: NaN"
    d = (g - want).abs()[fine]
    excess = d - bound.expand_as(want)[fine]
    assert torch.isfinite(g[fine]).all(), f"{what}: not finite"
    assert (excess <= 0).all(), f"{what}: worst excess {excess.max().item():.3g}, {(excess > 0).sum().item()} values"
    rest = ~fine & ~torch.isnan(want)
    assert ((g[rest].abs() >= top * (1 - 2.0 ** -6)) & (g[rest].sign() == want[rest].sign())).all(), f"{what}: large values"


def decode(codes, scales):
    """e4m3fn: bias 7, 0x7F is NaN, no infinity."""
    c = codes.to(torch.int64) & 0xFF
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2(e.double() - 7))
    v = torch.where((c & 127) == 127, torch.full_like(v, float("nan")), v)
    v = torch.where(c >= 128, -v, v)
    return v * scales.double().repeat_interleave(128, dim=-1)[..., :codes.shape[-1]]


def blocks(v):
    pad = -v.shape[-1] % 128
    return torch.nn.functional.pad(v.double(), (0, pad)).unflatten(-1, (-1, 128))


def scales_of(v):
    """2^ceil(log2(largest / 448)) of every block, 2^-126 at least; 1 where it holds an infinity or a NaN.  By comparison
    with exact powers of two: largest <= 448 * 2^e."""
    top = blocks(v).abs().amax(-1)
    bad = ~torch.isfinite(top)
    _, e = torch.frexp(torch.where(bad, torch.ones_like(top), top) / 448)
    e = e.double()
    for _ in range(2):      # the smallest e that holds
        e = torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e)
    e = torch.where(top == 0, torch.full_like(e, -126), e)
    return torch.where(bad, torch.ones_like(top), torch.exp2(e.clamp_min(-126)))


def quantized(v):
    """What the definition keeps of v in 64 bits."""
    b, s = blocks(v), scales_of(v)
    x = b / s.unsqueeze(-1)
    _, e = torch.frexp(x)
    step = torch.exp2((e.double() - 1).clamp_min(-6) - 3)
    out = torch.round(x / step) * step * s.unsqueeze(-1)
    out = torch.where(out.abs() == 2.0 ** 128, out.sign() * 1.875 * 2.0 ** 127, out)        # fp32 ends below 2^128
    out = torch.where(torch.isfinite(b).all(-1, keepdim=True), out, torch.full_like(out, float("nan")))
    return out.flatten(-2)[..., :v.shape[-1]]


def norm(x, residual, weight, eps):
    """(y, v, r)"""
    v = x.double() if residual is None else x.double() + residual.double()
    r = 1 / torch.sqrt(v.square().mean(-1, keepdim=True) + eps)
    return v * r * weight.double(), v, r


def norm_backward(dy, h, weight, dresidual, eps):
    """(dx, dweight, magnitude of dx's terms, of dweight's)"""
    dy, h = dy.double(), h.double()
    r = 1 / torch.sqrt(h.square().mean(-1, keepdim=True) + eps)
    n, g = h * r, dy * weight.double()
    dx = r * (g - n * (g * n).mean(-1, keepdim=True))
    size = r * (g.abs() + n.abs() * (g * n).abs().mean(-1, keepdim=True))
    if dresidual is not None:
        dx, size = dx + dresidual.double(), size + dresidual.double().abs()
    flat = (dy * n).flatten(0, -2) if dy.dim() > 1 else (dy * n)[None]
    return dx, flat.sum(0), size, flat.abs().sum(0)


def swiglu(gate, up):
    return gate * torch.sigmoid(gate) * up


def swiglu_backward(dact, gate, up):
    s = torch.sigmoid(gate)
    return dact * up * (s + gate * s * torch.sigmoid(-gate)), dact * gate * s
