"""Plain 64-bit forms of the layer operators (heads, matrix products), on torch
tensors of any device, and the error bounds their kernels are held to."""
import math

import torch

# half an ulp, relative: 2^-p for p significant bits
ROUND = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
# half the least subnormal step
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
F32 = 2.0 ** -24


def rotate(x, cos, sin, layout, sign=1.0):
    """x [B, S, H, D] float64; cos, sin [B, S, r/2]: the first r elements' pairs turned."""
    r = 2 * cos.shape[-1]
    y = x.clone()
    c, s = cos[:, :, None, :], sign * sin[:, :, None, :]
    ia = slice(0, r // 2) if layout == "half" else slice(0, r, 2)
    ib = slice(r // 2, r) if layout == "half" else slice(1, r, 2)
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y


def spread(x, cos, sin, layout):
    """|a cos| + |b sin| (and |b cos| + |a sin|): what a rotation's roundings scale with."""
    r = 2 * cos.shape[-1]
    y = x.abs()
    c, s = cos[:, :, None, :].abs(), sin[:, :, None, :].abs()
    ia = slice(0, r // 2) if layout == "half" else slice(0, r, 2)
    ib = slice(r // 2, r) if layout == "half" else slice(1, r, 2)
    a, b = x[..., ia].abs(), x[..., ib].abs()
    y[..., ia] = a * c + b * s
    y[..., ib] = b * c + a * s
    return y


def rstd(x, eps):
    return 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)


def norm_rotate(x, w, cos, sin, layout, eps):
    y = x * rstd(x, eps)
    return rotate(y if w is None else y * w, cos, sin, layout)


def norm_rotate_grad(dy, x, w, cos, sin, layout, eps):
    """(dx, dw, bound scales of dx and dw): the gradient written out."""
    r = rstd(x, eps)
    xhat = x * r
    g = rotate(dy, cos, sin, layout, -1.0)
    gs = spread(dy, cos, sin, layout)
    w = torch.ones(x.shape[-1], dtype=x.dtype, device=x.device) if w is None else w
    gw = g * w
    dx = r * (gw - xhat * (gw * xhat).mean(-1, keepdim=True))
    scale = r * (gs * w.abs() + xhat.abs() * (gs * w.abs() * xhat.abs()).mean(-1, keepdim=True))
    return dx, (g * xhat).sum((0, 1, 2)), scale, (gs * xhat.abs()).sum((0, 1, 2))


def check(got, want, scale, steps, what):
    """|got - want| within the type's rounding of want plus `steps` binary32
    roundings of the summed magnitudes `scale`."""
    dt = got.dtype
    bound = ROUND[dt] * (1 + steps * F32) * want.abs() + TINY[dt] + 1.1 * steps * F32 * scale
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    if bad.any():
        i = int(bad.flatten().nonzero()[0])
        raise AssertionError("%s: %d of %d values outside their bound; flat %d: got %r want %r "
                             "bound %.3g" % (what, int(bad.sum()), bad.numel(), i,
                                             float(got.flatten()[i]), float(want.flatten()[i]),
                                             float(bound.flatten()[i])))


def frequencies(r, base=10000.0, scaling="none", factor=1.0, trained_length=0.0, slow_turns=1.0,
                fast_turns=32.0):
    if scaling == "base":
        base = base * factor ** (r / (r - 2))
    out = []
    for j in range(r // 2):
        f = base ** (-2.0 * j / r)
        if scaling == "linear":
            f /= factor
        if scaling == "by_parts":
            t = trained_length * f / (2 * math.pi)
            g = min(max((t - slow_turns) / (fast_turns - slow_turns), 0.0), 1.0)
            f *= g + (1 - g) / factor
        out.append(f)
    return out


def table(positions, r, amplitude=1.0, first=0, **kw):
    """(cos, sin) float64 [positions, r/2]."""
    p = torch.arange(first, first + positions, dtype=torch.float64)[:, None]
    a = p * torch.tensor(frequencies(r, **kw), dtype=torch.float64)
    return a.cos() * amplitude, a.sin() * amplitude


def act(z, kind):
    if kind == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if kind == "silu":
        return z * torch.sigmoid(z)
    if kind == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0))
    if kind == "gelu_tanh":
        return z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))
    return z


def act_slope(z, kind):
    if kind == "relu":
        return (z > 0).double()
    if kind == "silu":
        return torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z)
    if kind == "gelu":
        return (0.5 * torch.special.erfc(-z / math.sqrt(2.0))
                + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
    if kind == "gelu_tanh":
        c = math.sqrt(8 / math.pi)
        u = c * (z + 0.044715 * z ** 3)
        return torch.sigmoid(u) + (z * c * (1 + 3 * 0.044715 * z ** 2) * torch.sigmoid(u)
                                   * torch.sigmoid(-u))
    return torch.ones_like(z)
