"""Plain 64-bit forms of dropout and of the norms around a block, on torch tensors of any
device, with the magnitudes that their binary32 roundings scale with."""
import numpy as np
import torch

EPS = 2.0 ** -24


# ------------------------------------------------------------------ random words

def philox(counter, key):
    """Philox4x32-10 of uint64 arrays that hold 32-bit words: four counters, two keys."""
    low = np.uint64(0xFFFFFFFF)
    c, k = [np.asarray(v, np.uint64) for v in counter], [np.uint64(v) for v in key]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        shift = np.uint64(32)
        c = [(b >> shift) ^ c[1] ^ k[0], b & low, (a >> shift) ^ c[3] ^ k[1], a & low]
        k = [(k[0] + np.uint64(0x9E3779B9)) & low, (k[1] + np.uint64(0xBB67AE85)) & low]
    return c


def words(seed, offset, rows, n):
    quads = -(-n // 4)
    col, row = np.meshgrid(np.arange(quads, dtype=np.uint64), np.arange(rows, dtype=np.uint64))
    low = 0xFFFFFFFF
    same = np.ones_like(col)
    w = philox([col, row, same * np.uint64(offset & low), same * np.uint64(offset >> 32 & low)],
               [seed & low, seed >> 32 & low])
    return np.stack(w, -1).reshape(rows, 4 * quads)[:, :n]


def bound(p):
    return round(p * 2 ** 32)


def mask(p, seed, offset, rows, n, device="cpu"):
    """1 / (1 - p) where an element is kept, else 0, float64."""
    keep = words(seed, offset, rows, n) >= np.uint64(bound(p))
    m = torch.from_numpy(keep.astype(np.float64) / (1.0 - bound(p) / 2.0 ** 32))
    return m.to(device)


# ------------------------------------------------------------------ a norm, its gradient, and what their roundings scale with

class Norm:
    """t normed over its rows.  `spread`: what t's own error scales with (|t| for an input).
    hat: the normed rows, s_hat: what their error scales with."""

    def __init__(self, t, kind, eps, spread=None):
        spread = t.abs() if spread is None else spread
        self.kind = kind
        if kind == "none":
            self.hat, self.s_hat, self.r, self.k = t, spread, 1.0, 0.0
            return
        mean = lambda v: v.mean(-1, keepdim=True)  # noqa: E731
        mu = mean(t) if kind == "layer" else torch.zeros_like(t[:, :1])
        c = t - mu
        self.r = 1.0 / torch.sqrt(mean(c * c) + eps)
        self.hat = c * self.r
        about = spread + mu.abs() + (mean(spread) if kind == "layer" else 0.0)
        # the deviation's relative error: the squares' own, and those of what is squared
        self.k = 1.0 + self.r * torch.sqrt(mean(about * about))
        self.s_hat = self.r * about + self.hat.abs() * self.k

    def back(self, d, s_d):
        """(gradient of the rows for the gradient d of hat, what its error scales with)."""
        if self.kind == "none":
            return d, s_d
        mean = lambda v: v.mean(-1, keepdim=True)  # noqa: E731
        out = d - self.hat * mean(d * self.hat)
        s = (s_d + self.hat.abs() * mean(s_d * self.hat.abs() + d.abs() * self.s_hat)
             + self.s_hat * mean((d * self.hat).abs()))
        if self.kind == "layer":
            out, s = out - mean(d), s + mean(s_d)
        return self.r * out, self.r * s + (self.r * out).abs() * self.k


def _rows(t, rows, n, default):
    """A parameter [n] or [groups, n] (None: default) for each row, float64."""
    if t is None:
        return default
    t = t.double()
    return t.expand(rows, n) if t.dim() == 1 else t.repeat_interleave(rows // t.shape[0], 0)


def block(x, y, post, pre, eps, eps_post, m, stream_scale, branch_scale, gate=None, w_post=None,
          b_post=None, w_pre=None, b_pre=None, scale=None, shift=None):
    """((h, scale of its error), (z, scale of its error)); m: the mask (1.0: none)."""
    rows, n = x.shape
    f = lambda t, d: _rows(t, rows, n, d)  # noqa: E731
    h = stream_scale * x.double()
    s_h = h.abs()
    if y is not None:
        v = Norm(y.double(), post, eps_post)
        g = branch_scale * f(gate, 1.0) * m
        w, b = f(w_post, 1.0), f(b_post, 0.0)
        h = h + g * (v.hat * w + b)
        s_h = s_h + abs(g) * (v.s_hat * abs(w) + abs(b))
    if pre == "none":
        return (h, s_h), None
    u = Norm(h, pre, eps, s_h)
    k, w, b = 1.0 + f(scale, 0.0), f(w_pre, 1.0), f(b_pre, 0.0)
    t = f(shift, 0.0)
    z = (u.hat * w + b) * k + t
    return (h, s_h), (z, (u.s_hat * abs(w) + abs(b)) * (1.0 + abs(f(scale, 0.0))) + abs(t))


def block_grad(dz, dh, h, y, post, pre, eps, eps_post, m, stream_scale, branch_scale, gate=None,
               w_post=None, b_post=None, w_pre=None, b_pre=None, scale=None, shift=None):
    """{name: (gradient, scale of its error)} of x, y and every parameter that is given."""
    like = dz if dz is not None else dh
    rows, n = like.shape
    f = lambda t, d: _rows(t, rows, n, d)  # noqa: E731
    out = {}

    def put(name, t, v, s):
        """The sum of v over the rows that share a row of the parameter t."""
        if t is None:
            return
        if t.dim() == 1:
            out[name] = v.sum(0), s.sum(0)
        else:
            fold = lambda q: q.reshape(t.shape[0], -1, n).sum(1)  # noqa: E731
            out[name] = fold(v), fold(s)

    d = torch.zeros(rows, n, dtype=torch.float64, device=like.device)
    d = d if dh is None else d + dh.double()
    s_d = d.abs()
    if pre != "none":
        u = Norm(h.double(), pre, eps)
        k, w, b = 1.0 + f(scale, 0.0), f(w_pre, 1.0), f(b_pre, 0.0)
        ak = 1.0 + abs(f(scale, 0.0))
        g = dz.double()
        put("scale", scale, g * (u.hat * w + b), g.abs() * (u.s_hat * abs(w) + abs(b)))
        put("shift", shift, g, g.abs())
        put("w_pre", w_pre, g * k * u.hat, g.abs() * ak * u.s_hat)
        put("b_pre", b_pre, g * k, g.abs() * ak)
        back, s_back = u.back(g * k * w, g.abs() * ak * abs(w))
        d, s_d = d + back, s_d + s_back
    out["x"] = stream_scale * d, abs(stream_scale) * s_d
    if y is None:
        return out
    e, s_e = branch_scale * m * d, abs(branch_scale) * m * s_d
    v = Norm(y.double(), post, eps_post)
    w, b, g = f(w_post, 1.0), f(b_post, 0.0), f(gate, 1.0)
    put("gate", gate, e * (v.hat * w + b),
        s_e * (abs(v.hat * w) + abs(b)) + abs(e) * (v.s_hat * abs(w) + abs(b)))
    put("w_post", w_post, e * g * v.hat, abs(g) * (s_e * abs(v.hat) + abs(e) * v.s_hat))
    put("b_post", b_post, e * g, abs(g) * s_e)
    out["y"] = v.back(e * g * w, s_e * abs(g * w))
    return out
