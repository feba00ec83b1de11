"""The weight gradients of the head norms in 64 bits, and how far a binary32 sum of them may be
off when its additions are counted as they are made.

dw = the sum over N rows of t = g xhat.  With u = 2^-24, s the magnitudes that enter a t, and a
factor 7 for sums of independent terms of either sign (Hoeffding: passed once in 10^10):
  each t is off by at most (D / 8 + 24) u s                      7 (D / 8 + 24) u |s|_2
  a thread adds L rows one after another; its sum stays below
  7 |s|_2 over its rows, and each addition is off by u of it     49 sqrt(L) u |s|_2
  the groups of a CTA (256 at most), the CTAs (1024 at most, 32 side
  by side, then those 32) add up the same way                    49 (16 + 8) u |s|_2
and 8 u |dw| for what a reciprocal root is off by the same way in every row.
"""
import torch

import layer_ref as ref

U = 2.0 ** -24


def chain(rows, share, sms):
    """The most rows that one thread adds: at least one CTA an SM, in proportion to the
    tensor's heads, eight groups each, four rows an item."""
    groups = max(1, min(rows // 4, int(sms * share) * 8))
    return -(-rows // groups) + 4


def terms(dy, x, cos, sin, layout, eps):
    """(t, s) [B, S, H, D]: the terms of dw and the magnitudes that enter them."""
    xhat = x * ref.rstd(x, eps)
    return (ref.rotate(dy, cos, sin, layout, -1.0) * xhat,
            ref.spread(dy, cos, sin, layout) * xhat.abs())


def bound(t, s, share, sms):
    D, rows = t.shape[-1], t[..., 0].numel()
    size = (s * s).sum((0, 1, 2)).sqrt()
    steps = 7 * (D / 8 + 24) + 49 * (chain(rows, share, sms) ** 0.5 + 16 + 8)
    return U * (steps * size + 8 * t.sum((0, 1, 2)).abs())


def outside(got, want, bound):
    """How many of the sums lie outside their bound."""
    return int((~((got.double() - want).abs() <= bound)).sum())
