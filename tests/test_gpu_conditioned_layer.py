"""The conditioned layer's example end to end: against a 64-bit form of the whole layer, and
its gradient against 64-bit automatic differentiation of the same formulas."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
import block_ref as ref  # noqa: E402
import broadcast_elementwise_gb300 as eb  # noqa: E402
import conditioned_layer as cl  # noqa: E402
import layer_ref  # noqa: E402

SIZES = [dict(width=256, heads=4, head_dim=128, hidden=320),
         dict(width=203, heads=2, head_dim=128, hidden=264)]


def inputs(layer, batch, tokens):
    g = torch.Generator(device="cuda")
    g.manual_seed(3)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    x = normal(batch, tokens, layer.width)
    condition = (0.5 * normal(batch, 6 * layer.width)).to(layer.dtype)
    positions = torch.randint(0, 64, (3, batch, tokens), generator=g, device="cuda")
    return normal, x, condition, positions


def test_example_runs():
    cl.main()


@pytest.mark.parametrize("kw", SIZES)
def test_layer(kw):
    """What the two blocks add to the stream: behind it lie at most eight roundings to bfloat16
    in a row (z, qkv, the heads, the attention, y, z, the hidden units, y), each below 2^-8 of
    its value; norms, softmax and products may pass a relative error on doubled: 2^-4."""
    layer = cl.Layer(dropout=0.2, **kw)
    B, S = 2, 37
    _, x, condition, positions = inputs(layer, B, S)
    out, _ = layer(x, condition, positions, seed=11, step=4)
    rows, n = B * S, layer.width
    s1, t1, g1, s2, t2, g2 = condition.double().repeat_interleave(S, 0).split(n, dim=1)
    m1, m2 = (ref.mask(0.2, 11, 8 + i, rows, n, "cuda") for i in range(2))

    def norm(t):
        t = t - t.mean(-1, keepdim=True)
        return t / (t.square().mean(-1, keepdim=True) + 1e-6).sqrt()

    w = {k: getattr(layer, k).double() for k in ("w_qkv", "w_out", "w_up", "w_down")}
    h = x.double().view(rows, n)
    z = norm(h) * (1 + s1) + t1
    q, k, v = (z @ w["w_qkv"].t()).view(B, S, -1, layer.head_dim).split(layer.heads, dim=2)
    index = torch.repeat_interleave(torch.arange(3, device="cuda"),
                                    torch.tensor(layer.axes, device="cuda"))
    at = positions[index].permute(1, 2, 0)
    column = torch.arange(len(index), device="cuda")
    c, s = layer.cos.double()[at, column], layer.sin.double()[at, column]
    q, k = (layer_ref.norm_rotate(t, None, c, s, "half", 1e-6) for t in (q, k))
    score = torch.einsum("bqhd,bkhd->bhqk", q, k) / layer.head_dim ** 0.5
    y = torch.einsum("bhqk,bkhd->bqhd", score.softmax(-1), v).reshape(rows, -1) @ w["w_out"].t()
    h = h + g1 * m1 * y
    z = norm(h) * (1 + s2) + t2
    y = layer_ref.act(z @ w["w_up"].t(), "gelu_tanh") @ w["w_down"].t()
    want = h + g2 * m2 * y - x.double().view(rows, n)
    got = (out.double() - x.double()).view(rows, n)
    assert (got - want).norm() < 2.0 ** -4 * want.norm()
    assert eb.get_device_status() == 0


@pytest.mark.parametrize("kw", SIZES)
def test_gradient_between_blocks(kw):
    """At the held h and y: a gradient's one rounding to bfloat16 is below 2^-8 of its values;
    what is float32 is off by far less."""
    layer = cl.Layer(dropout=0.2, **kw)
    B, S, n = 2, 37, layer.width
    normal, x, condition, positions = inputs(layer, B, S)
    _, kept = layer(x, condition, positions, seed=11, step=4)
    dz, dh = normal(B * S, n).to(layer.dtype), normal(B * S, n)
    got = layer.between_gradient(kept, condition, dz, dh, seed=11, step=4)
    h, y, _ = kept
    _, _, g1, s2, t2, _ = (t.double().requires_grad_() for t in condition.split(n, dim=1))
    m = ref.mask(0.2, 11, 8, B * S, n, "cuda")
    y64 = y.double().requires_grad_()
    before = (h.double() - (g1.repeat_interleave(S, 0) * m * y64)).detach().requires_grad_()
    stream = before + g1.repeat_interleave(S, 0) * m * y64
    t = stream - stream.mean(-1, keepdim=True)
    t = t / (t.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    z = t * (1 + s2.repeat_interleave(S, 0)) + t2.repeat_interleave(S, 0)
    want = torch.autograd.grad((z * dz.double()).sum() + (stream * dh.double()).sum(),
                               (before, y64, g1, s2, t2))
    for name, w in zip(("x", "y", "gate", "scale", "shift"), want):
        bound = 2.0 ** -8 if name == "y" else 1e-5
        assert (got[name].double() - w).norm() < bound * w.norm(), name
