"""The layer example end to end: prompt against single tokens over a cache, and
its gradients against 64-bit automatic differentiation of the same formulas."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
import broadcast_elementwise_gb300 as eb  # noqa: E402
import layer_ref as ref  # noqa: E402
import transformer_layer as tl  # noqa: E402


def test_example_runs():
    assert tl.main() < 0.02


@pytest.mark.parametrize("kw", [dict(width=256, q_heads=4, k_heads=2, head_dim=64, hidden=320),
                                dict(width=136, q_heads=3, k_heads=1, head_dim=40, hidden=200)])
def test_input_gradient(kw):
    """Relative 2-norm of each gradient's error: the results are rounded to
    bfloat16 (2^-9 each on average), as are qkv, dqkv and dz between the
    steps; four such roundings, each of relative 2-norm below 2^-8 / sqrt(3),
    add up to less than 2^-7."""
    layer = tl.Layer(positions=64, **kw)
    B, S, D = 2, 21, layer.head_dim
    g = torch.Generator(device="cuda")
    g.manual_seed(3)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(layer.dtype)

    x = normal(B, S, layer.width)
    dq, dk, dv = (normal(B, S, h, D) for h in (layer.q_heads, layer.k_heads, layer.k_heads))
    at = torch.arange(S, device="cuda", dtype=torch.int32)
    got = layer.input_gradient(x, dq, dk, dv, at)
    leaves = [t.double().requires_grad_() for t in (x, layer.w_qkv, layer.b_qkv, layer.q_norm,
                                                    layer.k_norm)]
    c, s = (t.double()[at.long()].expand(B, S, -1) for t in (layer.cos, layer.sin))
    qkv = leaves[0] @ leaves[1].t() + leaves[2]
    q, k, v = layer.heads(qkv, B, S)

    def turned(x, w):
        y = x * ref.rstd(x, 1e-6) * w
        a, b = y[..., :D // 2], y[..., D // 2:]
        cc, ss = c[:, :, None], s[:, :, None]
        return torch.cat((a * cc - b * ss, b * cc + a * ss), -1)

    loss = ((turned(q, leaves[3]) * dq.double()).sum() + (turned(k, leaves[4]) * dk.double()).sum()
            + (v * dv.double()).sum())
    for name, a, b in zip(("dx", "dw", "db", "dq_norm", "dk_norm"), got,
                          torch.autograd.grad(loss, leaves)):
        off = float((a.double() - b).norm() / b.norm())
        assert off < 2 ** -7, (name, off)
    assert eb.get_device_status() == 0
