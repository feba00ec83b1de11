"""A conditioned transformer layer for images and video on the engine: norms whose scale, shift
and gate come from a condition, rotary positions of several axes, dropout of each block's
output, and the gradient of the way in and out of a block.

    python examples/conditioned_layer.py

Attention itself is plain torch here; the engine runs what surrounds it:
  block_norm        the modulated norm before a block; between two blocks the gate, dropout,
                    scaled addition to the stream and the next block's norm in one pass
  gemm              the blocks' products
  qk_norm_rotary    head norms and rotation by a token's time, row and column
  block_norm_grad, dropout_grad, qk_norm_rotary_grad, gemm   the same, backwards
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import broadcast_elementwise_gb300 as eb  # noqa: E402


class Layer:
    def __init__(self, width=768, heads=6, head_dim=128, hidden=2048, dropout=0.1, seed=0,
                 dtype=torch.bfloat16):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.width, self.heads, self.head_dim, self.p, self.dtype = width, heads, head_dim, dropout, dtype

        def weight(n, k):
            return (torch.randn(n, k, generator=g, device="cuda") / math.sqrt(k)).to(dtype)

        self.w_qkv, self.w_out = weight(3 * heads * head_dim, width), weight(width, heads * head_dim)
        self.w_up, self.w_down = weight(hidden, width), weight(width, hidden)
        self.q_norm = torch.ones(head_dim, device="cuda", dtype=dtype)
        self.k_norm = torch.ones(head_dim, device="cuda", dtype=dtype)
        self.axes = (16, 24, 24)      # pairs of a head for time, row and column
        self.cos, self.sin = eb.rotary_table(64, head_dim, axes=self.axes)

    def attend(self, q, k, v):
        """Full attention in plain torch, [batch, tokens, heads, head_dim]."""
        score = torch.einsum("bqhd,bkhd->bhqk", q.float(), k.float()) / math.sqrt(self.head_dim)
        return torch.einsum("bhqk,bkhd->bqhd", score.softmax(-1), v.float()).to(self.dtype)

    def attention(self, z, batch, positions):
        qkv = eb.gemm(z, self.w_qkv, trans_b=True)
        q, k, v = qkv.view(batch, -1, 3 * self.heads, self.head_dim).split(self.heads, dim=2)
        eb.qk_norm_rotary(q, k, self.q_norm, self.k_norm, self.cos, self.sin, positions,
                          axes=self.axes, out=(q, k))
        return eb.gemm(self.attend(q, k, v).reshape(z.shape[0], -1), self.w_out, trans_b=True)

    def __call__(self, x, condition, positions, seed=0, step=0):
        """x [batch, tokens, width], a float32 stream; condition [batch, 6 width]: scale, shift and
        gate of each block; positions [3, batch, tokens].  The dropout of call ``step``
        draws offsets 2 step and 2 step + 1."""
        batch = x.shape[0]
        rows = x.reshape(-1, self.width)
        s1, t1, g1, s2, t2, g2 = condition.split(self.width, dim=1)
        kw = dict(pre="layer", dropout=self.p, seed=seed)
        _, z = eb.block_norm(rows, scale=s1, shift=t1, pre="layer", dtype=self.dtype)
        y = self.attention(z, batch, positions)
        h, z = eb.block_norm(rows, y, gate=g1, scale=s2, shift=t2, offset=2 * step, **kw)
        up = eb.gemm(z, self.w_up, trans_b=True, activation="gelu_tanh")
        y2 = eb.gemm(up, self.w_down, trans_b=True)
        out, _ = eb.block_norm(h, y2, gate=g2, dropout=self.p, seed=seed, offset=2 * step + 1,
                               pre="none")
        return out.view(x.shape), (h, y, y2)

    def between_gradient(self, kept, condition, dz, dh, seed=0, step=0):
        """The gradient of the way from the attention block into the feed-forward block."""
        h, y, _ = kept
        _, _, g1, s2, t2, _ = condition.split(self.width, dim=1)
        return eb.block_norm_grad(dz, dh, h, y, gate=g1, scale=s2, shift=t2, pre="layer",
                                  dropout=self.p, seed=seed, offset=2 * step)


def main():
    torch.manual_seed(1)
    layer = Layer()
    batch, frames, height, width = 2, 3, 6, 10
    tokens = frames * height * width
    x = torch.randn(batch, tokens, layer.width, device="cuda")
    condition = (0.5 * torch.randn(batch, 6 * layer.width, device="cuda")).to(layer.dtype)
    grid = torch.cartesian_prod(torch.arange(frames), torch.arange(height), torch.arange(width))
    positions = grid.t().contiguous().cuda()          # [3, tokens], shared by the batch
    out, kept = layer(x, condition, positions, seed=5, step=7)
    again, _ = layer(x, condition, positions, seed=5, step=7)
    other, _ = layer(x, condition, positions, seed=5, step=8)
    print("the same step twice: %s; another step: %s"
          % ("equal" if torch.equal(out, again) else "not equal",
             "equal" if torch.equal(out, other) else "not equal"))
    grads = layer.between_gradient(kept, condition, torch.randn_like(kept[1]),
                                   torch.randn_like(kept[0]), seed=5, step=7)
    print("gradients:", ", ".join("%s %s" % (k, tuple(v.shape)) for k, v in grads.items()))
    if eb.get_device_status() or not torch.equal(out, again) or torch.equal(out, other):
        raise SystemExit("the layer's steps disagree")


if __name__ == "__main__":
    main()
