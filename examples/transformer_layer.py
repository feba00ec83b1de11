"""One transformer layer's products, head norms and rotary positions on the engine:
a prompt, then single tokens against a cache, and the gradient of its first product.

    python examples/transformer_layer.py

Attention itself is plain torch here; the engine runs what surrounds it:
  gemm            x Wqkv^T + b; the output product into the residual stream; the
                  feed-forward block's products with GELU and residual
  qk_norm_rotary  the norm of each q and k head and the rotation, in place on the
                  views of the projection's output
  gemm_epilogue_grad, gemm, qk_norm_rotary_grad   the same, backwards
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import broadcast_elementwise_gb300 as eb  # noqa: E402


class Layer:
    def __init__(self, width=1024, q_heads=8, k_heads=2, head_dim=128, hidden=2816,
                 positions=8192, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.q_heads, self.k_heads, self.head_dim = q_heads, k_heads, head_dim
        self.width, self.dtype = width, dtype

        def weight(n, k):
            return (torch.randn(n, k, generator=g, device="cuda") / math.sqrt(k)).to(dtype)

        self.w_qkv = weight((q_heads + 2 * k_heads) * head_dim, width)
        self.b_qkv = (0.1 * torch.randn(self.w_qkv.shape[0], generator=g, device="cuda")).to(dtype)
        self.w_out = weight(width, q_heads * head_dim)
        self.w_up, self.w_down = weight(hidden, width), weight(width, hidden)
        self.b_up = torch.zeros(hidden, device="cuda", dtype=dtype)
        self.q_norm = torch.ones(head_dim, device="cuda", dtype=dtype)
        self.k_norm = torch.ones(head_dim, device="cuda", dtype=dtype)
        self.cos, self.sin = eb.rotary_table(positions, head_dim, base=500000.0,
                                             scaling="by_parts", factor=4.0,
                                             trained_length=positions / 4, fast_turns=4.0)

    def heads(self, qkv, batch, tokens):
        """Views of q, k and v inside the projection's output [batch * tokens, .]."""
        x = qkv.view(batch, tokens, self.q_heads + 2 * self.k_heads, self.head_dim)
        return x.split([self.q_heads, self.k_heads, self.k_heads], dim=2)

    def attention_input(self, x, positions):
        """q, k (normed and rotated, in place) and v of x [batch, tokens, width]."""
        batch, tokens, _ = x.shape
        qkv = eb.gemm(x.reshape(batch * tokens, -1), self.w_qkv, self.b_qkv, trans_b=True)
        q, k, v = self.heads(qkv, batch, tokens)
        eb.qk_norm_rotary(q, k, self.q_norm, self.k_norm, self.cos, self.sin, positions,
                          out=(q, k))
        return q, k, v

    def after_attention(self, x, attended):
        """The output product, and the feed-forward block, each into the residual stream."""
        rows = x.reshape(-1, self.width)
        h = eb.gemm(attended.reshape(rows.shape[0], -1), self.w_out, None, rows, trans_b=True)
        up = eb.gemm(h, self.w_up, self.b_up, trans_b=True, activation="gelu_tanh")
        return eb.gemm(up, self.w_down, None, h, trans_b=True).view(x.shape)

    def attend(self, q, k, v, first):
        """Causal attention in plain torch; q's token t sees keys up to first + t."""
        repeat = self.q_heads // self.k_heads
        k, v = k.repeat_interleave(repeat, 2), v.repeat_interleave(repeat, 2)
        score = torch.einsum("bqhd,bkhd->bhqk", q.float(), k.float()) / math.sqrt(self.head_dim)
        at = torch.arange(q.shape[1], device=q.device)[:, None] + first
        score = score.masked_fill(torch.arange(k.shape[1], device=q.device)[None] > at, -math.inf)
        return torch.einsum("bhqk,bkhd->bqhd", score.softmax(-1), v.float()).to(self.dtype)

    def __call__(self, x, cache=None):
        """(y, cache) for x [batch, tokens, width] that follows the cache's tokens."""
        batch, tokens, _ = x.shape
        first = 0 if cache is None else cache[0].shape[1]
        at = torch.arange(first, first + tokens, device=x.device, dtype=torch.int32)
        q, k, v = self.attention_input(x, at)
        if cache is not None:
            k, v = torch.cat((cache[0], k), 1), torch.cat((cache[1], v), 1)
        return self.after_attention(x, self.attend(q, k, v, first)), (k, v)

    def input_gradient(self, x, dq, dk, dv, positions):
        """Gradients of attention_input for the incoming dq, dk, dv: (dx, dw_qkv, db_qkv,
        dq_norm, dk_norm)."""
        batch, tokens, _ = x.shape
        rows = x.reshape(batch * tokens, -1)
        qkv = eb.gemm(rows, self.w_qkv, self.b_qkv, trans_b=True)
        q, k, _ = self.heads(qkv, batch, tokens)
        dqkv = torch.empty_like(qkv)
        gq, gk, gv = self.heads(dqkv, batch, tokens)
        _, _, dwq, dwk = eb.qk_norm_rotary_grad(dq, dk, q, k, self.q_norm, self.k_norm, self.cos,
                                                self.sin, positions, out=(gq, gk))
        gv.copy_(dv)
        dz, db = eb.gemm_epilogue_grad(dqkv, out=dqkv)
        return (eb.gemm(dz, self.w_qkv).view(x.shape), eb.gemm(dz, rows, trans_a=True), db, dwq,
                dwk)


def main():
    torch.manual_seed(1)
    layer = Layer()
    x = torch.randn(2, 300, layer.width, device="cuda").to(layer.dtype)
    whole, _ = layer(x)
    # the same tokens as a prompt of 296 and four single steps over the cache
    y, cache = layer(x[:, :296])
    parts = [y]
    for t in range(296, 300):
        y, cache = layer(x[:, t:t + 1], cache)
        parts.append(y)
    steps = torch.cat(parts, 1)
    off = (steps.float() - whole.float()).norm() / whole.float().norm()
    print("prompt and single tokens against the whole: relative difference %.2g" % off)
    at = torch.arange(300, device="cuda", dtype=torch.int32)
    dq = torch.randn(2, 300, layer.q_heads, layer.head_dim, device="cuda").to(layer.dtype)
    dk, dv = (torch.randn(2, 300, layer.k_heads, layer.head_dim, device="cuda").to(layer.dtype)
              for _ in range(2))
    grads = layer.input_gradient(x, dq, dk, dv, at)
    print("gradients:", ", ".join(str(tuple(g.shape)) for g in grads))
    if eb.get_device_status() or not off < 0.02:
        raise SystemExit("the layer's parts disagree")
    return float(off)


if __name__ == "__main__":
    main()
