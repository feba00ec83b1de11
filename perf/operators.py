"""The attention-layer operators of the engine as measured cases: what goes in,
their plain form in elementary torch operations, their definition in 64 bits,
and the calls a user makes of the engine.

Three operators that a transformer layer runs one after another around its
attention:

* rotary    rotary positions of q and k (RotaryEmbedding), and its gradient;
* qk_norm   the RMS norm of each q and k head and the rotation in one pass, and
            its gradient (dq, dk and the norm weights');
* gemm      a matrix product with bias, activation and residual in its
            epilogue, and its gradient (the epilogue's, then the two products).

Tensors of heads are [batch, tokens, heads, head_dim]; where a case says
`packed`, q and k are the views that a projection's [batch, tokens, q + k + v]
output gives.
"""
import math

import torch

own = False

DTYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}


# ------------------------------------------------------------------ the cases

def _heads(op, name, direction, dtype, batch, tokens, q_heads, k_heads, head_dim, rotary_dim,
           layout, packed, scaling, length):
    return {"op": op, "name": name, "direction": direction, "dtype": dtype, "batch": batch,
            "tokens": tokens, "q_heads": q_heads, "k_heads": k_heads, "head_dim": head_dim,
            "rotary_dim": rotary_dim, "layout": layout, "packed": packed, "scaling": scaling,
            "length": length}


def _gemm(name, direction, dtype, m, n, k, trans_b, bias, activation, residual):
    return {"op": "gemm", "name": name, "direction": direction, "dtype": dtype, "m": m, "n": n,
            "k": k, "trans_b": trans_b, "bias": bias, "activation": activation,
            "residual": residual}


def listed():
    return [
        # one new token of each of 16 sequences, each at a position of its own: a decode step
        _heads("rotary", "rotary decode", "forward", "bfloat16", 16, 1, 32, 8, 128, 128, "half",
               False, "none", 32768),
        # a long prompt, q and k as views of the projection's output, frequencies stretched for
        # a context eight times the trained one
        _heads("rotary", "rotary long prompt", "forward", "bfloat16", 1, 16384, 32, 8, 128, 128,
               "half", True, "by_parts", 16384),
        # a training step's gradient: ragged length, 16-bit floats, adjacent pairs, half the head
        _heads("rotary", "rotary gradient ragged", "gradient", "float16", 4, 2047, 16, 16, 64, 32,
               "interleaved", False, "linear", 4096),
        # a decode step of a large batch with normed heads
        _heads("qk_norm", "qk norm decode", "forward", "bfloat16", 64, 1, 32, 8, 128, 128, "half",
               True, "none", 32768),
        # prompts of two sequences
        _heads("qk_norm", "qk norm prompt", "forward", "bfloat16", 2, 4096, 32, 8, 128, 128,
               "half", True, "none", 4096),
        # the same sizes in training: dq, dk and the gradients of both norms' weights
        _heads("qk_norm", "qk norm gradient", "gradient", "bfloat16", 2, 4096, 32, 8, 128, 128,
               "half", False, "none", 4096),
        # 32-bit activations, odd numbers of tokens and heads, part of a head that is no power of two
        _heads("qk_norm", "qk norm f32 ragged", "forward", "float32", 3, 1021, 12, 3, 96, 48,
               "interleaved", False, "none", 4096),
        # four sequences' new tokens through a square projection, added to the residual stream
        _gemm("gemm decode", "forward", "bfloat16", 4, 4096, 4096, True, True, "none", True),
        # odd sizes throughout: rows of A and B off every vector width
        _gemm("gemm ragged", "forward", "float16", 1021, 1543, 2049, True, True, "silu", False),
        # a prompt through the widening product of a feed-forward block
        _gemm("gemm prompt gelu", "forward", "bfloat16", 4096, 8192, 4096, True, True, "gelu",
              False),
        # the gradient of such a product in training: dz and dbias, then dx and dw
        _gemm("gemm gradient", "gradient", "bfloat16", 4096, 4096, 4096, True, True, "silu",
              False),
        # the largest: a training batch's product, the weight stored [K, N], into the residual stream
        _gemm("gemm large", "forward", "bfloat16", 8192, 8192, 8192, False, False, "none", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        case = _drawn(rng)
        widths = [case[k] for k in ("m", "n", "k", "tokens", "length") if k in case]
        if "head_dim" in case:
            widths += [h * case["head_dim"] for h in
                       (case["q_heads"], case["k_heads"], case["q_heads"] + 2 * case["k_heads"])]
        if 3072 not in widths:      # a width that nothing here uses
            return case


def _drawn(rng):
    if rng.random() < 0.6:
        op = rng.choice(["rotary", "qk_norm"])
        head_dim = rng.choice([32, 64, 80, 96, 112, 128, 160, 192, 256])
        rotary_dim = rng.choice([head_dim, head_dim, head_dim // 2, head_dim // 2 - 2])
        k_heads = rng.randint(1, 12)
        q_heads = k_heads * rng.randint(1, 6)
        dtype = rng.choice(["bfloat16", "bfloat16", "float16", "float32"])
        most = 16384 * 40 * 128 // ((q_heads + k_heads) * head_dim)   # the long prompt's elements
        rows = _log(rng, 1, min(most, 16384))
        if op == "qk_norm" or dtype == "float32":
            rows = max(1, rows // 2)
        batch = rng.choice([1, 2, 3, 8, rows])
        batch = min(batch, rows)
        tokens = max(1, rows // batch)
        direction = rng.choice(["forward", "forward", "gradient"])
        return _heads(op, "", direction, dtype, batch, tokens, q_heads, k_heads, head_dim,
                      rotary_dim, rng.choice(["half", "interleaved"]), rng.random() < 0.5,
                      rng.choice(["none", "linear", "by_parts"]),
                      max(tokens, _log(rng, 512, 32768)))
    direction = rng.choice(["forward", "forward", "forward", "gradient"])
    size = lambda lo: _log(rng, lo, 8192)  # noqa: E731
    m = size(1)
    n, k = size(64), size(64)
    if rng.random() < 0.6:      # most widths are round numbers, some are not
        n, k = -(-n // 64) * 64, -(-k // 64) * 64
    while m * n * k * (2 if direction == "gradient" else 1) > 8192 ** 3:
        m = -(-m // 2)
    return _gemm("", direction, rng.choice(["bfloat16", "float16"]), m, n, k,
                 rng.random() < 0.7, rng.random() < 0.6,
                 rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]), rng.random() < 0.4)


# ------------------------------------------------------------------ what a program has in hand

def frequencies(case):
    """Rotation frequencies in 64 bits, radians per position, and the table's amplitude."""
    r = case["rotary_dim"]
    inv = 10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)
    factor = 8.0
    if case["scaling"] == "linear":
        return inv / factor, 1.0
    if case["scaling"] == "by_parts":      # turns within the trained length decide what is stretched
        turns = (case["length"] / factor) * inv / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        return inv * (keep + (1 - keep) / factor), 0.1 * math.log(factor) + 1
    return inv, 1.0


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _prepare_heads(case, seed):
    g = _generator(seed)
    dt = DTYPES[case["dtype"]]
    B, S, Hq, Hk, D = (case[k] for k in ("batch", "tokens", "q_heads", "k_heads", "head_dim"))

    def heads():
        if case["packed"]:
            qkv = torch.randn(B, S, (Hq + 2 * Hk) * D, generator=g, device="cuda").to(dt)
            return (qkv[..., :Hq * D].view(B, S, Hq, D),
                    qkv[..., Hq * D:(Hq + Hk) * D].view(B, S, Hk, D))
        return (torch.randn(B, S, Hq, D, generator=g, device="cuda").to(dt),
                torch.randn(B, S, Hk, D, generator=g, device="cuda").to(dt))

    st = {"case": case}
    st["q"], st["k"] = heads()
    angle, amplitude = frequencies(case)
    angle = torch.arange(case["length"], dtype=torch.float64, device="cuda")[:, None] * angle.cuda()
    st["cos"] = (angle.cos() * amplitude).float()
    st["sin"] = (angle.sin() * amplitude).float()
    first = torch.randint(0, case["length"] - S + 1, (B, 1), generator=g, device="cuda")
    st["positions"] = (first + torch.arange(S, device="cuda")).to(torch.int32).contiguous()
    if case["op"] == "qk_norm":
        st["wq"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt)
        st["wk"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt)
    if case["direction"] == "gradient":
        st["dq"] = torch.randn(B, S, Hq, D, generator=g, device="cuda").to(dt)
        st["dk"] = torch.randn(B, S, Hk, D, generator=g, device="cuda").to(dt)
    if own:      # the plan and the buffers that a program keeps
        import broadcast_elementwise_gb300 as eb
        norm = case["op"] == "qk_norm"
        gradient = case["direction"] == "gradient"
        st["plan"] = eb.HeadsPlan(
            dt, (B, S, Hq, D), (B, S, Hk, D), norm="rms" if norm else "none", epsilon=EPSILON,
            layout=case["layout"], rotary_dim=case["rotary_dim"], gradient=gradient,
            positions=torch.int32, table_positions=case["length"],
            q_strides=(st["dq"] if gradient and not norm else st["q"]).stride(),
            k_strides=(st["dk"] if gradient and not norm else st["k"]).stride())
        st["q_out"] = torch.empty(B, S, Hq, D, dtype=dt, device="cuda")
        st["k_out"] = torch.empty(B, S, Hk, D, dtype=dt, device="cuda")
        if norm and gradient:
            st["dwq"] = torch.empty(D, device="cuda")
            st["dwk"] = torch.empty(D, device="cuda")
            st["workspace"] = torch.empty(st["plan"].workspace_bytes, dtype=torch.uint8,
                                          device="cuda")
    return st


def _prepare_gemm(case, seed):
    g = _generator(seed)
    dt = DTYPES[case["dtype"]]
    m, n, k = case["m"], case["n"], case["k"]
    x = torch.randn(m, k, generator=g, device="cuda").to(dt)
    w = (torch.randn(*((n, k) if case["trans_b"] else (k, n)), generator=g, device="cuda")
         / math.sqrt(k)).to(dt)
    st = {"case": case, "x": x, "w": w, "bias": None, "residual": None}
    if case["bias"]:
        st["bias"] = (0.5 * torch.randn(n, generator=g, device="cuda")).to(dt)
    if case["residual"]:
        st["residual"] = torch.randn(m, n, generator=g, device="cuda").to(dt)
    if case["direction"] == "gradient":
        st["z"] = torch.randn(m, n, generator=g, device="cuda").to(dt)
        st["dy"] = torch.randn(m, n, generator=g, device="cuda").to(dt)
    if own:      # the plans and the buffers that a program keeps
        import broadcast_elementwise_gb300 as eb
        tb = case["trans_b"]

        def scratch(plan):
            return torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")

        if case["direction"] == "forward":
            st["plan"] = eb.GemmPlan(dt, m, n, k, trans_b=tb, bias=dt if case["bias"] else None,
                                     activation=case["activation"], residual=case["residual"])
            st["y"] = torch.empty(m, n, dtype=dt, device="cuda")
            st["workspace"] = scratch(st["plan"])
        else:
            st["plan_z"] = eb.EpilogueGradPlan(dt, m, n, activation=case["activation"],
                                               bias=case["bias"])
            st["plan_x"] = eb.GemmPlan(dt, m, k, n, trans_b=not tb)
            # dW[N, K] = dZ^T X, or dW[K, N] = X^T dZ: as the weight is stored
            st["plan_w"] = (eb.GemmPlan(dt, n, k, m, trans_a=True) if tb else
                            eb.GemmPlan(dt, k, n, m, trans_a=True))
            st["dz"] = torch.empty(m, n, dtype=dt, device="cuda")
            st["dx"] = torch.empty(m, k, dtype=dt, device="cuda")
            st["dw"] = torch.empty_like(w)
            st["dbias"] = torch.empty(n, device="cuda") if case["bias"] else None
            for p in ("z", "x", "w"):
                st["workspace_" + p] = scratch(st["plan_" + p])
    return st


EPSILON = 1e-6


def prepare(case, seed):
    return _prepare_gemm(case, seed) if case["op"] == "gemm" else _prepare_heads(case, seed)


# ------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    if own:
        return _own_gemm(state, case) if case["op"] == "gemm" else _own_heads(state, case)
    return _plain_gemm(state, case) if case["op"] == "gemm" else _plain_heads(state, case)


def _own_heads(st, case):
    import broadcast_elementwise_gb300 as eb
    if case["op"] == "rotary":
        x = ("dq", "dk") if case["direction"] == "gradient" else ("q", "k")
        eb.execute_heads(st["plan"], st[x[0]], st[x[1]], st["cos"], st["sin"], st["positions"],
                         st["q_out"], st["k_out"])
        return st["q_out"], st["k_out"]
    if case["direction"] == "forward":
        eb.execute_heads(st["plan"], st["q"], st["k"], st["cos"], st["sin"], st["positions"],
                         st["q_out"], st["k_out"], st["wq"], st["wk"])
        return st["q_out"], st["k_out"]
    eb.execute_heads_grad(st["plan"], st["dq"], st["dk"], st["q"], st["k"], st["cos"], st["sin"],
                          st["positions"], st["wq"], st["wk"], st["q_out"], st["k_out"],
                          st["dwq"], st["dwk"], st["workspace"])
    return st["q_out"], st["k_out"], st["dwq"], st["dwk"]


def _own_gemm(st, case):
    import broadcast_elementwise_gb300 as eb
    if case["direction"] == "forward":
        eb.execute_gemm(st["plan"], st["x"], st["w"], st["y"], bias=st["bias"],
                        residual=st["residual"], workspace=st["workspace"])
        return st["y"]
    eb.execute_epilogue_grad(st["plan_z"], st["dy"], st["z"], st["dz"], st["dbias"],
                             st["workspace_z"])
    eb.execute_gemm(st["plan_x"], st["dz"], st["w"], st["dx"], workspace=st["workspace_x"])
    a, b = (st["dz"], st["x"]) if case["trans_b"] else (st["x"], st["dz"])
    eb.execute_gemm(st["plan_w"], a, b, st["dw"], workspace=st["workspace_w"])
    return [st["dz"], st["dx"], st["dw"]] + ([st["dbias"]] if case["bias"] else [])


def _rotate(x, cos, sin, case, sign):
    """The pairs of the first rotary_dim elements turned by the position's angles (sign -1: back)."""
    r = case["rotary_dim"]
    sin = sin * sign
    if case["layout"] == "half":
        a, b, rest = x[..., :r // 2], x[..., r // 2:r], x[..., r:]
        return torch.cat((a * cos - b * sin, b * cos + a * sin, rest), dim=-1)
    a, b, rest = x[..., 0:r:2], x[..., 1:r:2], x[..., r:]
    turned = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    return torch.cat((turned, rest), dim=-1)


def _plain_heads(st, case):
    dt = DTYPES[case["dtype"]]
    at = st["positions"].long()
    cos, sin = st["cos"][at][:, :, None, :], st["sin"][at][:, :, None, :]
    if case["op"] == "rotary":
        x, sign = ("dq", "dk"), -1.0
        if case["direction"] == "forward":
            x, sign = ("q", "k"), 1.0
        return (_rotate(st[x[0]].float(), cos, sin, case, sign).to(dt),
                _rotate(st[x[1]].float(), cos, sin, case, sign).to(dt))

    def forward(x, w):
        x = x.float()
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPSILON) * w.float()
        return _rotate(y, cos, sin, case, 1.0).to(dt)

    def gradient(dy, x, w):
        x, w = x.float(), w.float()
        rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPSILON)
        xhat = x * rstd
        g = _rotate(dy.float(), cos, sin, case, -1.0)
        dw = (g * xhat).sum((0, 1, 2))
        g = g * w
        return (rstd * (g - xhat * (g * xhat).mean(-1, keepdim=True))).to(dt), dw

    if case["direction"] == "forward":
        return forward(st["q"], st["wq"]), forward(st["k"], st["wk"])
    dq, dwq = gradient(st["dq"], st["q"], st["wq"])
    dk, dwk = gradient(st["dk"], st["k"], st["wk"])
    return dq, dk, dwq, dwk


def _activate(z, activation):
    if activation == "relu":
        return z.clamp_min(0)
    if activation == "silu":
        return z / (1 + torch.exp(-z))
    if activation == "gelu":
        return z * 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
    if activation == "gelu_tanh":
        return z * 0.5 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _slope(z, activation):
    """The activation's derivative."""
    if activation == "relu":
        return (z > 0).to(z.dtype)
    if activation == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if activation == "gelu":
        return (0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    if activation == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _plain_gemm(st, case):
    dt = DTYPES[case["dtype"]]
    w = st["w"].float()
    if case["direction"] == "forward":
        z = st["x"].float() @ (w.t() if case["trans_b"] else w)
        if case["bias"]:
            z = z + st["bias"].float()
        y = _activate(z, case["activation"])
        if case["residual"]:
            y = y + st["residual"].float()
        return y.to(dt)
    full = st["dy"].float() * _slope(st["z"].float(), case["activation"])
    dz = full.to(dt)      # an output of its own, held in the inputs' type; the products read it
    back = dz.float()
    x = st["x"].float()
    dx = back @ (w if case["trans_b"] else w.t())
    dw = back.t() @ x if case["trans_b"] else x.t() @ back
    return [dz, dx.to(dt), dw.to(dt)] + ([full.sum(0)] if case["bias"] else [])


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    size = 4 if case["dtype"] == "float32" else 2
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        if case["direction"] == "forward":
            flops = 2.0 * m * n * k
            elements = m * k + n * k + m * n * (2 if case["residual"] else 1)
            elements += n if case["bias"] else 0
            return {"bytes": float(size * elements), "flops": flops}
        # dy, z, x, w in; dz, dx, dw (and dbias) out
        return {"bytes": float(size * (3 * m * n + 2 * m * k + 2 * n * k)
                               + (4 * n if case["bias"] else 0)), "flops": 4.0 * m * n * k}
    D = case["head_dim"]
    rows = case["batch"] * case["tokens"] * (case["q_heads"] + case["k_heads"])
    tokens = case["batch"] * case["tokens"]
    tensors = 3 if case["op"] == "qk_norm" and case["direction"] == "gradient" else 2
    used = min(tokens, case["length"])
    table = used * case["rotary_dim"] * 4 + 4 * tokens
    weights = 0
    if case["op"] == "qk_norm":
        weights = 2 * D * size + (2 * D * 4 if case["direction"] == "gradient" else 0)
    per = {"rotary": 3.0, "qk_norm": 7.0 if case["direction"] == "forward" else 16.0}[case["op"]]
    return {"bytes": float(tensors * rows * D * size + table + weights), "flops": per * rows * D}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "gemm":
        return _exact_gemm(case, st)
    # The rotation as complex numbers: the pair (a, b) times cos + i sin, or its conjugate.
    at = st["positions"].reshape(-1).long()
    turn = torch.complex(st["cos"].double()[at], st["sin"].double()[at])
    turn = turn.reshape(case["batch"], case["tokens"], 1, -1)
    half = case["rotary_dim"] // 2
    index = torch.arange(2 * half, device="cuda")
    first = index[:half] if case["layout"] == "half" else index[0::2]
    second = index[half:] if case["layout"] == "half" else index[1::2]

    def turned(x, factor):
        y = x.clone()
        pair = torch.complex(x[..., first], x[..., second]) * factor
        y[..., first], y[..., second] = pair.real, pair.imag
        return y

    def one(x, dy, w):
        x = x.double()
        if case["op"] == "rotary":
            return turned(dy.double(), turn.conj()) if dy is not None else turned(x, turn), None
        norm = (x.square().sum(-1, keepdim=True) / case["head_dim"] + EPSILON).sqrt()
        if dy is None:
            return turned(x / norm * w.double(), turn), None
        g = turned(dy.double(), turn.conj())
        dw = (g * x / norm).flatten(0, 2).sum(0)
        g = g * w.double()
        inner = (g * x).sum(-1, keepdim=True) / case["head_dim"]
        return g / norm - x * inner / norm ** 3, dw

    q, wq = one(st["q"], st.get("dq"), st.get("wq"))
    k, wk = one(st["k"], st.get("dk"), st.get("wk"))
    return (q, k) if wq is None else (q, k, wq, wk)


def _exact_gemm(case, st):
    x, w = st["x"].double(), st["w"].double()
    w = w if case["trans_b"] else w.t()          # [N, K]
    act = case["activation"]
    if case["direction"] == "forward":
        z = torch.einsum("mk,nk->mn", x, w)
        if st["bias"] is not None:
            z += st["bias"].double()
        if act == "relu":
            z = torch.where(z > 0, z, torch.zeros_like(z))
        elif act == "silu":
            z = z * torch.sigmoid(z)
        elif act == "gelu":
            z = 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0))
        elif act == "gelu_tanh":
            z = z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))
        return z if st["residual"] is None else z + st["residual"].double()
    z, dy = st["z"].double(), st["dy"].double()
    if act == "relu":
        full = torch.where(z > 0, dy, torch.zeros_like(dy))
    elif act == "silu":
        s = torch.sigmoid(z)
        full = dy * (s + z * s * torch.sigmoid(-z))
    elif act == "gelu":
        density = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        full = dy * (0.5 * torch.special.erfc(-z / math.sqrt(2.0)) + z * density)
    elif act == "gelu_tanh":
        c = math.sqrt(8 / math.pi)
        s = torch.sigmoid(c * (z + 0.044715 * z ** 3))
        full = dy * (s + z * s * (1 - s) * c * (1 + 3 * 0.044715 * z ** 2))
    else:
        full = dy
    held = full.to(DTYPES[case["dtype"]]).double()   # dz as it is held
    dx = torch.einsum("mn,nk->mk", held, w)
    dw = torch.einsum("mn,mk->nk", held, x)
    dw = dw if case["trans_b"] else dw.t().contiguous()
    return [full, dx, dw] + ([full.sum(0)] if case["bias"] else [])
