"""The operators of a conditioned transformer layer as measured cases: what goes
in, their plain form in elementary torch operations, their definition in 64
bits, and the calls a user makes of the engine.

* block    the norm after a block, its gate, dropout and scaled addition to the
           residual stream, and the modulated norm before the next block, in
           one pass; and its gradient
* dropout  residual + dropout(x + bias), the mask formed from a counter-based
           generator and never stored; and its gradient
* axes     rotary positions whose pairs of elements follow several axes (time,
           row, column of an image's or a video's token), with or without the
           norm of each head; and its gradient
"""
import math

import torch

own = False

DTYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}
EPSILON = 1e-6


# ------------------------------------------------------------------ the cases

def _block(name, direction, dtype, stream, groups, tokens, n, post, pre, affine, modulated, p,
           stream_scale, branch_scale):
    return {"op": "block", "name": name, "direction": direction, "dtype": dtype, "stream": stream,
            "groups": groups, "tokens": tokens, "n": n, "post": post, "pre": pre,
            "affine": affine, "modulated": modulated, "p": p, "stream_scale": stream_scale,
            "branch_scale": branch_scale}


def _dropout(name, direction, dtype, rows, n, p, bias, residual):
    return {"op": "dropout", "name": name, "direction": direction, "dtype": dtype, "rows": rows,
            "n": n, "p": p, "bias": bias, "residual": residual}


def _axes(name, direction, dtype, batch, tokens, q_heads, k_heads, head_dim, norm, layout, packed,
          order, sections, length):
    case = {"op": "axes", "name": name, "direction": direction, "dtype": dtype, "batch": batch,
            "tokens": tokens, "q_heads": q_heads, "k_heads": k_heads, "head_dim": head_dim,
            "norm": norm, "layout": layout, "packed": packed, "order": order, "length": length,
            "axes": len(sections)}
    case.update({"section%d" % i: s for i, s in enumerate(sections)})
    return case


def listed():
    return [
        # a decode step: one new token of each of 16 sequences enters the stream and is normed
        _block("block decode", "forward", "bfloat16", "bfloat16", 1, 16, 4096, "none", "rms",
               True, False, 0.0, 1.0, 1.0),
        # prompts of two sequences through a layer with norms on both sides of its blocks
        _block("block prompt", "forward", "bfloat16", "bfloat16", 1, 8192, 4096, "rms", "rms",
               True, False, 0.0, 1.0, 0.5),
        # two videos' tokens: a 32-bit stream, gate, scale and shift of each video's condition
        _block("block modulated", "forward", "bfloat16", "float32", 2, 8190, 1536, "none",
               "layer", False, True, 0.0, 1.0, 1.0),
        # the prompts' sizes in training: dx, dy and the gradients of both norms' weights
        _block("block gradient", "gradient", "bfloat16", "bfloat16", 1, 8192, 4096, "rms", "rms",
               True, False, 0.0, 1.0, 0.5),
        # training of a modulated layer with dropout: odd numbers of tokens in four images
        _block("block modulated gradient", "gradient", "bfloat16", "bfloat16", 4, 4097, 1152,
               "none", "layer", False, True, 0.1, 1.0, 1.0),
        # 32-bit training, rows off every vector, weights and biases on both sides
        _block("block f32 ragged gradient", "gradient", "float32", "float32", 1, 1021, 1543,
               "layer", "layer", True, False, 0.1, 0.9, 1.0),
        # a small fine-tuning step's block output into the stream
        _dropout("dropout small", "forward", "bfloat16", 64, 4096, 0.1, False, True),
        # the largest: a training batch's block output with bias, into the stream
        _dropout("dropout large", "forward", "bfloat16", 16384, 8192, 0.1, True, True),
        # its way back on odd sizes, with the bias's gradient
        _dropout("dropout ragged gradient", "gradient", "float16", 4095, 1543, 0.25, True, False),
        # four images of 16 x 16 patches: rows and columns in a vision encoder
        _axes("axes images", "forward", "float16", 4, 256, 16, 16, 80, False, "half", True,
              "blocks", (20, 20), 16),
        # a video of 21 x 30 x 52 patches: normed heads, adjacent pairs, three axes
        _axes("axes video", "forward", "bfloat16", 1, 32760, 40, 40, 128, True, "interleaved",
              False, "blocks", (22, 21, 21), 64),
        # training on text with images: axes dealt in turn, dq, dk and the norm weights'
        _axes("axes gradient", "gradient", "bfloat16", 2, 4095, 32, 8, 128, True, "half", False,
              "dealt", (24, 20, 20), 4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """Mostly round numbers, as models have them, and some that are not."""
    n = _log(rng, lo, hi)
    return -(-n // 64) * 64 if rng.random() < 0.65 else n


def draw(rng):
    op = rng.choice(["block", "block", "dropout", "axes"])
    direction = rng.choice(["forward", "gradient"])
    dtype = rng.choice(["bfloat16", "bfloat16", "float16", "float32"])
    if op == "block":
        n = _width(rng, 64, 8192)
        rows = _log(rng, 1, min(32768, 8192 * 4096 // n // (2 if dtype == "float32" else 1)))
        groups = min(rows, rng.choice([1, 1, 2, 3, 8]))
        tokens = max(1, rows // groups)
        modulated = groups > 1 or rng.random() < 0.3
        post, pre = rng.choice([("none", "rms"), ("none", "layer"), ("rms", "rms"),
                                ("layer", "layer"), ("rms", "none")])
        stream = "float32" if rng.random() < 0.3 else dtype
        return _block("", direction, dtype, stream, groups, tokens, n, post, pre,
                      rng.random() < 0.6, modulated, rng.choice([0.0, 0.0, 0.1, 0.3]),
                      rng.choice([1.0, 1.0, 0.9]), rng.choice([1.0, 0.5]))
    if op == "dropout":
        n = _width(rng, 64, 8192)
        rows = _log(rng, 1, min(65536, 16384 * 4096 // n))
        return _dropout("", direction, dtype, rows, n, rng.choice([0.0, 0.05, 0.1, 0.25, 0.5]),
                        rng.random() < 0.5, direction == "forward" and rng.random() < 0.7)
    head_dim = rng.choice([32, 64, 72, 80, 96, 112, 128, 160, 256])
    pairs = rng.choice([head_dim // 2, head_dim // 2, head_dim // 4])
    count = rng.randint(2, 4)
    cuts = sorted(rng.randint(1, pairs - 1) for _ in range(count - 1))
    if rng.random() < 0.5:      # sections are often whole quads of pairs
        cuts = [c // 4 * 4 for c in cuts]
    sections = [b - a for a, b in zip([0] + cuts, cuts + [pairs])]
    k_heads = rng.randint(1, 12)
    q_heads = k_heads * rng.randint(1, 4)
    rows = _log(rng, 1, min(32768, 16384 * 40 * 128 // ((q_heads + k_heads) * head_dim)))
    if dtype == "float32":
        rows = max(1, rows // 2)
    batch = min(rows, rng.choice([1, 2, 3, rows]))
    return _axes("", direction, dtype, batch, max(1, rows // batch), q_heads, k_heads, head_dim,
                 rng.random() < 0.5, rng.choice(["half", "interleaved"]), rng.random() < 0.5,
                 rng.choice(["blocks", "dealt"]), sections, _log(rng, 16, 16384))


# ------------------------------------------------------------------ what a program has in hand

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _stream_state(case):
    """Whether a pass has w_post, b_post, w_pre, b_pre."""
    return {"w_post": case["affine"] and case["post"] != "none",
            "b_post": case["affine"] and case["post"] == "layer",
            "w_pre": case["affine"] and case["pre"] != "none",
            "b_pre": case["affine"] and case["pre"] == "layer"}


def _prepare_block(case, seed):
    g = _generator(seed)
    dt, ds = DTYPES[case["dtype"]], DTYPES[case["stream"]]
    G, n = case["groups"], case["n"]
    rows = G * case["tokens"]
    has_z = case["pre"] != "none"

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    # channels of a stream differ in size, and some lie off zero
    size, middle = torch.exp(0.5 * normal(n)), 0.3 * normal(n)
    st = {"case": case, "seed": int(seed) * 7919 + 13, "offset": int(seed) * 31 + 5}
    st["y"] = normal(rows, n).to(dt)
    for name, there in _stream_state(case).items():
        st[name] = None
        if there:
            st[name] = ((name[0] == "w") + 0.2 * normal(n)).to(dt)
    for name, there in (("gate", case["modulated"]), ("scale", case["modulated"] and has_z),
                        ("shift", case["modulated"] and has_z)):
        st[name] = (0.5 * normal(G, n)).to(dt) if there else None
    gradient = case["direction"] == "gradient"
    stream = normal(rows, n) * size + middle
    if gradient:
        st["h"] = stream.to(ds)
        st["dh"] = normal(rows, n).to(ds)
        st["dz"] = normal(rows, n).to(dt) if has_z else None
    else:
        st["x"] = stream.to(ds)
    if own:      # the plan and the buffers that a program keeps
        import broadcast_elementwise_gb300 as eb
        per = case["tokens"] if case["modulated"] else None
        st["plan"] = eb.BlockNormPlan(
            dt, rows, n, stream_dtype=ds, post=case["post"], pre=case["pre"], epsilon=EPSILON,
            dropout=case["p"], stream_scale=case["stream_scale"],
            branch_scale=case["branch_scale"], gate_rows=per, mod_rows=per, gradient=gradient)

        def empty(dtype, *shape):
            return torch.empty(*shape, dtype=dtype, device="cuda")

        if gradient:
            st["dx"], st["dy"] = empty(ds, rows, n), empty(dt, rows, n)
            for name in ("gate", "scale", "shift"):
                st["d" + name] = empty(torch.float32, G, n) if st[name] is not None else None
            for name in ("w_post", "b_post", "w_pre", "b_pre"):
                st["d" + name] = empty(torch.float32, n) if st[name] is not None else None
            st["workspace"] = empty(torch.uint8, st["plan"].workspace_bytes)
        else:
            st["h_out"] = empty(ds, rows, n)
            st["z_out"] = empty(dt, rows, n) if has_z else None
    return st


def _prepare_dropout(case, seed):
    g = _generator(seed)
    dt = DTYPES[case["dtype"]]
    rows, n = case["rows"], case["n"]
    st = {"case": case, "seed": int(seed) * 104729 + 7, "offset": int(seed) * 17 + 3,
          "bias": None, "residual": None}
    st["x"] = torch.randn(rows, n, generator=g, device="cuda").to(dt)    # gradient: dy
    if case["bias"] and case["direction"] == "forward":
        st["bias"] = (0.3 * torch.randn(n, generator=g, device="cuda")).to(dt)
    if case["residual"]:
        st["residual"] = torch.randn(rows, n, generator=g, device="cuda").to(dt)
    if own:
        import broadcast_elementwise_gb300 as eb
        gradient = case["direction"] == "gradient"
        st["plan"] = eb.DropoutPlan(dt, rows, n, case["p"], bias=dt if case["bias"] else None,
                                    residual=case["residual"], gradient=gradient)
        st["y"] = torch.empty(rows, n, dtype=dt, device="cuda")
        if gradient:
            st["dbias"] = torch.empty(n, device="cuda") if case["bias"] else None
            st["workspace"] = torch.empty(st["plan"].workspace_bytes, dtype=torch.uint8,
                                          device="cuda")
    return st


def _sections(case):
    return [case["section%d" % i] for i in range(case["axes"])]


def _axis_of_pair(case):
    """The axis of each pair: blocks of pairs in order, or dealt in turn to the axes with pairs left."""
    sections = _sections(case)
    if case["order"] == "blocks":
        return [a for a, s in enumerate(sections) for _ in range(s)]
    turns = [(i, a) for a, s in enumerate(sections) for i in range(s)]
    return [a for _, a in sorted(turns)]


def _prepare_axes(case, seed):
    g = _generator(seed)
    dt = DTYPES[case["dtype"]]
    B, S, Hq, Hk, D = (case[k] for k in ("batch", "tokens", "q_heads", "k_heads", "head_dim"))
    gradient = case["direction"] == "gradient"

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dt)

    def heads():
        if case["packed"]:
            qkv = normal(B, S, (Hq + 2 * Hk) * D)
            return (qkv[..., :Hq * D].view(B, S, Hq, D),
                    qkv[..., Hq * D:(Hq + Hk) * D].view(B, S, Hk, D))
        return normal(B, S, Hq, D), normal(B, S, Hk, D)

    st = {"case": case}
    st["q"], st["k"] = heads()
    if gradient:
        st["dq"], st["dk"] = normal(B, S, Hq, D), normal(B, S, Hk, D)
    st["wq"] = st["wk"] = None
    if case["norm"]:
        st["wq"], st["wk"] = ((1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt)
                              for _ in range(2))
    pairs = sum(_sections(case))
    angle = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64, device="cuda") / pairs)
    angle = torch.arange(case["length"], dtype=torch.float64, device="cuda")[:, None] * angle
    st["cos"], st["sin"] = angle.cos().float(), angle.sin().float()
    st["positions"] = torch.randint(0, case["length"], (case["axes"], B, S), generator=g,
                                    device="cuda", dtype=torch.int32)
    st["axis"] = torch.tensor(_axis_of_pair(case), device="cuda")
    if own:
        import broadcast_elementwise_gb300 as eb
        rotated = gradient and not case["norm"]
        st["plan"] = eb.HeadsPlan(
            dt, (B, S, Hq, D), (B, S, Hk, D), norm="rms" if case["norm"] else "none",
            epsilon=EPSILON, layout=case["layout"], rotary_dim=2 * pairs, gradient=gradient,
            positions=torch.int32, table_positions=case["length"], axes=_sections(case),
            axes_order=case["order"], q_strides=(st["dq"] if rotated else st["q"]).stride(),
            k_strides=(st["dk"] if rotated else st["k"]).stride())
        st["q_out"] = torch.empty(B, S, Hq, D, dtype=dt, device="cuda")
        st["k_out"] = torch.empty(B, S, Hk, D, dtype=dt, device="cuda")
        if case["norm"] and gradient:
            st["dwq"], st["dwk"] = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
            st["workspace"] = torch.empty(st["plan"].workspace_bytes, dtype=torch.uint8,
                                          device="cuda")
    return st


def prepare(case, seed):
    return {"block": _prepare_block, "dropout": _prepare_dropout,
            "axes": _prepare_axes}[case["op"]](case, seed)


# ------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    if own:
        return {"block": _own_block, "dropout": _own_dropout,
                "axes": _own_axes}[case["op"]](state, case)
    return {"block": _plain_block, "dropout": _plain_dropout,
            "axes": _plain_axes}[case["op"]](state, case)


def _block_outputs(case, first, second, dgate, dscale, dshift, dw_post, db_post, dw_pre, db_pre):
    named = {"first": first, "second": second, "dgate": dgate, "dscale": dscale, "dshift": dshift,
             "dw_post": dw_post, "db_post": db_post, "dw_pre": dw_pre, "db_pre": db_pre}
    return {k: v for k, v in named.items() if v is not None}


def _own_block(st, case):
    import broadcast_elementwise_gb300 as eb
    if case["direction"] == "forward":
        eb.execute_block_norm(st["plan"], st["x"], st["y"], st["h_out"], st["z_out"],
                              gate=st["gate"], w_post=st["w_post"], b_post=st["b_post"],
                              w_pre=st["w_pre"], b_pre=st["b_pre"], scale=st["scale"],
                              shift=st["shift"], seed=st["seed"], offset=st["offset"])
        return _block_outputs(case, st["h_out"], st["z_out"], *[None] * 7)
    eb.execute_block_norm_grad(
        st["plan"], st["dz"], st["dh"], st["h"], st["y"], st["dx"], st["dy"], gate=st["gate"],
        w_post=st["w_post"], b_post=st["b_post"], w_pre=st["w_pre"], b_pre=st["b_pre"],
        scale=st["scale"], dgate=st["dgate"], dscale=st["dscale"], dshift=st["dshift"],
        dw_post=st["dw_post"], db_post=st["db_post"], dw_pre=st["dw_pre"], db_pre=st["db_pre"],
        workspace=st["workspace"], seed=st["seed"], offset=st["offset"])
    return _block_outputs(case, st["dx"], st["dy"], st["dgate"], st["dscale"], st["dshift"],
                          st["dw_post"], st["db_post"], st["dw_pre"], st["db_pre"])


def _own_dropout(st, case):
    import broadcast_elementwise_gb300 as eb
    if case["direction"] == "forward":
        eb.execute_dropout(st["plan"], st["x"], st["y"], st["seed"], st["offset"],
                           bias=st["bias"], residual=st["residual"])
        return st["y"]
    eb.execute_dropout_grad(st["plan"], st["x"], st["y"], st["seed"], st["offset"],
                            dbias=st["dbias"], workspace=st["workspace"])
    return [st["y"]] + ([st["dbias"]] if case["bias"] else [])


def _own_axes(st, case):
    import broadcast_elementwise_gb300 as eb
    gradient = case["direction"] == "gradient"
    if not case["norm"] or not gradient:
        q, k = ("dq", "dk") if gradient else ("q", "k")
        eb.execute_heads(st["plan"], st[q], st[k], st["cos"], st["sin"], st["positions"],
                         st["q_out"], st["k_out"], st["wq"], st["wk"])
        return st["q_out"], st["k_out"]
    eb.execute_heads_grad(st["plan"], st["dq"], st["dk"], st["q"], st["k"], st["cos"], st["sin"],
                          st["positions"], st["wq"], st["wk"], st["q_out"], st["k_out"],
                          st["dwq"], st["dwk"], st["workspace"])
    return st["q_out"], st["k_out"], st["dwq"], st["dwk"]


_MASK = 0xFFFFFFFF


def _words(seed, offset, rows, n):
    """Philox4x32-10 (Salmon, Moraes, Dror and Shaw, 2011): word col % 4 of the block with key
    seed and counter (col / 4, row, offset), [rows, n] in int64."""
    quads = -(-n // 4)
    c0 = torch.arange(quads, device="cuda").expand(rows, quads)
    c1 = torch.arange(rows, device="cuda")[:, None].expand(rows, quads)
    c2 = torch.full_like(c0, offset & _MASK)
    c3 = torch.full_like(c0, offset >> 32 & _MASK)
    k0, k1 = seed & _MASK, seed >> 32 & _MASK
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57      # low 64 bits; signed, so shifts are masked
        c0, c1 = (b >> 32 & _MASK) ^ c1 ^ k0, b & _MASK
        c2, c3 = (a >> 32 & _MASK) ^ c3 ^ k1, a & _MASK
        k0, k1 = k0 + 0x9E3779B9 & _MASK, k1 + 0xBB67AE85 & _MASK
    return torch.stack((c0, c1, c2, c3), -1).view(rows, 4 * quads)[:, :n]


def _kept(x, p, seed, offset):
    """x / (1 - p) where it is kept, 0 where it is dropped."""
    least = round(p * 2 ** 32)
    if least == 0:
        return x
    keep = _words(seed, offset, *x.shape) >= least
    return torch.where(keep, x * (1.0 / (1.0 - least / 2 ** 32)), torch.zeros_like(x))


def _plain_dropout(st, case):
    dt = DTYPES[case["dtype"]]
    x = st["x"].float()
    if case["direction"] == "gradient":
        dx = _kept(x, case["p"], st["seed"], st["offset"])
        return [dx.to(dt)] + ([dx.sum(0)] if case["bias"] else [])
    if st["bias"] is not None:
        x = x + st["bias"].float()
    y = _kept(x, case["p"], st["seed"], st["offset"])
    if st["residual"] is not None:
        y = st["residual"].float() + y
    return y.to(dt)


def _normed(x, kind):
    """(x normed, 1 / its deviation)."""
    if kind == "none":
        return x, None
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPSILON)
    return x * r, r


def _norm_back(dy, xhat, r, kind):
    if kind == "none":
        return dy
    d = dy - xhat * (dy * xhat).mean(-1, keepdim=True)
    if kind == "layer":
        d = d - dy.mean(-1, keepdim=True)
    return d * r


def _plain_block(st, case):
    dt, ds = DTYPES[case["dtype"]], DTYPES[case["stream"]]
    G, T, n = case["groups"], case["tokens"], case["n"]
    a, b, p = case["stream_scale"], case["branch_scale"], case["p"]
    full = {k: st[k].float() for k in ("w_post", "b_post", "w_pre", "b_pre") if st[k] is not None}
    rows = {k: st[k].float().repeat_interleave(T, 0) for k in ("gate", "scale", "shift")
            if st[k] is not None}
    yhat, ry = _normed(st["y"].float(), case["post"])
    v = yhat * full.get("w_post", 1.0) + full.get("b_post", 0.0)
    if case["direction"] == "forward":
        h = a * st["x"].float() + b * rows.get("gate", 1.0) * _kept(v, p, st["seed"], st["offset"])
        if case["pre"] == "none":
            return _block_outputs(case, h.to(ds), None, *[None] * 7)
        z = _normed(h, case["pre"])[0] * full.get("w_pre", 1.0) + full.get("b_pre", 0.0)
        z = z * (1 + rows.get("scale", 0.0)) + rows.get("shift", 0.0)
        return _block_outputs(case, h.to(ds), z.to(dt), *[None] * 7)
    got = dict.fromkeys(("dscale", "dshift", "dw_pre", "db_pre", "dgate", "dw_post", "db_post"))
    back = st["dh"].float()
    if case["pre"] != "none":
        dz = st["dz"].float()
        hhat, r = _normed(st["h"].float(), case["pre"])
        if case["modulated"]:
            got["dscale"] = (dz * (hhat * full.get("w_pre", 1.0) + full.get("b_pre", 0.0))
                             ).view(G, T, n).sum(1)
            got["dshift"] = dz.view(G, T, n).sum(1)
        dn = dz * (1 + rows.get("scale", 0.0))
        if "w_pre" in full:
            got["dw_pre"] = (dn * hhat).sum(0)
        if "b_pre" in full:
            got["db_pre"] = dn.sum(0)
        back = back + _norm_back(dn * full.get("w_pre", 1.0), hhat, r, case["pre"])
    e = b * _kept(back, p, st["seed"], st["offset"])
    if case["modulated"]:
        got["dgate"] = (e * v).view(G, T, n).sum(1)
    e = e * rows.get("gate", 1.0)
    if "w_post" in full:
        got["dw_post"] = (e * yhat).sum(0)
    if "b_post" in full:
        got["db_post"] = e.sum(0)
    dy = _norm_back(e * full.get("w_post", 1.0), yhat, ry, case["post"])
    return _block_outputs(case, (a * back).to(ds), dy.to(dt), **got)


def _turn(x, cos, sin, case):
    """The pairs of the leading elements of x [B, S, H, D] turned; cos, sin [B, S, 1, pairs]."""
    m = cos.shape[-1]
    if case["layout"] == "half":
        u, v, rest = x[..., :m], x[..., m:2 * m], x[..., 2 * m:]
        return torch.cat((u * cos - v * sin, v * cos + u * sin, rest), -1)
    u, v, rest = x[..., 0:2 * m:2], x[..., 1:2 * m:2], x[..., 2 * m:]
    return torch.cat((torch.stack((u * cos - v * sin, v * cos + u * sin), -1).flatten(-2), rest),
                     -1)


def _plain_axes(st, case):
    dt = DTYPES[case["dtype"]]
    at = st["positions"].long()[st["axis"]]                 # [pairs, B, S]
    column = torch.arange(at.shape[0], device="cuda")[:, None, None]
    cos = st["cos"][at, column].permute(1, 2, 0)[:, :, None]
    sin = st["sin"][at, column].permute(1, 2, 0)[:, :, None]
    gradient = case["direction"] == "gradient"
    if not case["norm"]:
        q, k, s = (st["dq"], st["dk"], -sin) if gradient else (st["q"], st["k"], sin)
        return _turn(q.float(), cos, s, case).to(dt), _turn(k.float(), cos, s, case).to(dt)

    def one(x, w, dy):
        xhat, r = _normed(x.float(), "rms")
        if dy is None:
            return _turn(xhat * w.float(), cos, sin, case).to(dt), None
        g = _turn(dy.float(), cos, -sin, case)
        return _norm_back(g * w.float(), xhat, r, "rms").to(dt), (g * xhat).sum((0, 1, 2))

    q, wq = one(st["q"], st["wq"], st.get("dq"))
    k, wk = one(st["k"], st["wk"], st.get("dk"))
    return (q, k, wq, wk) if gradient else (q, k)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    size = 4 if case["dtype"] == "float32" else 2
    forward = case["direction"] == "forward"
    if case["op"] == "block":
        wide = 4 if case["stream"] == "float32" else 2
        rows, n = case["groups"] * case["tokens"], case["n"]
        has_z = case["pre"] != "none"
        # a gradient reads y where it norms or gates it
        reads_y = forward or case["post"] != "none" or case["modulated"]
        if forward:
            per = 2 * wide + size * (1 + has_z)
        else:
            per = 2 * wide + has_z * (wide + size) + size * (1 + reads_y)
        weights = sum(_stream_state(case).values()) * n
        mods = case["modulated"] * case["groups"] * n * (1 + 2 * has_z)
        small = size * (weights + mods) + (0 if forward else 4 * (weights + mods))
        ops = 15.0 if forward else 40.0
        return {"bytes": float(rows * n * per + small), "flops": ops * rows * n}
    if case["op"] == "dropout":
        rows, n = case["rows"], case["n"]
        small = case["bias"] * n * (size if forward else 4)
        return {"bytes": float(size * rows * n * (2 + case["residual"]) + small),
                "flops": 3.0 * rows * n}
    D, tokens = case["head_dim"], case["batch"] * case["tokens"]
    rows = tokens * (case["q_heads"] + case["k_heads"])
    tensors = 3 if case["norm"] and not forward else 2
    pairs = sum(_sections(case))
    table = min(case["axes"] * tokens, case["length"]) * pairs * 8 + 4 * case["axes"] * tokens
    weights = 2 * D * (size + (0 if forward else 4)) if case["norm"] else 0
    ops = 3.0 if not case["norm"] else 7.0 if forward else 16.0
    return {"bytes": float(size * tensors * rows * D + table + weights), "flops": ops * rows * D}


# ------------------------------------------------------------------ the definition in 64 bits

def _times(m, c):
    """(high, low) 32 bits of the product of two 32-bit numbers, through 16-bit parts."""
    high, low = c * (m >> 16), c * (m & 0xFFFF)
    t = low + ((high & 0xFFFF) << 16)
    return (high >> 16) + (t >> 32), t & _MASK


def _exact_kept(x, p, seed, offset):
    rows, n = x.shape
    least = round(p * 2 ** 32)
    word = torch.zeros(rows, n, dtype=torch.int64, device="cuda")
    first = torch.arange(0, n, 4, device="cuda")
    counter = [(first // 4)[None].repeat(rows, 1),
               torch.arange(rows, device="cuda")[:, None].repeat(1, first.numel()),
               torch.zeros(rows, first.numel(), dtype=torch.int64, device="cuda") + offset % 2 ** 32,
               torch.zeros(rows, first.numel(), dtype=torch.int64, device="cuda")
               + offset // 2 ** 32 % 2 ** 32]
    key = [seed % 2 ** 32, seed // 2 ** 32 % 2 ** 32]
    for r in range(10):
        h0, l0 = _times(0xD2511F53, counter[0])
        h1, l1 = _times(0xCD9E8D57, counter[2])
        ka, kb = (key[0] + r * 0x9E3779B9) % 2 ** 32, (key[1] + r * 0xBB67AE85) % 2 ** 32
        counter = [h1 ^ counter[1] ^ ka, l1, h0 ^ counter[3] ^ kb, l0]
    for i in range(4):
        word[:, i::4] = counter[i][:, :word[:, i::4].shape[1]]
    x = x / (1.0 - least / 2.0 ** 32)
    x[word < least] = 0.0
    return x


def _exact_block(case, st):
    G, T, n, p = case["groups"], case["tokens"], case["n"], case["p"]
    one = torch.ones(1, 1, n, dtype=torch.float64, device="cuda")

    def wide(t, default):
        return one * default if t is None else t.double().reshape(-1, 1, n)

    def center(t, kind):
        """(t less its mean, its deviation)"""
        if kind == "none":
            return t, torch.ones_like(t[..., :1])
        if kind == "layer":
            t = t - t.sum(-1, keepdim=True) / n
        return t, (t.square().sum(-1, keepdim=True) / n + EPSILON).sqrt()

    def kept(t):
        return _exact_kept(t.reshape(G * T, n).clone(), p, st["seed"], st["offset"]).view(G, T, n)

    def norm_gradient(dy, t, dev, kind):
        if kind == "none":
            return dy
        out = dy / dev - t * ((dy * t).sum(-1, keepdim=True) / n / dev ** 3)
        return out - out.sum(-1, keepdim=True) / n if kind == "layer" else out

    gate, w1, b1 = wide(st["gate"], 1.0), wide(st["w_post"], 1.0), wide(st["b_post"], 0.0)
    scale, w2, b2 = wide(st["scale"], 0.0) + 1, wide(st["w_pre"], 1.0), wide(st["b_pre"], 0.0)
    y, dev_y = center(st["y"].double().view(G, T, n), case["post"])
    v = y / dev_y * w1 + b1
    flat = lambda t: t.reshape(G * T, n)  # noqa: E731
    if case["direction"] == "forward":
        h = (case["stream_scale"] * st["x"].double().view(G, T, n)
             + case["branch_scale"] * (gate * kept(v)))
        if case["pre"] == "none":
            return _block_outputs(case, flat(h), None, *[None] * 7)
        c, dev = center(h, case["pre"])
        z = (c / dev * w2 + b2) * scale + wide(st["shift"], 0.0)
        return _block_outputs(case, flat(h), flat(z), *[None] * 7)
    got = dict.fromkeys(("dscale", "dshift", "dw_pre", "db_pre", "dgate", "dw_post", "db_post"))
    total = st["dh"].double().view(G, T, n)
    if case["pre"] != "none":
        dz = st["dz"].double().view(G, T, n)
        c, dev = center(st["h"].double().view(G, T, n), case["pre"])
        if st["scale"] is not None:
            got["dscale"] = torch.einsum("gtn,gtn->gn", dz, c / dev * w2 + b2)
            got["dshift"] = dz.sum(1)
        if st["w_pre"] is not None:
            got["dw_pre"] = torch.einsum("gtn,gtn->n", dz * scale, c / dev)
        if st["b_pre"] is not None:
            got["db_pre"] = (dz * scale).sum((0, 1))
        total = total + norm_gradient(dz * scale * w2, c, dev, case["pre"])
    e = case["branch_scale"] * kept(total)
    if st["gate"] is not None:
        got["dgate"] = torch.einsum("gtn,gtn->gn", e, v)
    e = e * gate
    if st["w_post"] is not None:
        got["dw_post"] = torch.einsum("gtn,gtn->n", e, y / dev_y)
    if st["b_post"] is not None:
        got["db_post"] = e.sum((0, 1))
    return _block_outputs(case, flat(case["stream_scale"] * total),
                          flat(norm_gradient(e * w1, y, dev_y, case["post"])), **got)


def _exact_axes(case, st):
    B, S = case["batch"], case["tokens"]
    m = st["cos"].shape[1]
    turn = torch.empty(B, S, 1, m, dtype=torch.complex128, device="cuda")
    for j, axis in enumerate(_axis_of_pair(case)):
        at = st["positions"][axis].long()
        turn[:, :, 0, j] = torch.complex(st["cos"][:, j].double()[at], st["sin"][:, j].double()[at])
    index = torch.arange(2 * m, device="cuda")
    first, second = ((index[:m], index[m:]) if case["layout"] == "half" else
                     (index[0::2], index[1::2]))

    def turned(x, by):
        x = x.clone()
        pair = torch.complex(x[..., first], x[..., second]) * by
        x[..., first], x[..., second] = pair.real, pair.imag
        return x

    def each(x, w, dy):
        x = x.double()
        if not case["norm"]:
            return turned(x, turn) if dy is None else turned(dy.double(), turn.conj()), None
        dev = (x.square().sum(-1, keepdim=True) / case["head_dim"] + EPSILON).sqrt()
        if dy is None:
            return turned(x / dev * w.double(), turn), None
        g = turned(dy.double(), turn.conj())
        dw = (g * x / dev).flatten(0, 2).sum(0)
        g = g * w.double()
        return g / dev - x * ((g * x).sum(-1, keepdim=True) / case["head_dim"] / dev ** 3), dw

    q, wq = each(st["q"], st["wq"], st.get("dq"))
    k, wk = each(st["k"], st["wk"], st.get("dk"))
    return (q, k) if wq is None else (q, k, wq, wk)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "block":
        return _exact_block(case, st)
    if case["op"] == "axes":
        return _exact_axes(case, st)
    x = st["x"].double()
    if case["direction"] == "gradient":
        dx = _exact_kept(x.clone(), case["p"], st["seed"], st["offset"])
        return [dx] + ([dx.sum(0)] if case["bias"] else [])
    if st["bias"] is not None:
        x = x + st["bias"].double()
    y = _exact_kept(x.clone(), case["p"], st["seed"], st["offset"])
    return y if st["residual"] is None else y + st["residual"].double()
