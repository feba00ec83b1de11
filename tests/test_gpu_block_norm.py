"""The norms around a block on the GPU against a plain 64-bit form (block_ref).

Bounds: the output type's rounding of the true value, plus binary32 roundings of the summed
magnitudes that block_ref gives.  A row's sum takes at most n / 32 + 24 additions one after
another (a thread's share of at least 32, then trees) and the products around it stay below 40;
a parameter's gradient adds up to `rows` more."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

import block_ref as ref  # noqa: E402
import broadcast_elementwise_gb300 as eb  # noqa: E402
import layer_ref  # noqa: E402

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
SEED, OFFSET = 0xC0FFEE1234567, 77


def normal(seed, *shape, dtype=F32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def matrix(seed, rows, n, dtype, how="dense", scale=1.0, middle=0.0):
    def make(*shape):
        return (middle + scale * normal(seed, *shape)).to(dtype)

    if how == "strided":
        return make(rows, n + 24)[:, 8:8 + n]
    if how == "odd stride":
        return make(rows, n + 7)[:, :n]
    if how == "off":
        return make(rows * n + 1)[1:].view(rows, n)
    return make(rows, n)


def steps(n):
    return n / 32 + 64


def operands(rows, n, dtype, stream, groups, how="dense", weights=F32, mods=F32, affine=True,
             modulated=True, scale=1.0, middle=0.0):
    t = {"x": matrix(1, rows, n, stream, how, scale, middle),
         "y": matrix(2, rows, n, dtype, how, 0.7 * scale, middle)}
    p = {}
    if affine:
        for i, name in enumerate(("w_post", "b_post", "w_pre", "b_pre")):
            p[name] = ((name[0] == "w") + 0.3 * normal(3 + i, n)).to(weights)
    if modulated:
        for i, name in enumerate(("gate", "scale", "shift")):
            shape = (n,) if groups == 0 else (groups, n)
            p[name] = (0.5 * normal(7 + i, *shape)).to(mods)
    return t, p


def keep_of(p, rows, n):
    return ref.mask(p, SEED, OFFSET, rows, n, "cuda") if p else 1.0


def valid(p, post, pre, branch=True):
    drop = set()
    if post == "none":
        drop |= {"w_post", "b_post"}
    if pre == "none":
        drop |= {"w_pre", "b_pre", "scale", "shift"}
    if not branch:
        drop |= {"gate"}
    return {k: v for k, v in p.items() if k not in drop}


def check_forward(t, p, post, pre, drop=0.0, a=1.0, b=1.0, eps=1e-5, eps_post=1e-3, dtype=None):
    rows, n = t["x"].shape
    y = t.get("y")
    h, z = eb.block_norm(t["x"], y, post=post, pre=pre, epsilon=eps, epsilon_post=eps_post,
                         dropout=drop, seed=SEED, offset=OFFSET, stream_scale=a, branch_scale=b,
                         dtype=dtype, **p)
    a, b = float(torch.tensor(a)), float(torch.tensor(b))      # as binary32 holds them
    want_h, want_z = ref.block(t["x"], y, post, pre, float(torch.tensor(eps)),
                               float(torch.tensor(eps_post)), keep_of(drop, rows, n), a, b, **p)
    if y is not None:
        layer_ref.check(h, *want_h, steps(n), "h")
    else:
        assert h is None
    if pre == "none":
        assert z is None
    else:
        layer_ref.check(z, *want_z, steps(n), "z")
    return h, z


def check_gradient(t, p, post, pre, drop=0.0, a=1.0, b=1.0, eps=1e-5, eps_post=1e-3, dh=True):
    rows, n = t["x"].shape
    y = t.get("y")
    kind = t["dtype"] if y is None else y.dtype
    dz = matrix(21, rows, n, kind) if pre != "none" else None
    dh = matrix(22, rows, n, t["x"].dtype) if dh else None
    h = t["x"] if pre != "none" else None
    kw = dict(post=post, pre=pre, epsilon=eps, epsilon_post=eps_post, dropout=drop, seed=SEED,
              offset=OFFSET, stream_scale=a, branch_scale=b, **p)
    got = eb.block_norm_grad(dz, dh, h, y, **kw)
    again = eb.block_norm_grad(dz, dh, h, y, **kw)
    a, b = float(torch.tensor(a)), float(torch.tensor(b))
    want = ref.block_grad(dz, dh, h, y, post, pre, float(torch.tensor(eps)),
                          float(torch.tensor(eps_post)), keep_of(drop, rows, n), a, b, **p)
    for name, (value, scale) in want.items():
        k = steps(n) if name in ("x", "y") else steps(n) + rows
        layer_ref.check(got[name], value.reshape(got[name].shape), scale.reshape(got[name].shape),
                        k, "d" + name)
        assert torch.equal(got[name], again[name]), name
    assert {k for k, v in got.items() if v is not None} == set(want)
    return got


NORMS = [("none", "rms"), ("none", "layer"), ("rms", "rms"), ("layer", "layer"), ("rms", "none"),
         ("layer", "none"), ("none", "none"), ("rms", "layer")]
WIDTHS = [1, 2, 8, 31, 64, 256, 264, 520, 1021, 1152, 2048, 3080, 4096, 8192]
TYPES = [(BF16, BF16), (F16, F16), (F32, F32), (BF16, F32), (F16, F32)]


@pytest.mark.parametrize("dtype,stream", TYPES)
@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("post,pre", NORMS)
def test_widths(n, post, pre, dtype, stream):
    t, p = operands(12, n, dtype, stream, 3)
    p = valid(p, post, pre)
    check_forward(t, p, post, pre, 0.25, 0.9, 0.5)
    check_gradient(t, p, post, pre, 0.25, 0.9, 0.5)


@pytest.mark.parametrize("n", [9000, 16384, 16392, 20001, 32768, 40000])
@pytest.mark.parametrize("dtype,stream", TYPES)
def test_wide_rows(n, dtype, stream):
    t, p = operands(5, n, dtype, stream, 0)
    check_forward(t, p, "rms", "layer", 0.1)
    check_gradient(t, p, "layer", "rms", 0.1)


@pytest.mark.parametrize("n", [8200, 12288, 16384])
@pytest.mark.parametrize("post,pre", [("rms", "rms"), ("none", "layer")])
@pytest.mark.parametrize("dtype,stream", [(BF16, BF16), (F32, F32), (F16, F32)])
def test_many_wide_rows(n, post, pre, dtype, stream):
    t, p = operands(400, n, dtype, stream, 0)
    p = valid(p, post, pre)
    check_forward(t, p, post, pre)
    check_gradient(t, p, post, pre)


@pytest.mark.parametrize("how", ["strided", "odd stride", "off"])
@pytest.mark.parametrize("dtype,stream", TYPES)
@pytest.mark.parametrize("n", [40, 256, 1160])
def test_strides_and_alignment(n, how, dtype, stream):
    t, p = operands(10, n, dtype, stream, 2, how)
    check_forward(t, valid(p, "rms", "layer"), "rms", "layer", 0.1)
    check_gradient(t, p, "layer", "layer", 0.1)


@pytest.mark.parametrize("rows,groups", [(1, 1), (1, 0), (7, 7), (700, 1), (700, 100), (999, 3),
                                         (5000, 0), (5000, 5), (2049, 683)])
@pytest.mark.parametrize("n", [72, 1024])
def test_rows_and_groups(rows, groups, n):
    t, p = operands(rows, n, BF16, BF16, groups, mods=BF16, weights=BF16)
    check_forward(t, p, "rms", "rms")
    check_gradient(t, p, "rms", "rms")
    p = {k: v for k, v in p.items() if k in ("gate", "scale", "shift")}
    check_gradient(t, p, "layer", "layer", 0.1)


@pytest.mark.parametrize("dtype,stream", TYPES)
@pytest.mark.parametrize("n", [1, 7, 77, 256, 515, 1021, 2052, 4097, 8191])
@pytest.mark.parametrize("post,pre", [("none", "rms"), ("none", "layer"), ("rms", "rms"),
                                      ("layer", "layer")])
def test_many_ragged_rows(n, post, pre, dtype, stream):
    """Enough rows that a CTA walks several, each tensor off the vectors in a way of its own."""
    rows, groups = 636, 2
    t, p = operands(rows, n, dtype, stream, groups, weights=dtype, mods=dtype)
    t["x"] = matrix(31, rows, n, stream, "odd stride")
    t["y"] = matrix(32, rows, n, dtype, "off")
    p = valid(p, post, pre)
    h, z = check_forward(t, p, post, pre, 0.25, 0.9, 0.5)
    kw = dict(post=post, pre=pre, epsilon=1e-5, epsilon_post=1e-3, dropout=0.25, seed=SEED,
              offset=OFFSET, stream_scale=0.9, branch_scale=0.5, **p)
    for how_h, how_z in (("strided", "off"), ("odd stride", "odd stride")):
        oh, oz = matrix(33, rows, n, stream, how_h), matrix(34, rows, n, dtype, how_z)
        eb.block_norm(t["x"], t["y"], out=(oh, oz), **kw)
        assert torch.equal(oh, h) and torch.equal(oz, z)
    whole = torch.full((rows * n + 64,), 7.0, device="cuda", dtype=dtype)
    inside = whole[33:33 + rows * n].view(rows, n)
    eb.block_norm(t["x"], t["y"], out=(None, inside), **kw)
    assert torch.equal(inside, z)
    assert (whole[:33] == 7).all() and (whole[33 + rows * n:] == 7).all()
    got = check_gradient(t, p, post, pre, 0.25, 0.9, 0.5)
    dz, dh = matrix(21, rows, n, dtype), matrix(22, rows, n, stream)
    dx, dy = matrix(35, rows, n, stream, "off"), matrix(36, rows, n, dtype, "odd stride")
    eb.block_norm_grad(dz, dh, t["x"], t["y"], out=(dx, dy), **kw)
    assert torch.equal(dx, got["x"]) and torch.equal(dy, got["y"])


@pytest.mark.parametrize("n", [520, 523])
@pytest.mark.parametrize("rows", [305, 1000])
def test_many_rows_in_place(rows, n):
    t, p = operands(rows, n, BF16, BF16, 0)
    kw = dict(post="layer", pre="rms", dropout=0.1, **p)
    want = eb.block_norm(t["x"], t["y"], **kw)
    for ho, zo in (("x", "y"), ("y", "x")):
        c = {k: v.clone() for k, v in t.items()}
        for a, b in zip(eb.block_norm(c["x"], c["y"], out=(c[ho], c[zo]), **kw), want):
            assert torch.equal(a, b)
    dz, dh = matrix(21, rows, n, BF16), matrix(22, rows, n, BF16)
    want = eb.block_norm_grad(dz, dh, t["x"], t["y"], **kw)
    for names in (("dh", "y"), ("h", "dz"), ("dz", "dh"), ("y", "h")):
        c = {"dz": dz.clone(), "dh": dh.clone(), "h": t["x"].clone(), "y": t["y"].clone()}
        got = eb.block_norm_grad(c["dz"], c["dh"], c["h"], c["y"],
                                 out=(c[names[0]], c[names[1]]), **kw)
        for k in want:
            assert torch.equal(got[k], want[k]), (names, k)


def test_one_gate_beside_grouped_scales():
    for gate, mods in ((0, 4), (4, 0)):
        t, p = operands(48, 264, BF16, F32, gate)
        _, q = operands(48, 264, BF16, F32, mods)
        p.update(scale=q["scale"], shift=q["shift"])
        check_forward(t, p, "layer", "rms")
        check_gradient(t, p, "layer", "rms", 0.2)


@pytest.mark.parametrize("one", [("gate",), ("scale", "shift"), ("gate", "scale", "shift")])
@pytest.mark.parametrize("n", [264, 203])
def test_one_row_is_a_row_for_all(one, n):
    """A parameter [1, n] is the row [n], beside groups of the others."""
    t, p = operands(48, n, BF16, F32, 4)
    p.update({k: p[k][2:3] for k in one})
    flat = dict(p, **{k: p[k][0] for k in one})
    h, z = check_forward(t, p, "layer", "rms", 0.2)
    kw = dict(post="layer", pre="rms", epsilon=1e-5, epsilon_post=1e-3, dropout=0.2, seed=SEED,
              offset=OFFSET)
    for a, b in zip(eb.block_norm(t["x"], t["y"], **kw, **flat), (h, z)):
        assert torch.equal(a, b)
    got = check_gradient(t, p, "layer", "rms", 0.2)
    dz, dh = matrix(21, 48, n, BF16), matrix(22, 48, n, F32)
    want = eb.block_norm_grad(dz, dh, t["x"], t["y"], **kw, **flat)
    for k, v in want.items():
        assert torch.equal(got[k].view(v.shape), v), k


@pytest.mark.parametrize("given", [(), ("w_pre",), ("b_pre",), ("b_post",), ("w_post", "gate"),
                                   ("scale",), ("shift",), ("gate",), ("gate", "b_post", "shift")])
@pytest.mark.parametrize("n", [200, 203])
def test_parameters_left_out(given, n):
    t, p = operands(20, n, BF16, BF16, 2, weights=BF16, mods=BF16)
    p = {k: v for k, v in p.items() if k in given}
    check_forward(t, p, "rms", "layer", 0.1)
    check_gradient(t, p, "rms", "layer", 0.1)
    check_gradient(t, p, "rms", "layer", dh=False)


@pytest.mark.parametrize("dtype,stream", TYPES)
@pytest.mark.parametrize("n", [264, 33])
def test_without_a_branch(n, dtype, stream):
    t, p = operands(30, n, dtype, stream, 3)
    del t["y"]
    t["dtype"] = dtype
    p = valid(p, "none", "layer", branch=False)
    check_forward(t, p, "none", "layer", a=1.5, dtype=dtype)
    check_gradient(t, p, "none", "layer", a=1.5)
    check_gradient(t, p, "none", "rms", dh=False)


def test_views_of_one_projection():
    """gate, scale and shift as parts of a condition's projection [groups, 6 n]."""
    t, p = operands(24, 256, BF16, BF16, 4, affine=False)
    all6 = (0.5 * normal(30, 4, 6 * 256)).to(BF16)
    p = {"gate": all6[:, 512:768], "scale": all6[:, :256], "shift": all6[:, 1024:1280]}
    check_forward(t, p, "none", "layer")
    check_gradient(t, p, "none", "layer")


@pytest.mark.parametrize("n", [1024, 1000, 333])
@pytest.mark.parametrize("middle", [100.0, -3000.0])
def test_rows_far_from_zero(n, middle):
    """A mean of thousands of deviations costs a layer norm its share of the bound, no more."""
    t, p = operands(16, n, F32, F32, 0, middle=middle)
    check_forward(t, p, "layer", "layer")
    check_gradient(t, p, "layer", "layer")


@pytest.mark.parametrize("n", [512, 77])
def test_rows_of_zeros_and_of_one_value(n):
    for fill in (0.0, 0.75):
        t, p = operands(8, n, BF16, BF16, 0)
        for x in t.values():
            x[::2] = fill
        check_forward(t, valid(p, "rms", "rms"), "rms", "rms")
        check_forward(t, p, "layer", "layer")
        check_gradient(t, p, "layer", "layer")
    z = eb.block_norm(torch.zeros(3, n, device="cuda"), pre="layer")[1]
    assert (z == 0).all()


@pytest.mark.parametrize("n", [512, 77])
def test_bad_rows_stay_alone(n):
    """NaN and infinities of a row reach no other row; dropped elements of a branch without
    a norm add exactly 0."""
    t, p = operands(9, n, BF16, BF16, 0)
    good = eb.block_norm(t["x"], t["y"], post="rms", pre="rms")
    t["y"][4, 3], t["x"][6, 5] = float("nan"), float("inf")
    bad = eb.block_norm(t["x"], t["y"], post="rms", pre="rms")
    rest = [i for i in range(9) if i not in (4, 6)]
    for a, b in zip(good, bad):
        assert torch.equal(a[rest], b[rest])
    assert bad[0][4].isnan().all() and bad[1][6].isnan().any()
    m = keep_of(0.5, 9, n)
    y = normal(50, 9, n)
    broken = torch.where(m == 0, torch.full_like(y, float("inf")), y)
    kw = dict(pre="rms", dropout=0.5, seed=SEED, offset=OFFSET)
    for a, b in zip(eb.block_norm(y, y, **kw), eb.block_norm(y, broken, **kw)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("rows,groups", [(9, 0), (9, 9), (700, 0)])
@pytest.mark.parametrize("n", [512, 1543, 9000, 16400])
@pytest.mark.parametrize("post", ["none", "rms", "layer"])
def test_dropped_places_add_nothing_to_gradients(post, n, rows, groups):
    """Infinities and NaN of dh, and without a norm after the block of y, in dropped places: the
    gradients of y and of every parameter are those of finite numbers there."""
    t, p = operands(rows, n, BF16, F32, groups)
    p = valid(p, post, "rms")
    gone = keep_of(0.5, rows, n) == 0
    dz, dh = matrix(61, rows, n, BF16), normal(62, rows, n)
    h, y = t["x"], t["y"].contiguous()
    kw = dict(post=post, pre="rms", dropout=0.5, seed=SEED, offset=OFFSET, **p)
    want = eb.block_norm_grad(dz, torch.where(gone, 0.0, dh), h,
                              torch.where(gone, 0.0, y) if post == "none" else y, **kw)
    assert all(v.isfinite().all() for v in want.values() if v is not None)
    for bad in (float("inf"), float("nan")):
        got = eb.block_norm_grad(dz, torch.where(gone, bad, dh), h,
                                 torch.where(gone, bad, y) if post == "none" else y, **kw)
        for name, value in want.items():
            if name == "x":
                assert torch.equal(got[name][~gone], value[~gone])
                assert not got[name][gone].isfinite().any()
            elif value is not None:
                assert torch.equal(got[name], value), name


@pytest.mark.parametrize("n", [1024, 1021, 16384, 20000])
def test_in_place(n):
    t, p = operands(21, n, BF16, BF16, 3)
    kw = dict(post="rms", pre="layer", **p)
    want = eb.block_norm(t["x"], t["y"], **kw)
    for ho, zo in (("x", "y"), ("y", "x"), ("x", None), (None, "x")):
        c = {k: v.clone() for k, v in t.items()}
        got = eb.block_norm(c["x"], c["y"], out=(ho and c[ho], zo and c[zo]), **kw)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    dz, dh = matrix(21, 21, n, BF16), matrix(22, 21, n, BF16)
    want = eb.block_norm_grad(dz, dh, t["x"], t["y"], **kw)
    for names in (("dh", "y"), ("h", "dz"), ("dz", "dh"), ("y", "h")):
        c = {"dz": dz.clone(), "dh": dh.clone(), "h": t["x"].clone(), "y": t["y"].clone()}
        got = eb.block_norm_grad(c["dz"], c["dh"], c["h"], c["y"],
                                 out=(c[names[0]], c[names[1]]), **kw)
        for k in want:
            assert torch.equal(got[k], want[k]), (names, k)


def test_what_is_around_the_rows_stays():
    n, rows = 264, 37
    t, p = operands(rows, n, BF16, F32, 0)
    wide_h = torch.full((rows + 2, n + 16), 7.0, device="cuda")
    wide_z = torch.full((rows + 2, n + 16), 7.0, device="cuda", dtype=BF16)
    h, z = wide_h[1:-1, 8:-8], wide_z[1:-1, 8:-8]
    want = eb.block_norm(t["x"], t["y"], **valid(p, "none", "rms"))
    eb.block_norm(t["x"], t["y"], out=(h, z), **valid(p, "none", "rms"))
    assert torch.equal(h, want[0]) and torch.equal(z, want[1])
    for w in (wide_h, wide_z):
        w[1:-1, 8:-8] = 7
        assert (w == 7).all()


@pytest.mark.parametrize("post,pre", [("rms", "rms"), ("layer", "layer"), ("none", "layer")])
def test_gradient_against_differences(post, pre):
    """The gradient's products with directions against central differences of the 64-bit
    forward form, h = 1e-5: h^2 and 1e-11 / h apart from float32's own share."""
    rows, n, eps = 12, 96, 1e-4
    t, p = operands(rows, n, F32, F32, 3)
    p = valid(p, post, pre)
    dz, dh = matrix(21, rows, n, F32), matrix(22, rows, n, F32)
    m = keep_of(0.3, rows, n)
    both = dict(p, x=t["x"], y=t["y"])
    way = {k: normal(60 + i, *v.shape) for i, (k, v) in enumerate(both.items())}

    def forward(s):
        q = {k: v.double() + s * way[k].double() for k, v in both.items()}
        x, y = q.pop("x"), q.pop("y")
        h, z = ref.block(x, y, post, pre, eps, eps, m, 0.9, 0.5, **q)
        return h[0], z[0]

    def loss(s):
        h, z = forward(s)
        return float((dh.double() * h).sum() + (dz.double() * z).sum())

    h = forward(0.0)[0].float()
    got = eb.block_norm_grad(dz, dh, h, t["y"], post=post, pre=pre, epsilon=eps, dropout=0.3,
                             seed=SEED, offset=OFFSET, stream_scale=0.9, branch_scale=0.5, **p)
    along = sum(float((got[k].double() * way[k].double()).sum()) for k in both)
    differ = (loss(1e-5) - loss(-1e-5)) / 2e-5
    assert abs(along - differ) < 1e-4 * math.sqrt(rows * n) * max(1.0, abs(differ)) ** 0.5


def test_graphs_streams_and_workspaces_apart():
    """Two captured steps with a workspace each, replayed on two streams at once."""
    n, rows = 512, 600
    sides, graphs, outs = [torch.cuda.Stream() for _ in range(2)], [], []
    t, p = operands(rows, n, BF16, BF16, 2)
    dz, dh = matrix(21, rows, n, BF16), matrix(22, rows, n, BF16)
    word = torch.zeros(1, dtype=torch.int64, device="cuda")
    kw = dict(post="rms", pre="layer", dropout=0.1)
    fwd = eb.BlockNormPlan(BF16, rows, n, weight_dtype=F32, mod_dtype=F32, gate_rows=rows // 2,
                           mod_rows=rows // 2, **kw)
    bwd = eb.BlockNormPlan(BF16, rows, n, weight_dtype=F32, mod_dtype=F32, gate_rows=rows // 2,
                           mod_rows=rows // 2, gradient=True, **kw)
    for side in sides:
        h, z, dx, dy = (torch.empty(rows, n, dtype=BF16, device="cuda") for _ in range(4))
        g = {"d" + k: torch.empty(v.shape, device="cuda") for k, v in p.items()}
        work = torch.empty(bwd.workspace_bytes, dtype=torch.uint8, device="cuda")
        q = {k: v for k, v in p.items() if k != "shift"}

        def step():
            eb.execute_block_norm(fwd, t["x"], t["y"], h, z, seed=SEED, offset=3,
                                  offset_device=word, **p)
            eb.execute_block_norm_grad(bwd, dz, dh, h, t["y"], dx, dy, workspace=work, seed=SEED,
                                       offset=3, offset_device=word, **q, **g)

        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        graphs.append(graph)
        outs.append((h, z, dx, dy, g))
    word.fill_(9)
    torch.cuda.synchronize()
    for _ in range(3):
        for side, graph in zip(sides, graphs):
            with torch.cuda.stream(side):
                graph.replay()
    torch.cuda.synchronize()
    h, z = eb.block_norm(t["x"], t["y"], seed=SEED, offset=12, **kw, **p)
    want = eb.block_norm_grad(dz, dh, h, t["y"], seed=SEED, offset=12, **kw, **p)
    for oh, oz, dx, dy, g in outs:
        assert torch.equal(oh, h) and torch.equal(oz, z)
        assert torch.equal(dx, want["x"]) and torch.equal(dy, want["y"])
        for k in p:
            assert torch.equal(g["d" + k], want[k])
    s = sides[0]
    s.wait_stream(torch.cuda.current_stream())
    got = eb.block_norm(t["x"], t["y"], seed=SEED, offset=12, stream=s, **kw, **p)
    s.synchronize()
    assert torch.equal(got[0], h) and torch.equal(got[1], z)


def test_empty_shapes():
    for rows, n in ((0, 16), (4, 0), (0, 0)):
        x, y = (torch.empty(rows, n, dtype=BF16, device="cuda") for _ in range(2))
        w, gate = torch.ones(n, device="cuda"), torch.ones(2, n, device="cuda")
        h, z = eb.block_norm(x, y, w_pre=w, gate=gate)
        assert h.shape == z.shape == x.shape
        g = eb.block_norm_grad(y, x, h, y, w_pre=w, gate=gate)
        assert g["x"].shape == x.shape and (g["w_pre"] == 0).all() and (g["gate"] == 0).all()
        assert g["gate"].shape == gate.shape


def test_an_empty_batch():
    """No sequences: no rows and no groups; a row for all has a gradient of 0."""
    x, y, none = (torch.empty(0, 64, dtype=BF16, device="cuda") for _ in range(3))
    one = torch.ones(1, 64, dtype=BF16, device="cuda")
    for kw in (dict(gate=none, scale=none, shift=none), dict(gate=none, scale=one, shift=one),
               dict(gate=one, scale=none), dict(gate=one[0], shift=none)):
        h, z = eb.block_norm(x, y, pre="layer", **kw)
        assert h.shape == z.shape == x.shape
        g = eb.block_norm_grad(y, x, h, y, pre="layer", **kw)
        for k, t in kw.items():
            assert g[k].shape == t.shape and (g[k] == 0).all()


def test_outputs_that_are_not_wanted():
    t, p = operands(33, 264, BF16, BF16, 0)
    kw = dict(weight_dtype=F32, mod_dtype=F32, post="rms", pre="layer")
    fwd, bwd = eb.BlockNormPlan(BF16, 33, 264, **kw), eb.BlockNormPlan(BF16, 33, 264, gradient=True,
                                                                      **kw)
    h, z = eb.block_norm(t["x"], t["y"], post="rms", pre="layer", **p)
    for want_h, want_z in ((True, False), (False, True), (False, False)):
        a, b = torch.empty_like(h), torch.empty_like(z)
        eb.execute_block_norm(fwd, t["x"], t["y"], a if want_h else None, b if want_z else None,
                              **p)
        assert not want_h or torch.equal(a, h)
        assert not want_z or torch.equal(b, z)
    dz, dh = matrix(21, 33, 264, BF16), matrix(22, 33, 264, BF16)
    want = eb.block_norm_grad(dz, dh, h, t["y"], post="rms", pre="layer", **p)
    q = {k: v for k, v in p.items() if k != "shift"}
    work = torch.empty(bwd.workspace_bytes, dtype=torch.uint8, device="cuda")
    for only in ("x", "y", "gate", "w_post", "b_post", "w_pre", "b_pre", "scale", "shift"):
        out = torch.empty_like(want[only])
        kw = {"d" + only: out, "workspace": work} if only not in ("x", "y") else {}
        eb.execute_block_norm_grad(bwd, dz, dh, h, t["y"], out if only == "x" else None,
                                   out if only == "y" else None, **q, **kw)
        assert torch.equal(out, want[only]), only


@pytest.mark.parametrize("dtype,stream", TYPES)
@pytest.mark.parametrize("rows,n", [(30, 264), (30, 33), (5000, 1536), (2500, 4097), (9, 40000)])
def test_the_stream_alone_scaled_and_normed(rows, n, dtype, stream):
    """Without a branch h is stream_scale x, where a tensor for it is given: x itself too."""
    t, p = operands(rows, n, dtype, stream, 0)
    p = valid(p, "none", "layer", branch=False)
    kw = dict(pre="layer", stream_scale=1.5, dtype=dtype, **p)
    alone, z = eb.block_norm(t["x"], **kw)
    assert alone is None
    want = (1.5 * t["x"].double()).to(stream)
    h, again = eb.block_norm(t["x"], out=(torch.empty_like(t["x"]), None), **kw)
    assert torch.equal(h, want) and torch.equal(again, z)
    x = t["x"].clone()
    h, again = eb.block_norm(x, out=(x, None), **kw)
    assert h is x and torch.equal(x, want) and torch.equal(again, z)
