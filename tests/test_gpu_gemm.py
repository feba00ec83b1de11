"""Matrix products with an epilogue on the GPU against a plain 64-bit form.

Bounds: the output type's rounding, plus binary32 roundings.  Products of
16-bit values are exact in binary32; a sum of k of them is off by at most
(k + 4) 2^-23 of the sum of magnitudes in any order, with truncation allowed
for (tests use that times 1.1).  An activation of slope at most 1.13 passes
that on, and adds its own error: a few units of 2^-23 of |z| (the fast
exponential, the quotient, erf), 16 allowed.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

import broadcast_elementwise_gb300 as eb  # noqa: E402
import layer_ref as ref  # noqa: E402

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def matrix(g, rows, cols, dtype, how, trans=False):
    """A matrix (stored transposed with trans): dense, with a row stride, or
    one element off every alignment."""
    r, c = (cols, rows) if trans else (rows, cols)
    if how == "strided":
        return normal(g, r, c + 24, dtype=dtype)[:, 8:8 + c]
    if how == "odd":
        return normal(g, r * (c + 3) + 1, dtype=dtype)[1:].view(r, c + 3)[:, :c]
    return normal(g, r, c, dtype=dtype)


def reference(a, b, bias, res, kind, ta, tb):
    """(z, y, bound scale of z, of y) in 64 bits."""
    A = (a.t() if ta else a).double()
    B = (b.t() if tb else b).double()
    z, sz = A @ B, A.abs() @ B.abs()
    if bias is not None:
        z, sz = z + bias.double(), sz + bias.double().abs()
    k = A.shape[1]
    sum_error = sz * (k + 4) * 2 * ref.F32
    y = ref.act(z, kind)
    y_error = 1.13 * sum_error + (0 if kind == "none" else 32 * ref.F32 * z.abs())
    if res is not None:
        y = y + res.double()
        y_error = y_error + 2 * ref.F32 * y.abs()
    return z, y, sum_error, y_error


def check(got, want, error, what):
    ref.check(got, want, error / ref.F32, 1, what)


SIZES = [(1, 1, 1), (1, 64, 64), (1, 4096, 512), (2, 130, 96), (3, 33, 7), (4, 512, 1024),
         (7, 96, 4096), (16, 256, 256), (17, 200, 520), (33, 1000, 72), (64, 384, 640),
         (65, 129, 200), (100, 100, 100), (128, 128, 128), (129, 257, 65), (200, 72, 1000),
         (256, 512, 64), (300, 520, 1032), (513, 300, 321), (1024, 1024, 256), (640, 2304, 128),
         (2049, 257, 40), (1, 7, 100), (5, 8, 2048), (1500, 1, 64)]


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("ta,tb", [(False, False), (False, True), (True, False), (True, True)])
def test_product(size, ta, tb):
    m, n, k = size
    g = gen(1)
    dtype = BF16 if (m + n) % 2 else F16
    a, b = matrix(g, m, k, dtype, "dense", ta), matrix(g, k, n, dtype, "dense", tb)
    z, y, ez, ey = reference(a, b, None, None, "none", ta, tb)
    got = eb.gemm(a, b, trans_a=ta, trans_b=tb)
    check(got, y, ey, "product")
    assert torch.equal(got, eb.gemm(a, b, trans_a=ta, trans_b=tb))
    assert eb.get_device_status() == 0


# one size for every tile and split that the plan can pick on 152 SMs, and the
# paired tiles once more where n lets rows go out in vectors
TILES = [(270, 3650, 520), (270, 3648, 520), (779, 5700, 264), (779, 5696, 264),
         (1672, 5572, 520), (1672, 5568, 520), (561, 4838, 1032), (561, 4832, 1032),
         (2634, 1397, 4096), (2634, 1392, 4096), (82, 16, 40), (68, 5117, 264), (68, 5120, 264),
         (272, 5164, 200), (4844, 43, 4096), (2418, 18, 2048), (70, 16, 2048), (1, 17, 40),
         (1, 4647, 2048), (1, 16, 1032), (1, 16, 2048), (20, 17, 40), (17, 4705, 2048),
         (20, 16, 1032), (22, 17, 2048), (36, 16, 40), (34, 4704, 2048), (35, 16, 1032),
         (34, 16, 2048), (561, 4838, 2048), (561, 4832, 2048), (346, 5212, 520), (65, 7305, 4096)]


@pytest.mark.parametrize("size", TILES, ids=str)
@pytest.mark.parametrize("ta,tb", [(False, False), (False, True), (True, False), (True, True)])
def test_every_tile(size, ta, tb):
    m, n, k = size
    g = gen(11)
    dtype = BF16 if (ta + tb) % 2 else F16
    a = matrix(g, m, k, dtype, "dense", ta)
    b = (matrix(g, k, n, F32, "dense", tb) / math.sqrt(k)).to(dtype)
    bias, r = normal(g, n), normal(g, m, n, dtype=dtype)
    pre = torch.empty(m, n, dtype=dtype, device="cuda")
    z, y, ez, ey = reference(a, b, bias, r, "gelu", ta, tb)
    got = eb.gemm(a, b, bias, r, trans_a=ta, trans_b=tb, activation="gelu", preact=pre)
    check(got, y, ey, "y")
    check(pre, z, ez, "z")
    assert torch.equal(got, eb.gemm(a, b, bias, r, trans_a=ta, trans_b=tb, activation="gelu"))
    assert eb.get_device_status() == 0


def test_output_past_32_bits():
    """y of over 2^31 elements: the last rows against the same rows alone."""
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB of device memory")
    g = gen(12)
    m, n, k = 70016, 32768, 64
    a, b = normal(g, m, k, dtype=BF16), normal(g, n, k, dtype=BF16)
    y = eb.gemm(a, b, trans_b=True)
    for rows in (slice(0, 256), slice(65536, 65792), slice(m - 256, m)):
        assert torch.equal(y[rows], eb.gemm(a[rows], b, trans_b=True))
    dz, _ = eb.gemm_epilogue_grad(y, y, activation="relu", out=y)
    for rows in (slice(0, 256), slice(m - 256, m)):
        want = eb.gemm(a[rows], b, trans_b=True)
        assert torch.equal(dz[rows], want.clamp_min(0))


@pytest.mark.parametrize("size", [(1, 512, 768), (9, 264, 512), (70, 130, 200), (260, 520, 136),
                                  (1100, 700, 264)], ids=str)
@pytest.mark.parametrize("kind", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype,bias_dtype,res", [(BF16, BF16, True), (F16, F32, False),
                                                  (F16, None, True), (BF16, F32, False)])
def test_epilogue(size, kind, dtype, bias_dtype, res):
    m, n, k = size
    g = gen(2)
    a = normal(g, m, k, dtype=dtype)
    b = (normal(g, n, k) * (3 / math.sqrt(k))).to(dtype)
    bias = None if bias_dtype is None else normal(g, n).to(bias_dtype)
    r = normal(g, m, n, dtype=dtype) if res else None
    z, y, ez, ey = reference(a, b, bias, r, kind, False, True)
    pre = torch.empty(m, n, dtype=dtype, device="cuda")
    got = eb.gemm(a, b, bias, r, trans_b=True, activation=kind, preact=pre)
    check(got, y, ey, kind)
    check(pre, z, ez, "pre-activation")
    # without the pre-activation the same y
    assert torch.equal(got, eb.gemm(a, b, bias, r, trans_b=True, activation=kind))


@pytest.mark.parametrize("how", ["strided", "odd"])
@pytest.mark.parametrize("ta,tb", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("size", [(5, 130, 264), (200, 310, 130)], ids=str)
def test_strides_and_alignment(size, how, ta, tb):
    m, n, k = size
    g = gen(3)
    a, b = matrix(g, m, k, BF16, how, ta), matrix(g, k, n, BF16, how, tb)
    bias, r = normal(g, n), matrix(g, m, n, BF16, how)
    out, pre = matrix(g, m, n, BF16, how), matrix(g, m, n, BF16, how)
    frame = out._base.clone()
    z, y, ez, ey = reference(a, b, bias, r, "silu", ta, tb)
    eb.gemm(a, b, bias, r, trans_a=ta, trans_b=tb, activation="silu", out=out, preact=pre)
    check(out, y, ey, "y")
    check(pre, z, ez, "z")
    # nothing outside the output's elements is written
    now = out._base.clone()
    out.zero_()
    cleared = out._base.clone()
    inside = cleared != now
    assert torch.equal(now[~inside & (cleared != 0)], frame[~inside & (cleared != 0)])


def test_residual_in_place_and_empty():
    g = gen(4)
    a, b, r = normal(g, 70, 64, dtype=F16), normal(g, 64, 96, dtype=F16), normal(g, 70, 96, dtype=F16)
    want = eb.gemm(a, b, None, r)
    eb.gemm(a, b, None, r, out=r)
    assert torch.equal(r, want)
    bias = normal(g, 96, dtype=F16)
    got = eb.gemm(a[:, :0], b[:0], bias, activation="relu")       # k = 0: z is the bias
    assert torch.equal(got, bias.clamp_min(0).expand(70, 96))
    assert (eb.gemm(a[:, :0], b[:0]) == 0).all()
    assert eb.gemm(a[:0], b).shape == (0, 96)
    assert eb.gemm(a, b[:, :0]).shape == (70, 0)


def test_infinities_and_nans_stay_in_their_rows():
    g = gen(5)
    for m, n, k in ((40, 200, 160), (3, 300, 1024), (300, 520, 70)):
        a, b = normal(g, m, k, dtype=BF16), normal(g, n, k, dtype=BF16)
        clean = eb.gemm(a, b, trans_b=True)
        bad = a.clone()
        bad[1, 3] = math.nan
        bad[2, k - 1] = math.inf
        got = eb.gemm(bad, b, trans_b=True)
        assert got[1].isnan().all()
        assert not got[2].isfinite().any()
        keep = torch.ones(m, dtype=torch.bool, device="cuda")
        keep[1] = keep[2] = False
        assert torch.equal(got[keep], clean[keep])


def test_large_values_overflow_to_infinity():
    a = torch.full((3, 64), 200.0, dtype=F16, device="cuda")
    b = torch.full((64, 130), 200.0, dtype=F16, device="cuda")
    assert (eb.gemm(a, b) == math.inf).all()          # 64 * 40000 passes 65504
    bias = torch.full((130,), -64 * 40000.0, device="cuda")
    assert (eb.gemm(a, b, bias) == 0).all()           # held in 32 bits until the end


def test_another_stream_and_a_graph():
    g = gen(6)
    a, b = normal(g, 130, 256, dtype=BF16), normal(g, 300, 256, dtype=BF16)
    want = eb.gemm(a, b, trans_b=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    plan = eb.GemmPlan(BF16, 130, 300, 256, trans_b=True)
    work = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(want)
    with torch.cuda.stream(s):
        eb.execute_gemm(plan, a, b, out, workspace=work)
    s.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        eb.execute_gemm(plan, a, b, out, workspace=work)
    a.copy_(normal(g, 130, 256))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eb.gemm(a, b, trans_b=True))


def test_back_to_back_products_read_each_other():
    """Launches overlap at their ends; each reads what the one before wrote."""
    g = gen(7)
    w = [(normal(g, 512, 512) / math.sqrt(512)).to(BF16) for _ in range(6)]
    x = normal(g, 300, 512, dtype=BF16)
    for _ in range(3):
        steps, y = [], x
        for m in w:
            y = eb.gemm(y, m, trans_b=True, activation="silu")
            steps.append(y)
        torch.cuda.synchronize()
        y = x
        for m, s in zip(w, steps):
            z, want, ez, ey = reference(y, m, None, None, "silu", False, True)
            check(s, want, ey, "chain")
            y = s


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("kind", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("m,n", [(1, 1), (1, 300), (37, 64), (513, 136), (1000, 2052), (70, 33)])
def test_epilogue_gradient(m, n, kind, dtype):
    """dz: 24 binary32 roundings of |dy| (1 + |z| |act''|-like terms, at most
    2 |z| + 2); dbias: a thread adds its rows, then warps and CTAs join."""
    g = gen(8)
    dy, z = normal(g, m, n, dtype=dtype), (2 * normal(g, m, n)).to(dtype)
    dz, db = eb.gemm_epilogue_grad(dy, z, activation=kind)
    want = dy.double() * ref.act_slope(z.double(), kind)
    scale = dy.double().abs() * (2 + 2 * z.double().abs())
    ref.check(dz, want, scale, 24, "dz")
    ref.check(db, want.sum(0), scale.sum(0), 24 + m, "dbias")
    again = eb.gemm_epilogue_grad(dy, z, activation=kind)
    assert torch.equal(dz, again[0]) and torch.equal(db, again[1])
    assert torch.equal(dz, eb.gemm_epilogue_grad(dy, z, activation=kind, bias=False)[0])


@pytest.mark.parametrize("kind", ["relu", "gelu", "gelu_tanh", "silu"])
def test_slopes_far_out(kind):
    """Large pre-activations: the slope is 0 or 1 there, never a NaN."""
    z = torch.tensor([[-3e38, -1e30, -1e5, -60.0, -20.0, 0.0, 20.0, 60.0, 1e5, 1e30, 3e38]],
                     device="cuda")
    dz, _ = eb.gemm_epilogue_grad(torch.ones_like(z), z, activation=kind)
    want = ref.act_slope(z.double().clamp(-1e6, 1e6), kind)
    assert ((dz.double() - want).abs() <= 1e-6).all(), dz


def test_epilogue_gradient_strided_in_place_and_empty():
    g = gen(9)
    dy, z = matrix(g, 50, 70, BF16, "odd"), matrix(g, 50, 70, BF16, "strided")
    dz, db = eb.gemm_epilogue_grad(dy, z, activation="gelu")
    got, gb = eb.gemm_epilogue_grad(dy, z, activation="gelu", out=dy)
    assert torch.equal(got, dz) and torch.equal(db, gb)
    dz, db = eb.gemm_epilogue_grad(dy[:0], z[:0], activation="gelu")
    assert dz.shape == (0, 70) and (db == 0).all()


@pytest.mark.parametrize("kind", ["gelu", "gelu_tanh", "silu"])
def test_gradient_against_differences(kind):
    """The whole layer's gradient (dz, dx, dw, dbias) against central
    differences of the 64-bit forward form.  The kernels' results are rounded
    to float16 (2^-11 each, dz's rounding included): their projections on
    random directions are off by about 2^-11 sqrt(2) of the summed squares;
    6 standard deviations are allowed."""
    g = gen(10)
    m, n, k = 24, 40, 32
    x, w = normal(g, m, k, dtype=F16), (normal(g, n, k) / math.sqrt(k)).to(F16)
    bias, dy = normal(g, n, dtype=F16), normal(g, m, n, dtype=F16)
    z = torch.empty(m, n, dtype=F16, device="cuda")
    eb.gemm(x, w, bias, trans_b=True, activation=kind, preact=z)
    dz, db = eb.gemm_epilogue_grad(dy, z, activation=kind)
    dx = eb.gemm(dz, w)                       # [m, n] [n, k]
    dw = eb.gemm(dz, x, trans_a=True)         # [n, m] [m, k]
    v = {"x": normal(g, m, k).double(), "w": normal(g, n, k).double(), "b": normal(g, n).double()}

    def loss(h, which):
        d = {key: h * (key == which) for key in v}
        zz = ((x.double() + d["x"] * v["x"]) @ (w.double() + d["w"] * v["w"]).t()
              + bias.double() + d["b"] * v["b"])
        return float((dy.double() * ref.act(zz, kind)).sum())

    h = 1e-5
    for which, got in (("x", dx), ("w", dw), ("b", db)):
        d = (loss(h, which) - loss(-h, which)) / (2 * h)
        p = got.double() * v[which]
        # z's own rounding moves dz by up to 2^-11 |z| of a slope's change
        spread = float((p * p).sum().sqrt()) * 2 ** -11 * 6 * 3
        assert abs(float(p.sum()) - d) <= spread + 1e-6 * abs(d), (which, float(p.sum()), d)
