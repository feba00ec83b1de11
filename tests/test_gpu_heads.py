"""Rotary positions and head norms on the GPU against a plain 64-bit form.

Bounds: the output type's rounding of the true value, plus the binary32
roundings of the formula scaled by the magnitudes that enter it.  A rotation
takes 3 roundings (tests allow 4); the norm's sum of head_dim squares, its
square root and the products take at most head_dim / 8 + 16 (a lane sums at
most an eighth of a head, then the lanes join in a tree).
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


def views(g, B, S, Hq, Hk, D, dtype, how):
    """q and k as dense tensors, as views of one packed projection, as
    [B, H, S, D] storage, or one element off every alignment."""
    if how == "packed":
        x = normal(g, B, S, (Hq + 2 * Hk) * D, dtype=dtype)
        return (x[..., :Hq * D].unflatten(-1, (Hq, D)),
                x[..., Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D)))
    if how == "heads_first":
        return (normal(g, B, Hq, S, D, dtype=dtype).transpose(1, 2),
                normal(g, B, Hk, S, D, dtype=dtype).transpose(1, 2))
    if how == "odd":
        x = normal(g, B * S * (Hq + Hk) * D + 1, dtype=dtype)[1:]
        return (x[:B * S * Hq * D].view(B, S, Hq, D), x[B * S * Hq * D:].view(B, S, Hk, D))
    return normal(g, B, S, Hq, D, dtype=dtype), normal(g, B, S, Hk, D, dtype=dtype)


def tables(length, r):
    c, s = ref.table(length, r)
    return c.float().cuda(), s.float().cuda()


def rows(table, positions):
    return table.double()[positions.long()]


SHAPES = [
    # B, S, Hq, Hk, D, r, layout, how
    (1, 1, 1, 1, 2, 2, "half", "dense"),
    (1, 1, 32, 8, 128, 128, "half", "dense"),
    (16, 1, 32, 8, 128, 128, "half", "packed"),
    (2, 37, 4, 2, 64, 64, "half", "dense"),
    (2, 37, 4, 2, 64, 32, "interleaved", "packed"),
    (3, 5, 6, 3, 80, 80, "half", "heads_first"),
    (3, 5, 7, 1, 96, 48, "half", "dense"),
    (3, 5, 7, 1, 96, 46, "half", "dense"),
    (3, 5, 7, 1, 96, 46, "interleaved", "dense"),
    (2, 9, 5, 5, 112, 54, "half", "packed"),
    (1, 33, 3, 1, 256, 256, "interleaved", "dense"),
    (1, 33, 3, 1, 256, 64, "half", "dense"),
    (2, 17, 3, 3, 192, 192, "half", "odd"),
    (2, 17, 3, 3, 64, 64, "interleaved", "odd"),
    (2, 3, 5, 2, 33, 22, "half", "dense"),
    (2, 3, 5, 2, 33, 22, "interleaved", "dense"),
    (2, 3, 2, 1, 520, 520, "half", "dense"),
    (2, 3, 2, 1, 1024, 1000, "interleaved", "dense"),
    (1, 2, 1, 1, 1, 0, "half", "dense"),
    (1, 700, 9, 3, 32, 14, "half", "dense"),
    (1, 700, 9, 3, 32, 32, "half", "packed"),
    (1, 130, 40, 8, 72, 36, "half", "dense"),
    (1, 130, 40, 8, 40, 40, "interleaved", "dense"),
    (1, 61, 4, 4, 8, 8, "half", "dense"),
    (1, 61, 4, 4, 16, 8, "interleaved", "dense"),
]

# enough rows that groups of lanes walk several items each
MANY = [
    (2, 4096, 32, 8, 128, 128, "half", "packed"),
    (1, 9001, 20, 5, 96, 46, "half", "dense"),
    (3, 4099, 13, 3, 80, 40, "interleaved", "packed"),
    (1, 12001, 9, 9, 64, 32, "half", "heads_first"),
]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("shape", SHAPES + MANY, ids=str)
@pytest.mark.parametrize("gradient", [False, True])
def test_rotary(shape, dtype, gradient):
    B, S, Hq, Hk, D, r, layout, how = shape
    if r == 0:
        pytest.skip("nothing to rotate")
    g = gen(1)
    q, k = views(g, B, S, Hq, Hk, D, dtype, how)
    cos, sin = tables(4 * S + 3, r)
    at = torch.randint(0, 4 * S + 3, (B, S), generator=g, device="cuda", dtype=torch.int32)
    got = eb.rotary(q, k, cos, sin, at, layout=layout, gradient=gradient)
    c, s = rows(cos, at), rows(sin, at)
    for x, y in zip((q, k), got):
        want = ref.rotate(x.double(), c, s, layout, -1.0 if gradient else 1.0)
        ref.check(y, want, ref.spread(x.double(), c, s, layout), 4, "rotary")
    assert eb.get_device_status() == 0


@pytest.mark.parametrize("dtype,wdtype", [(BF16, BF16), (F16, F32), (F32, F32), (BF16, None)])
@pytest.mark.parametrize("shape", SHAPES + MANY, ids=str)
def test_norm_rotary(shape, dtype, wdtype):
    B, S, Hq, Hk, D, r, layout, how = shape
    g = gen(2)
    q, k = views(g, B, S, Hq, Hk, D, dtype, how)
    wq = wk = None
    if wdtype is not None:
        wq, wk = ((1 + 0.3 * normal(g, D)).to(wdtype) for _ in range(2))
    cos, sin = tables(S + 3, r) if r else (None, None)
    at = torch.randint(0, S + 3, (B, S), generator=g, device="cuda") if r else None
    eps = 1e-5
    got = eb.qk_norm_rotary(q, k, wq, wk, cos, sin, at, epsilon=eps, layout=layout)
    c, s = (rows(cos, at), rows(sin, at)) if r else (torch.empty(B, S, 0).double().cuda(),) * 2
    for x, w, y in ((q, wq, got[0]), (k, wk, got[1])):
        x = x.double()
        w = torch.ones(D, device="cuda").double() if w is None else w.double()
        want = ref.norm_rotate(x, w, c, s, layout, eps)
        scale = ref.spread(x * ref.rstd(x, eps) * w, c, s, layout)
        ref.check(y, want, scale, D / 8 + 16, "norm and rotary")


@pytest.mark.parametrize("dtype,wdtype", [(BF16, BF16), (F16, F32), (F32, F32), (BF16, None)])
@pytest.mark.parametrize("shape", SHAPES + MANY, ids=str)
def test_norm_rotary_gradient(shape, dtype, wdtype):
    B, S, Hq, Hk, D, r, layout, how = shape
    g = gen(3)
    q, k = views(g, B, S, Hq, Hk, D, dtype, how)
    dq, dk = views(g, B, S, Hq, Hk, D, dtype, "heads_first" if how == "dense" else how)
    wq = wk = None
    if wdtype is not None:
        wq, wk = ((1 + 0.3 * normal(g, D)).to(wdtype) for _ in range(2))
    cos, sin = tables(S + 3, r) if r else (None, None)
    at = torch.randint(0, S + 3, (B, S), generator=g, device="cuda") if r else None
    eps = 1e-5
    got = eb.qk_norm_rotary_grad(dq, dk, q, k, wq, wk, cos, sin, at, epsilon=eps, layout=layout)
    again = eb.qk_norm_rotary_grad(dq, dk, q, k, wq, wk, cos, sin, at, epsilon=eps, layout=layout)
    c, s = (rows(cos, at), rows(sin, at)) if r else (torch.empty(B, S, 0).double().cuda(),) * 2
    for x, d, w, dx, dw, H in ((q, dq, wq, got[0], got[2], Hq), (k, dk, wk, got[1], got[3], Hk)):
        want, want_w, scale, scale_w = ref.norm_rotate_grad(
            d.double(), x.double(), None if w is None else w.double(), c, s, layout, eps)
        ref.check(dx, want, scale, D / 4 + 32, "dx")
        # a thread adds rows one after another, then threads, warps and CTAs join
        ref.check(dw, want_w, scale_w, D / 8 + 48 + B * S * H, "dw")
    for a, b in zip(got, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("layout,r", [("half", 32), ("interleaved", 20), ("half", 18)])
def test_gradient_against_differences(layout, r):
    """sum(dx v) is the derivative of sum(dy y(x + h v)) at 0: central
    differences of the 64-bit forward form, h = 1e-5, err ~ h^2 and 1e-11 / h."""
    g = gen(4)
    B, S, H, D, eps = 2, 7, 3, 32, 1e-4
    x, dy, v = (normal(g, B, S, H, D) for _ in range(3))
    w, vw = 1 + 0.3 * normal(g, D), normal(g, D)
    cos, sin = tables(S, r)
    at = torch.arange(S, device="cuda").expand(B, S)
    dx, _, dw, _ = eb.qk_norm_rotary_grad(dy, None, x, None, w, None, cos, sin, at, epsilon=eps,
                                          layout=layout)
    c, s = rows(cos, at), rows(sin, at)

    def loss(t, u):
        y = ref.norm_rotate(x.double() + t * v.double(), w.double() + u * vw.double(), c, s,
                            layout, eps)
        return float((dy.double() * y).sum())

    h = 1e-5
    for got, d in ((float((dx.double() * v.double()).sum()), (loss(h, 0) - loss(-h, 0)) / (2 * h)),
                   (float((dw.double() * vw.double()).sum()), (loss(0, h) - loss(0, -h)) / (2 * h))):
        assert abs(got - d) < 2e-5 * math.sqrt(B * S * H * D) * max(1.0, abs(d)) ** 0.5, (got, d)


def test_positions_default_types_and_strides():
    g = gen(5)
    B, S, H, D = 3, 11, 4, 64
    q, k = normal(g, B, S, H, D, dtype=BF16), normal(g, B, S, 2, D, dtype=BF16)
    cos, sin = tables(32, D)
    plain = eb.rotary(q, k, cos, sin)
    index = torch.arange(S, device="cuda")
    for at in (index, index.to(torch.int32), index.expand(B, S),
               torch.stack([index, index + 5], 1).to(torch.int32)[:, 0].expand(B, S),
               index.repeat(B, 1).t().contiguous().t()):
        for a, b in zip(plain, eb.rotary(q, k, cos, sin, at)):
            assert torch.equal(a, b)
    only = eb.rotary(q, None, cos, sin)
    assert only[1] is None and torch.equal(only[0], plain[0])


@pytest.mark.parametrize("S", [6, 20000])
@pytest.mark.parametrize("D,r", [(64, 64), (64, 30)])
def test_positions_outside_the_table(D, r, S):
    """Rows of a token outside the table are zeros, set the status bit and add
    nothing to the weight gradients; the others are untouched."""
    g = gen(6)
    B, H = 2, 3
    q, k = normal(g, B, S, H, D, dtype=BF16), normal(g, B, S, H, D, dtype=BF16)
    cos, sin = tables(16, r)
    at = torch.randint(0, 16, (B, S), generator=g, device="cuda")
    bad = at.clone()
    bad[0, 2], bad[1, 5] = -1, 16
    keep = torch.ones(B, S, dtype=torch.bool, device="cuda")
    keep[0, 2] = keep[1, 5] = False
    want = eb.rotary(q, k, cos, sin, at)
    assert eb.get_device_status() == 0
    got = eb.rotary(q, k, cos, sin, bad)
    assert eb.get_device_status() == eb.DEVICE_POSITION_RANGE
    assert eb.get_device_status() == 0
    for a, b in zip(want, got):
        assert torch.equal(a[keep], b[keep])
        assert (b[~keep] == 0).all()
    w = torch.ones(D, device="cuda", dtype=BF16)
    normed = eb.qk_norm_rotary(q, k, w, w, cos, sin, at)
    got = eb.qk_norm_rotary(q, k, w, w, cos, sin, bad)
    assert eb.get_device_status() == eb.DEVICE_POSITION_RANGE
    for a, b in zip(normed, got):
        assert torch.equal(a[keep], b[keep])
        assert (b[~keep] == 0).all()
    zero = q.clone()
    zero[~keep] = 0
    full = eb.qk_norm_rotary_grad(zero, zero, q, k, w, w, cos, sin, at)
    part = eb.qk_norm_rotary_grad(q, q, q, k, w, w, cos, sin, bad)
    assert eb.get_device_status() == eb.DEVICE_POSITION_RANGE
    for a, b in zip(full, part):
        assert torch.equal(a, b)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,r", [(64, 16), (64, 14), (33, 10)])
def test_infinities_and_nans_stay_in_their_pairs(layout, D, r):
    """An infinity or a NaN in a pair reaches that pair alone, and one past
    rotary_dim passes through, whatever the angle."""
    g = gen(7)
    q = normal(g, 1, 3, 2, D, dtype=BF16)
    cos, sin = tables(3, r)
    clean = eb.rotary(q, None, cos, sin, layout=layout)[0]
    dirty = q.clone()
    dirty[0, 1, 0, D - 1] = math.inf        # past rotary_dim
    dirty[0, 1, 1, D - 2] = math.nan
    dirty[0, 2, 0, 1] = math.inf            # in a pair
    got = eb.rotary(dirty, None, cos, sin, layout=layout)[0]
    pair = (1, 1 + r // 2) if layout == "half" else (0, 1)
    same = torch.ones_like(clean, dtype=torch.bool)
    same[0, 1, 0, D - 1] = same[0, 1, 1, D - 2] = False
    same[0, 2, 0, list(pair)] = False
    assert torch.equal(clean[same], got[same])
    assert got[0, 1, 0, D - 1] == math.inf and got[0, 1, 1, D - 2].isnan()
    assert not got[0, 2, 0, list(pair)].isfinite().any()


@pytest.mark.parametrize("D,r", [(64, 64), (80, 30)])
def test_in_place_and_packed_in_place(D, r):
    g = gen(8)
    B, S, Hq, Hk = 2, 19, 4, 2
    w = 1 + 0.2 * normal(g, D).to(BF16)
    cos, sin = tables(S, r)
    q, k = views(g, B, S, Hq, Hk, D, BF16, "packed")
    want = eb.qk_norm_rotary(q, k, w, w, cos, sin)
    v = q._base.clone()[..., (Hq + Hk) * D:]
    eb.qk_norm_rotary(q, k, w, w, cos, sin, out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(q._base[..., (Hq + Hk) * D:], v)      # the values beside them are untouched
    dq, dk = views(g, B, S, Hq, Hk, D, BF16, "packed")
    want = eb.qk_norm_rotary_grad(dq, dk, q, k, w, w, cos, sin)
    got = eb.qk_norm_rotary_grad(dq, dk, q, k, w, w, cos, sin, out=(dq, dk))
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_empty_shapes():
    cos, sin = tables(4, 8)
    for B, S, Hq, Hk in ((0, 3, 2, 1), (2, 0, 2, 1), (2, 3, 0, 0)):
        q, k = torch.empty(B, S, Hq, 8, device="cuda"), torch.empty(B, S, Hk, 8, device="cuda")
        a, b = eb.rotary(q, k, cos, sin)
        assert a.shape == q.shape and b.shape == k.shape
        _, _, dwq, dwk = eb.qk_norm_rotary_grad(q, k, q, k, None, None, cos, sin)
        assert (dwq == 0).all() and (dwk == 0).all()
    k = torch.randn(2, 3, 2, 8, device="cuda")
    a, b = eb.rotary(torch.empty(2, 3, 0, 8, device="cuda"), k, cos, sin)
    assert torch.equal(b, eb.rotary(k, None, cos, sin)[0])


def test_another_stream_and_a_graph():
    g = gen(9)
    q, k = normal(g, 1, 50, 8, 128, dtype=BF16), normal(g, 1, 50, 2, 128, dtype=BF16)
    cos, sin = tables(64, 128)
    want = eb.rotary(q, k, cos, sin)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = eb.rotary(q, k, cos, sin)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    plan = eb.HeadsPlan(BF16, q.shape, k.shape, table_positions=64)
    out = torch.empty_like(q), torch.empty_like(k)
    with torch.cuda.stream(s):
        eb.execute_heads(plan, q, k, cos, sin, None, out[0], out[1])   # the stream's status word
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        eb.execute_heads(plan, q, k, cos, sin, None, out[0], out[1])
    q.copy_(normal(g, 1, 50, 8, 128))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], eb.rotary(q, k, cos, sin)[0])


def test_offsets_past_32_bits():
    """A head far into a buffer of over 2^32 elements, as a long cache has it."""
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB of device memory")
    step = (1 << 32) + 64
    buf = torch.empty(step + 4096, dtype=BF16, device="cuda")
    q = buf.as_strided((2, 2, 3, 64), (step, 192, 64, 1))
    x = normal(gen(10), 2, 2, 3, 64, dtype=BF16)
    q.copy_(x)
    cos, sin = tables(8, 64)
    want = eb.rotary(x, None, cos, sin)[0]
    eb.rotary(q, None, cos, sin, out=(q, None))
    assert torch.equal(q, want)


@pytest.mark.parametrize("kw", [
    dict(), dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0),
    dict(scaling="by_parts", factor=16.0, trained_length=4096.0, amplitude=1.2),
    dict(base=500000.0, scaling="by_parts", factor=8.0, trained_length=8192.0, fast_turns=4.0)])
@pytest.mark.parametrize("r", [2, 6, 64, 128])
def test_rotary_table(kw, r):
    """Binary64 angles: the error is the binary32 rounding of the result plus
    the binary64 angle's, at most position * 2^-50."""
    if r == 2 and kw.get("scaling") == "base":
        pytest.skip("no base scaling for one frequency")
    for first in (0, 1_000_000):
        cos, sin = eb.rotary_table(300, r, first_position=first, **kw)
        c, s = ref.table(300, r, first=first, **kw)
        for got, want in ((cos, c), (sin, s)):
            off = (got.double().cpu() - want).abs()
            assert float(off.max()) <= 1.2 * 2.0 ** -24 + (first + 300) * 2.0 ** -50
