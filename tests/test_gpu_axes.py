"""Rotary positions with several axes on the GPU: against the 64-bit form of one axis on tables
gathered for each token, with its bounds; in the half layout bit for bit against the engine's
own one-axis form on those tables.  (Interleaved, the two take a head's vectors in other units,
and a unit that rotates in part sums fma(b, -s, fl(a c)) where a whole one sums fma(a, c,
fl(-b s)): one rounded product and one fused sum each, so within the same bound, but not the
same bits.)"""
import pytest
import torch

pytestmark = pytest.mark.gpu

import broadcast_elementwise_gb300 as eb  # noqa: E402
import layer_ref as ref  # noqa: E402

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def normal(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def axis_of_pair(sections, order):
    if order == "blocks":
        return [a for a, s in enumerate(sections) for _ in range(s)]
    left, out = list(sections), []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def gathered(table, positions, sections, order):
    """[B, S, pairs]: each pair's entry at its axis' position."""
    index = torch.tensor(axis_of_pair(sections, order), device="cuda")
    at = positions.long()[index].permute(1, 2, 0)
    return table[at, torch.arange(len(index), device="cuda")]


CASES = [
    # B, S, Hq, Hk, D, layout, sections, order, where the buffers start
    (1, 1, 32, 8, 128, "half", (16, 24, 24), "blocks", 0),
    (2, 1, 4, 2, 128, "half", (24, 20, 20), "dealt", 0),
    (2, 37, 4, 2, 64, "interleaved", (8, 12, 12), "blocks", 0),
    (2, 37, 4, 2, 64, "interleaved", (10, 11, 11), "blocks", 0),
    (3, 5, 6, 3, 80, "half", (20, 20), "blocks", 0),
    (3, 5, 6, 3, 80, "half", (19, 21), "dealt", 0),
    (3, 5, 7, 1, 96, "half", (7, 8, 8), "blocks", 0),        # half of no whole vector
    (3, 5, 7, 1, 96, "interleaved", (3, 5, 7, 8), "dealt", 0),
    (1, 9, 2, 0, 32, "half", (16,), "blocks", 0),
    (1, 9, 2, 1, 32, "half", (0, 9, 0, 7), "dealt", 0),
    (2, 17, 3, 3, 64, "half", (11, 10, 11), "blocks", 1),
    (2, 17, 3, 3, 64, "interleaved", (11, 10, 11), "dealt", 1),
    (2, 3, 2, 1, 33, "half", (5, 6), "blocks", 0),
    (2, 3, 2, 1, 1024, "half", (100, 212, 100, 100), "dealt", 0),
    (1, 2, 1, 1, 2, "half", (1,), "blocks", 0),
    (2, 4099, 32, 8, 128, "interleaved", (22, 21, 21), "blocks", 0),
    (2, 4099, 20, 5, 96, "half", (12, 12, 24), "dealt", 0),
    (1, 6001, 9, 3, 72, "half", (18, 18), "blocks", 0),
]


def inputs(case, dtype, seed):
    B, S, Hq, Hk, D, layout, sections, order, off = case
    g = gen(seed)

    def heads(H):
        return normal(g, B * S * H * D + off, dtype=dtype)[off:].view(B, S, H, D) if H else None

    length = 53
    c, s = ref.table(length, 2 * sum(sections))
    at = torch.randint(0, length, (len(sections), B, S), generator=g, device="cuda",
                       dtype=torch.int32)
    return g, heads, c.float().cuda(), s.float().cuda(), at


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("gradient", [False, True])
def test_rotary(case, dtype, gradient):
    B, S, Hq, Hk, D, layout, sections, order, off = case
    g, heads, cos, sin, at = inputs(case, dtype, 1)
    q, k = heads(Hq), heads(Hk)
    kw = dict(layout=layout, gradient=gradient)
    got = eb.rotary(q, k, cos, sin, at, axes=sections, axes_order=order, **kw)
    c, s = (gathered(t, at, sections, order) for t in (cos, sin))
    one = eb.rotary(q, k, c.reshape(B * S, -1).contiguous(), s.reshape(B * S, -1).contiguous(),
                    torch.arange(B * S, device="cuda").view(B, S), **kw)
    for x, y, z in ((q, got[0], one[0]), (k, got[1], one[1])):
        if x is None:
            assert y is None
            continue
        want = ref.rotate(x.double(), c.double(), s.double(), layout, -1.0 if gradient else 1.0)
        ref.check(y, want, ref.spread(x.double(), c.double(), s.double(), layout), 4, "rotary")
        assert layout != "half" or torch.equal(y, z)
    assert eb.get_device_status() == 0


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_norm_and_its_gradient(case, dtype):
    B, S, Hq, Hk, D, layout, sections, order, off = case
    g, heads, cos, sin, at = inputs(case, dtype, 2)
    q, k, dq, dk = heads(Hq), heads(Hk), heads(Hq), heads(Hk)
    wq, wk = ((1 + 0.3 * normal(g, D)).to(dtype) for _ in range(2))
    eps = 1e-5
    kw = dict(epsilon=eps, layout=layout, axes=sections, axes_order=order)
    got = eb.qk_norm_rotary(q, k, wq, wk, cos, sin, at, **kw)
    back = eb.qk_norm_rotary_grad(dq, dk, q, k, wq, wk, cos, sin, at, **kw)
    c, s = (gathered(t, at, sections, order).double() for t in (cos, sin))
    for i, (x, d, w, H) in enumerate(((q, dq, wq, Hq), (k, dk, wk, Hk))):
        if x is None:
            continue
        want = ref.norm_rotate(x.double(), w.double(), c, s, layout, eps)
        scale = ref.spread(x.double() * ref.rstd(x.double(), eps) * w.double(), c, s, layout)
        ref.check(got[i], want, scale, D / 8 + 16, "norm and rotary")
        want, want_w, scale, scale_w = ref.norm_rotate_grad(d.double(), x.double(), w.double(), c,
                                                            s, layout, eps)
        ref.check(back[i], want, scale, D / 4 + 32, "dx")
        ref.check(back[2 + i], want_w, scale_w, D / 8 + 48 + B * S * H, "dw")
    assert eb.get_device_status() == 0


def test_positions_of_every_type_and_stride():
    g = gen(3)
    q, k = normal(g, 3, 11, 4, 64, dtype=BF16), normal(g, 3, 11, 2, 64, dtype=BF16)
    c, s = (t.float().cuda() for t in ref.table(40, 64))
    at = torch.randint(0, 40, (3, 3, 11), generator=g, device="cuda", dtype=torch.int32)
    kw = dict(axes=(16, 8, 8))
    want = eb.rotary(q, k, c, s, at, **kw)
    for p in (at.long(), at.permute(1, 2, 0).contiguous().permute(2, 0, 1),
              torch.stack((at, at), -1)[..., 1]):
        for a, b in zip(eb.rotary(q, k, c, s, p, **kw), want):
            assert torch.equal(a, b)
    shared = at[:, 0]      # one row of positions for the batch
    for a, b in zip(eb.rotary(q, k, c, s, shared, **kw),
                    eb.rotary(q, k, c, s, shared[:, None].expand(3, 3, 11).contiguous(), **kw)):
        assert torch.equal(a, b)
    # the same position on each axis is the one-axis form
    for a, b in zip(eb.rotary(q, k, c, s, at[:1].expand(3, 3, 11), **kw),
                    eb.rotary(q, k, c, s, at[0])):
        assert torch.equal(a, b)


@pytest.mark.parametrize("S", [3, 3000])
@pytest.mark.parametrize("D", [64, 33])
def test_positions_outside_the_table(S, D):
    g = gen(4)
    r, sections = D // 4 * 2, (D // 4 - 5, 5, 0)
    q, k = normal(g, 2, S, 12, D, dtype=BF16), normal(g, 2, S, 3, D, dtype=BF16)
    w = normal(g, D, dtype=BF16)
    c, s = (t.float().cuda() for t in ref.table(16, r))
    at = torch.randint(0, 16, (3, 2, S), generator=g, device="cuda")
    good = eb.rotary(q, k, c, s, at, axes=sections)
    at[2] = 1 << 40        # an axis without pairs is not read
    for a, b in zip(eb.rotary(q, k, c, s, at, axes=sections), good):
        assert torch.equal(a, b)
    assert eb.get_device_status() == 0
    grads = eb.qk_norm_rotary_grad(q, k, q, k, w, w, c, s, at, axes=sections)
    bad = torch.zeros(2, S, dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[1, S - 1] = True
    at[0, 0, 1], at[1, 1, S - 1] = -1, 16
    got = eb.rotary(q, k, c, s, at, axes=sections)
    assert eb.get_device_status() == eb.DEVICE_POSITION_RANGE
    for a, b in zip(got, good):
        assert (a[bad] == 0).all() and torch.equal(a[~bad], b[~bad])
    normed = eb.qk_norm_rotary(q, k, w, w, c, s, at, axes=sections)
    assert eb.get_device_status() == eb.DEVICE_POSITION_RANGE
    assert (normed[0][bad] == 0).all() and (normed[1][bad] == 0).all()
    back = eb.qk_norm_rotary_grad(q, k, q, k, w, w, c, s, at, axes=sections)
    assert eb.get_device_status() == eb.DEVICE_POSITION_RANGE
    for a, b in zip(back[:2], grads[:2]):
        assert (a[bad] == 0).all() and torch.equal(a[~bad], b[~bad])


@pytest.mark.parametrize("sections,order", [((8, 12, 12), "blocks"), ((24, 20, 20), "dealt"),
                                            ((3, 0, 2), "dealt"), ((1,), "blocks")])
def test_tables_of_own_frequencies(sections, order):
    r = 2 * sum(sections)
    cos, sin = eb.rotary_table(50, r, base=500.0, axes=sections, axes_order=order, amplitude=1.5,
                               first_position=7)
    place = [0] * len(sections)
    f = []
    for a in axis_of_pair(sections, order):
        f.append(500.0 ** (-place[a] / sections[a]))
        place[a] += 1
    angle = torch.arange(7, 57, dtype=torch.float64)[:, None] * torch.tensor(f, dtype=torch.float64)
    # one rounding to float32, and the binary64 angle's own error
    assert (cos.double().cpu() - 1.5 * angle.cos()).abs().max() < 1.5 * 2 ** -24 + 1e-12
    assert (sin.double().cpu() - 1.5 * angle.sin()).abs().max() < 1.5 * 2 ** -24 + 1e-12


def test_captured_and_in_place():
    g = gen(5)
    q, k = normal(g, 2, 40, 4, 64, dtype=BF16), normal(g, 2, 40, 2, 64, dtype=BF16)
    c, s = (t.float().cuda() for t in ref.table(64, 64))
    at = torch.randint(0, 64, (2, 2, 40), generator=g, device="cuda", dtype=torch.int32)
    want = eb.rotary(q, k, c, s, at, axes=(16, 16))
    qi, ki = q.clone(), k.clone()
    eb.rotary(qi, ki, c, s, at, axes=(16, 16), out=(qi, ki))
    assert torch.equal(qi, want[0]) and torch.equal(ki, want[1])
    plan = eb.HeadsPlan(BF16, q.shape, k.shape, positions=torch.int32, table_positions=64,
                        axes=(16, 16))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        eb.execute_heads(plan, q, k, c, s, at, qi, ki)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        eb.execute_heads(plan, q, k, c, s, at, qi, ki)
    at.copy_((at + 5) % 64)
    graph.replay()
    want = eb.rotary(q, k, c, s, at, axes=(16, 16))
    assert torch.equal(qi, want[0]) and torch.equal(ki, want[1])


WIDER = [
    # interleaved heads of 5, 9, 32 and 64 vectors of 16-bit elements, parts of them turned
    (2, 9, 5, 2, 40, "interleaved", (6, 7, 7), "dealt", 0),
    (2, 9, 5, 2, 72, "interleaved", (12, 12, 12), "blocks", 0),
    (2, 9, 5, 2, 72, "interleaved", (9, 4), "blocks", 0),
    (2, 9, 5, 2, 256, "interleaved", (40, 44, 44), "dealt", 0),
    (2, 9, 5, 2, 512, "interleaved", (64, 96, 96), "blocks", 0),
    (2, 9, 5, 2, 512, "interleaved", (33, 0, 0, 100), "dealt", 0),
    (1, 2049, 9, 5, 512, "interleaved", (64, 96, 96), "blocks", 0),
    (1, 4100, 3, 17, 8, "interleaved", (1, 2, 1), "blocks", 0),
    (1, 3000, 13, 1, 40, "half", (8, 6, 6), "dealt", 0),
]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("case", WIDER, ids=str)
def test_heads_of_other_widths(case, dtype):
    for gradient in (False, True):
        test_rotary(case, dtype, gradient)
    test_norm_and_its_gradient(case, dtype)
