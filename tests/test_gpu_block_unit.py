"""The norms around a block on so many rows that a CTA takes a unit of them, its teams walking the
rows in turn with others on their way to shared memory: on the vectors and off them, a team of
one warp and of several, against the 64-bit form with test_gpu_block_norm's bounds.

Forward a unit holds two rows for each of its teams, and all rows are more than two a CTA: so
5000 rows of 1536 columns (teams of two warps), 2500 of 4096 (four), 1300 of 8192 (eight)."""
import functools

import pytest
import torch

pytestmark = pytest.mark.gpu

import block_ref as ref  # noqa: E402
import broadcast_elementwise_gb300 as eb  # noqa: E402
from test_gpu_block_norm import (BF16, F16, F32, OFFSET, SEED, TYPES, check_forward,  # noqa: E402
                                 check_gradient, keep_of, matrix, operands, valid)


@pytest.fixture(autouse=True)
def masks_once(monkeypatch):
    """A mask of millions of elements takes a second on the host."""
    monkeypatch.setattr(ref, "mask", _mask)


_mask = functools.lru_cache(maxsize=16)(ref.mask)

SHAPES = [(5000, 0, 72), (9000, 3, 264), (5001, 3, 520), (5000, 5, 1536), (3000, 2, 2048),
          (2500, 0, 4096), (1000, 0, 5120), (1300, 2, 8192)]
NORMS = [("none", "rms"), ("none", "layer"), ("rms", "rms"), ("layer", "layer")]


@pytest.mark.parametrize("rows,groups,n", SHAPES)
@pytest.mark.parametrize("dtype,stream", TYPES)
@pytest.mark.parametrize("post,pre", NORMS)
def test_on_vectors(post, pre, dtype, stream, rows, groups, n):
    t, p = operands(rows, n, dtype, stream, groups, weights=dtype, mods=dtype)
    p = valid(p, post, pre)
    check_forward(t, p, post, pre, 0.25, 0.9, 0.5)
    check_gradient(t, p, post, pre, 0.25, 0.9, 0.5)


@pytest.mark.parametrize("given", [(), ("w_pre",), ("w_post", "gate"), ("b_post", "scale"),
                                   ("b_pre",), ("shift", "gate")])
@pytest.mark.parametrize("drop", [0.0, 0.25])
def test_parameters_left_out(given, drop):
    t, p = operands(5000, 1536, BF16, F32, 5)
    p = {k: v for k, v in p.items() if k in given}
    check_forward(t, p, "rms", "layer", drop)
    check_gradient(t, p, "rms", "rms", drop)
    check_gradient(t, p, "rms", "layer", drop, dh=False)


@pytest.mark.parametrize("given", [("w_pre", "w_post"), ("w_pre", "b_pre", "w_post"),
                                   ("w_pre", "w_post", "b_post"), ("scale", "shift")])
@pytest.mark.parametrize("rows,groups,n", [(2500, 0, 4096), (9000, 3, 264), (2500, 0, 4097),
                                           (3000, 0, 1023), (1300, 2, 8192)])
def test_rms_norms_by_the_sums_that_are_wanted(rows, groups, n, given):
    """A bias's or a shift's gradient takes another kernel, on units of another count."""
    t, p = operands(rows, n, BF16, BF16, groups)
    p = {k: v for k, v in p.items() if k in given}
    check_gradient(t, p, "rms", "rms", 0.25)
    check_gradient(t, p, "rms", "rms")


@pytest.mark.parametrize("dtype,stream", TYPES)
@pytest.mark.parametrize("rows,n", [(5000, 1536), (2500, 4096)])
def test_strided_rows_and_no_branch(rows, n, dtype, stream):
    t, p = operands(rows, n, dtype, stream, 0, "strided")
    check_forward(t, p, "rms", "layer", 0.25)
    check_gradient(t, p, "rms", "layer", 0.25)
    del t["y"]
    t["dtype"] = dtype
    p = valid(p, "none", "layer", branch=False)
    check_forward(t, p, "none", "layer", a=1.5, dtype=dtype)
    check_gradient(t, p, "none", "layer", a=1.5)


@pytest.mark.parametrize("post,pre", [("rms", "rms"), ("layer", "rms"), ("none", "layer")])
@pytest.mark.parametrize("dtype,stream", [(BF16, BF16), (F32, F32), (F16, F32)])
@pytest.mark.parametrize("rows,n", [(9000, 264), (5000, 1024), (2500, 4096), (2000, 8184),
                                    (5000, 523), (2500, 4097)])
def test_in_place(rows, n, dtype, stream, post, pre):
    """An output in an input's place, while the rows behind it are on their way from there."""
    t, p = operands(rows, n, dtype, stream, 0)
    p = valid(p, post, pre)
    kw = dict(post=post, pre=pre, dropout=0.1, seed=SEED, offset=OFFSET, **p)
    same = dtype == stream
    want = eb.block_norm(t["x"], t["y"], **kw)
    for ho, zo in (("x", "y"),) + ((("y", "x"),) if same else ()):
        c = {k: v.clone() for k, v in t.items()}
        for a, b in zip(eb.block_norm(c["x"], c["y"], out=(c[ho], c[zo]), **kw), want):
            assert torch.equal(a, b)
    dz, dh = matrix(21, rows, n, dtype), matrix(22, rows, n, stream)
    want = eb.block_norm_grad(dz, dh, t["x"], t["y"], **kw)
    for names in (("dh", "y"), ("h", "dz")) + ((("dz", "dh"), ("y", "h")) if same else ()):
        c = {"dz": dz.clone(), "dh": dh.clone(), "h": t["x"].clone(), "y": t["y"].clone()}
        got = eb.block_norm_grad(c["dz"], c["dh"], c["h"], c["y"],
                                 out=(c[names[0]], c[names[1]]), **kw)
        for k in want:
            assert torch.equal(got[k], want[k]), (names, k)


def surrounded(x, fill, off, gap):
    """A copy of x [rows, n] whose rows lie `gap` elements apart and begin `off` into a buffer that
    holds `fill` everywhere else; the buffer too."""
    rows, n = x.shape
    whole = torch.full((off + rows * (n + gap) + 29,), fill, dtype=x.dtype, device="cuda")
    view = whole[off:off + rows * (n + gap)].view(rows, n + gap)[:, :n]
    view.copy_(x)
    return view, whole


@pytest.mark.parametrize("post,pre", [("rms", "rms"), ("layer", "layer"), ("none", "layer")])
@pytest.mark.parametrize("dtype,stream", TYPES)
@pytest.mark.parametrize("rows,n,off,gap", [(5000, 1536, 32, 16), (2500, 4096, 8, 8),
                                            (5000, 523, 33, 0), (5000, 3, 7, 0),
                                            (2500, 4097, 5, 0), (2600, 2051, 3, 1),
                                            (400, 4097, 1, 0)])
def test_what_lies_around_the_rows(rows, n, off, gap, dtype, stream, post, pre):
    """Infinities around the inputs change nothing, and what lies around the outputs stays."""
    t, p = operands(rows, n, dtype, stream, 0)
    p = valid(p, post, pre)
    kw = dict(post=post, pre=pre, dropout=0.25, seed=SEED, offset=OFFSET, **p)
    dz, dh = matrix(21, rows, n, dtype), matrix(22, rows, n, stream)
    h, z = eb.block_norm(t["x"], t["y"], **kw)
    want = eb.block_norm_grad(dz, dh, t["x"], t["y"], **kw)
    inf = float("inf")
    x, y, dz, dh = (surrounded(v, inf, off, gap)[0] for v in (t["x"], t["y"], dz, dh))
    off += n % 8 != 0       # off the vectors, each in a way of its own
    outs = [surrounded(torch.zeros_like(v), 7.0, off, gap) for v in (h, z, want["x"], want["y"])]
    eb.block_norm(x, y, out=(outs[0][0], outs[1][0]), **kw)
    got = eb.block_norm_grad(dz, dh, x, y, out=(outs[2][0], outs[3][0]), **kw)
    for (view, whole), v in zip(outs, (h, z, want["x"], want["y"])):
        assert torch.equal(view, v)
        view.fill_(7)
        assert (whole == 7).all()
    for k in p:
        assert torch.equal(got[k], want[k]), k


@pytest.mark.parametrize("dtype,stream", [(BF16, BF16), (F16, F32), (F32, F32)])
@pytest.mark.parametrize("rows,n", [(5000, 1536), (2500, 4096), (1300, 8192), (2500, 4097),
                                    (5000, 523)])
def test_bad_rows_stay_alone(rows, n, dtype, stream):
    """NaN and infinities of some rows reach no other row, and what is dropped of a branch
    without a norm adds exactly 0."""
    t, p = operands(rows, n, dtype, stream, 0)
    dz, dh = matrix(21, rows, n, dtype), matrix(22, rows, n, stream)
    kw = dict(post="layer", pre="rms", **p)
    good = eb.block_norm(t["x"], t["y"], **kw)
    back = eb.block_norm_grad(dz, dh, t["x"], t["y"], **kw)
    bad = list(range(3, rows, 97))
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    rest[bad] = False
    x, y = t["x"].clone(), t["y"].clone()
    for i, r in enumerate(bad):
        (x, y)[i % 2][r, (37 * i) % n] = (float("nan"), float("inf"))[i // 2 % 2]
    for a, b in zip(good, eb.block_norm(x, y, **kw)):
        assert torch.equal(a[rest], b[rest]) and not b[~rest].isfinite().all()
    got = eb.block_norm_grad(dz, dh, x, y, **kw)
    for k in ("x", "y"):
        assert torch.equal(got[k][rest], back[k][rest])
    gone = keep_of(0.5, rows, n) == 0
    broken = torch.where(gone, torch.full_like(t["y"], float("inf")), t["y"])
    kw = dict(pre="rms", dropout=0.5, seed=SEED, offset=OFFSET, **valid(p, "none", "rms"))
    for a, b in zip(eb.block_norm(t["x"], t["y"], **kw), eb.block_norm(t["x"], broken, **kw)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("rows", [7, 400, 5000])
@pytest.mark.parametrize("n", [264, 523, 9001])
def test_columns_of_one_buffer(rows, n):
    """Inputs and outputs side by side in one buffer, each in place or beside the others."""
    rows = min(rows, 4000000 // n)
    t, p = operands(rows, n, BF16, BF16, 0)
    kw = dict(post="rms", pre="layer", dropout=0.1, seed=SEED, offset=OFFSET, **p)
    dz, dh = matrix(21, rows, n, BF16), matrix(22, rows, n, BF16)
    want = eb.block_norm(t["x"], t["y"], **kw)
    back = eb.block_norm_grad(dz, dh, t["x"], t["y"], **kw)
    for names in ((0, 1), (1, 0), (2, 3), (3, 0)):
        x, y, *_ = both = torch.cat((t["x"], t["y"], dz, dh), 1).split(n, 1)
        h, z = (both[i] for i in names)
        eb.block_norm(x, y, out=(h, z), **kw)
        assert torch.equal(h, want[0]) and torch.equal(z, want[1])
        for i in set(range(4)) - set(names):
            assert torch.equal(both[i], (t["x"], t["y"], dz, dh)[i])
        h, y, dz_, dh_ = both = torch.cat((t["x"], t["y"], dz, dh), 1).split(n, 1)
        got = eb.block_norm_grad(dz_, dh_, h, y, out=[both[i] for i in names], **kw)
        for k, v in back.items():
            assert torch.equal(got[k], v), k
        for i in set(range(4)) - set(names):
            assert torch.equal(both[i], (t["x"], t["y"], dz, dh)[i])
