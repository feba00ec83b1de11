"""Dropout on the GPU against a plain 64-bit form whose mask comes from a numpy Philox.

Bounds: the type's rounding of the true value plus, for each of the formula's steps (the bias,
the scale and its own rounding, the residual: 4), a binary32 rounding of the summed
magnitudes; dbias as many more as rows are added.  What is dropped is exactly the residual."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import block_ref as ref  # noqa: E402
import broadcast_elementwise_gb300 as eb  # noqa: E402
import layer_ref  # noqa: E402

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def normal(seed, *shape, dtype=F32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def matrix(seed, rows, n, dtype, how):
    """Dense, with a row stride on and off the vectors, or starting off them."""
    if how == "strided":
        return normal(seed, rows, n + 24, dtype=dtype)[:, 8:8 + n]
    if how == "odd stride":
        return normal(seed, rows, n + 7, dtype=dtype)[:, :n]
    if how == "off":
        return normal(seed, rows * n + 1, dtype=dtype)[1:].view(rows, n)
    return normal(seed, rows, n, dtype=dtype)


SHAPES = [(1, 1), (1, 3), (1, 4), (1, 8), (3, 5), (7, 32), (2, 256), (5, 257), (33, 1021),
          (64, 4096), (9, 1000), (1, 65536), (4099, 24), (1031, 520), (300, 8)]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("how", ["dense", "strided", "odd stride", "off"])
@pytest.mark.parametrize("rows,n", SHAPES)
def test_dropout(rows, n, how, dtype):
    p, seed, offset = 0.3, 0x123456789ABCDEF0, 2 ** 40 + rows
    x, res = matrix(1, rows, n, dtype, how), matrix(2, rows, n, dtype, how)
    bias = normal(3, n, dtype=dtype)
    m = ref.mask(p, seed, offset, rows, n, "cuda")
    got = eb.dropout(x, p, seed, offset, bias=bias, residual=res)
    kept = m * (x.double() + bias.double())
    want = kept + res.double()
    scale = m * (x.double().abs() + bias.double().abs()) + res.double().abs()
    layer_ref.check(got, want, scale, 4, "dropout")
    assert torch.equal(got[m == 0], res[m == 0])
    plain = eb.dropout(x, p, seed, offset)
    layer_ref.check(plain, m * x.double(), m * x.double().abs(), 2, "dropout alone")
    assert (plain[m == 0] == 0).all()
    dx, db = eb.dropout_grad(x, p, seed, offset, bias=True)
    assert torch.equal(dx, plain)
    layer_ref.check(db, (m * x.double()).sum(0), (m * x.double().abs()).sum(0), rows + 4, "dbias")
    again = eb.dropout_grad(x, p, seed, offset, bias=True)
    assert torch.equal(again[1], db)
    assert torch.equal(eb.dropout_grad(x, p, seed, offset)[0], dx)


def test_bias_types_and_in_place():
    x, res = normal(1, 40, 96, dtype=BF16), normal(2, 40, 96, dtype=BF16)
    b = normal(3, 96)
    m = ref.mask(0.5, 7, 9, 40, 96, "cuda")
    want = eb.dropout(x, 0.5, 7, 9, bias=b, residual=res)
    layer_ref.check(want, m * (x.double() + b.double()) + res.double(),
                    m * (x.double().abs() + b.double().abs()) + res.double().abs(), 4, "float32 bias")
    y = x.clone()
    assert eb.dropout(y, 0.5, 7, 9, bias=b, residual=res, out=y) is y
    assert torch.equal(y, want)
    y = res.clone()
    eb.dropout(x, 0.5, 7, 9, bias=b, residual=y, out=y)
    assert torch.equal(y, want)
    same = eb.dropout(x, 0.5, 7, 9, residual=x)
    layer_ref.check(same, m * x.double() + x.double(), (m + 1) * x.double().abs(), 4, "x twice")
    d = x.clone()
    eb.dropout_grad(d, 0.5, 7, 9, out=d)
    assert torch.equal(d, eb.dropout(x, 0.5, 7, 9))


@pytest.mark.parametrize("p", [0.0, 2.0 ** -33, 2.0 ** -32, 0.1, 0.5, 1 - 2.0 ** -32])
def test_probabilities(p):
    x = normal(1, 16, 264)
    m = ref.mask(p, 3, 0, 16, 264, "cuda")
    got = eb.dropout(x, p, 3)
    layer_ref.check(got, m * x.double(), m * x.double().abs(), 2, "p %g" % p)
    if ref.bound(p) == 0:
        assert torch.equal(got, x)


def test_nothing_of_a_dropped_element_is_left():
    """Infinities and NaN in dropped places add exactly 0, forward and backward."""
    m = ref.mask(0.5, 11, 2, 32, 64, "cuda")
    x, res = normal(1, 32, 64), normal(2, 32, 64)
    bad = x.clone()
    for i, v in enumerate((float("inf"), -float("inf"), float("nan"))):
        bad[(m == 0) & (torch.arange(64, device="cuda") % 3 == i)] = v
    assert torch.equal(eb.dropout(bad, 0.5, 11, 2, residual=res),
                       eb.dropout(x, 0.5, 11, 2, residual=res))
    for a, b in zip(eb.dropout_grad(bad, 0.5, 11, 2, bias=True),
                    eb.dropout_grad(x, 0.5, 11, 2, bias=True)):
        assert torch.equal(a, b)


def test_offsets_on_the_device_and_graphs():
    x = normal(1, 64, 256, dtype=BF16)
    word = torch.tensor([5], device="cuda")
    assert torch.equal(eb.dropout(x, 0.2, 9, 100, offset_device=word), eb.dropout(x, 0.2, 9, 105))
    word.fill_(-1)      # wraps: 2^64 - 1
    assert torch.equal(eb.dropout(x, 0.2, 9, 100, offset_device=word), eb.dropout(x, 0.2, 9, 99))
    assert not torch.equal(eb.dropout(x, 0.2, 9, 100), eb.dropout(x, 0.2, 9, 101))
    assert not torch.equal(eb.dropout(x, 0.2, 9, 100), eb.dropout(x, 0.2, 9 + 2 ** 32, 100))
    y = torch.empty_like(x)
    plan = eb.DropoutPlan(BF16, 64, 256, 0.2)
    grad = eb.DropoutPlan(BF16, 64, 256, 0.2, bias=F32, gradient=True)
    work = torch.empty(grad.workspace_bytes, dtype=torch.uint8, device="cuda")
    dx, db = torch.empty_like(x), torch.empty(256, device="cuda")
    word.fill_(0)

    def step():
        eb.execute_dropout(plan, x, y, 9, 200, offset_device=word)
        eb.execute_dropout_grad(grad, x, dx, 9, 200, dbias=db, workspace=work, offset_device=word)
        word.add_(1)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    word.fill_(0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    word.fill_(0)
    for t in range(3):
        graph.replay()
        want = eb.dropout_grad(x, 0.2, 9, 200 + t, bias=True)
        assert torch.equal(y, eb.dropout(x, 0.2, 9, 200 + t))
        assert torch.equal(dx, want[0]) and torch.equal(db, want[1])


def test_streams_and_empty_shapes():
    x = normal(1, 256, 512, dtype=F16)
    want = eb.dropout(x, 0.4, 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = eb.dropout(x, 0.4, 1, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    for shape in ((0, 8), (8, 0), (0, 0)):
        t = torch.empty(shape, dtype=BF16, device="cuda")
        assert eb.dropout(t, 0.5, 1).shape == t.shape
        dx, db = eb.dropout_grad(t, 0.5, 1, bias=True)
        assert dx.shape == t.shape and (db == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,n", [(40, 96), (300, 257)])
def test_columns_of_one_buffer(rows, n, dtype):
    x, res = normal(1, rows, n, dtype=dtype), normal(2, rows, n, dtype=dtype)
    want = eb.dropout(x, 0.4, 3, 9, residual=res)
    for i in range(3):
        both = torch.cat((x, res, x), 1).split(n, 1)
        assert eb.dropout(both[0], 0.4, 3, 9, residual=both[1], out=both[i]) is both[i]
        for j, v in enumerate((x, res, x)):
            assert torch.equal(both[j], want if j == i else v)
    both = torch.cat((x, res), 1).split(n, 1)
    eb.dropout_grad(both[0], 0.4, 3, 9, out=both[1])
    assert torch.equal(both[0], x) and torch.equal(both[1], eb.dropout(x, 0.4, 3, 9))
