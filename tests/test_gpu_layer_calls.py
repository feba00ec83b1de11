"""The one-call forms of the layer operators on the GPU: refusals that keep broadcast
matrices from the kernels, and calls on another stream than torch's current one."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import broadcast_elementwise_gb300 as eb  # noqa: E402

BF16 = torch.bfloat16


def normal(seed, *shape, dtype=BF16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def test_broadcast_matrices_are_refused():
    a, b, row = normal(1, 8, 32), normal(2, 32, 16), normal(3, 1, 16)
    before = eb.lib.ebin_launch_count()
    for kw in (dict(residual=row.expand(8, 16)), dict(out=row.expand(8, 16)),
               dict(preact=row.expand(8, 16))):
        with pytest.raises(ValueError):
            eb.gemm(a, b, **kw)
    with pytest.raises(ValueError):
        eb.gemm(normal(4, 1, 32).expand(8, 32), b)
    y = normal(5, 8, 1).requires_grad_()
    dy, = torch.autograd.grad(y.sum(), y)        # a scalar, expanded
    if dy.stride() == (0, 0):
        with pytest.raises(ValueError):
            eb.gemm_epilogue_grad(dy)
    assert eb.lib.ebin_launch_count() == before
    # its copy is taken, and adds the row to every row
    got = eb.gemm(a, b, None, row.expand(8, 16).contiguous())
    assert torch.equal(got, eb.gemm(a, b, residual=row.repeat(8, 1)))


def calls():
    """(name, call) of every one-call form whose kernels use memory that the call allocates."""
    a, b = normal(1, 300, 261), normal(2, 261, 521)       # odd rows: both are laid out anew
    dy, z = normal(3, 4000, 264), normal(4, 4000, 264)
    q, k = normal(5, 2, 700, 6, 64), normal(6, 2, 700, 2, 64)
    dq, dk = normal(7, 2, 700, 6, 64), normal(8, 2, 700, 2, 64)
    cos, sin = eb.rotary_table(700, 64)
    x = normal(9, 8, 48, 1000, dtype=torch.float32)
    block = normal(10, 48, 4, dtype=torch.float32).abs().t()     # copied: not contiguous
    return [("gemm", lambda s: [eb.gemm(a, b, stream=s)]),
            ("gemm_epilogue_grad",
             lambda s: list(eb.gemm_epilogue_grad(dy, z, activation="silu", stream=s))),
            ("qk_norm_rotary", lambda s: list(eb.qk_norm_rotary(q, k, None, None, cos, sin,
                                                               stream=s))),
            ("qk_norm_rotary_grad",
             lambda s: list(eb.qk_norm_rotary_grad(dq, dk, q, k, None, None, cos, sin, stream=s))),
            ("rotary_table", lambda s: list(eb.rotary_table(900, 64, stream=s))),
            ("binary", lambda s: [eb.binary("BatchNormalization", x, block, epsilon=1e-5,
                                            stream=s)])]


@pytest.mark.parametrize("how", ["stream", "address"])
def test_another_stream_beside_a_busy_current_one(how):
    """The call's stream is held back while the current stream takes and fills blocks of
    every size that the call used, and the other way round; results are unchanged."""
    s = torch.cuda.Stream()
    for name, call in calls():
        want = call(None)
        torch.cuda.synchronize()
        for held in (s, torch.cuda.current_stream()):
            with torch.cuda.stream(held):
                torch.cuda._sleep(20_000_000)
                dropped = [torch.full((1 << n,), 255, dtype=torch.uint8, device="cuda")
                           for n in range(9, 23)] if held is not s else None
            del dropped
            got = call(s if how == "stream" else s.cuda_stream)
            blocks = [torch.full((1 << n,), 255, dtype=torch.uint8, device="cuda")
                      for n in range(9, 23) for _ in range(4)]
            torch.cuda.synchronize()
            for x, y in zip(got, want):
                assert torch.equal(x, y), name
            del blocks, got
    assert eb.get_device_status(s) == 0


@pytest.mark.parametrize("dtype", [BF16, torch.float16, torch.float32])
@pytest.mark.parametrize("tokens", [3, 9000])
@pytest.mark.parametrize("D,r,layout", [(64, 64, "half"), (64, 32, "interleaved"), (64, 14, "half"),
                                        (33, 10, "half")])
def test_a_table_without_rows(D, r, layout, tokens, dtype):
    """Every position is outside it: rows of zeros, the status bit, no weight gradients, and
    no table is read (addresses of one element stand in for the tables, or none)."""
    q, k = normal(1, 2, tokens, 3, D, dtype=dtype), normal(2, 2, tokens, 1, D, dtype=dtype)
    one = torch.full((1,), float("nan"), device="cuda")
    for tables in ((one, one), (None, None)):
        for kw in (dict(), dict(gradient=True), dict(norm="rms")):
            plan = eb.HeadsPlan(dtype, q.shape, k.shape, rotary_dim=r, layout=layout,
                                table_positions=0, **kw)
            qo, ko = torch.full_like(q, 7), torch.full_like(k, 7)
            eb.execute_heads(plan, q, k, *tables, None, qo, ko)
            assert eb.get_device_status() == eb.DEVICE_POSITION_RANGE
            assert (qo == 0).all() and (ko == 0).all()
        plan = eb.HeadsPlan(dtype, q.shape, k.shape, rotary_dim=r, layout=layout, norm="rms",
                            gradient=True, table_positions=0)
        work = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        dw = torch.full((2, D), 7.0, device="cuda")
        qo, ko = torch.full_like(q, 7), torch.full_like(k, 7)
        eb.execute_heads_grad(plan, q, k, q, k, *tables, None, None, None, qo, ko, dw[0], dw[1],
                              work)
        assert eb.get_device_status() == eb.DEVICE_POSITION_RANGE
        assert (qo == 0).all() and (ko == 0).all() and (dw == 0).all()
    none = torch.empty(0, r // 2, device="cuda")
    got = eb.rotary(q, k, none, none, layout=layout)
    assert eb.get_device_status() == eb.DEVICE_POSITION_RANGE
    assert (got[0] == 0).all() and (got[1] == 0).all()


def packed(order, batch, tokens, q_heads, k_heads, dim):
    """(buffer, q, k) of one projection, its buffer laid out in the given order."""
    h = q_heads + 2 * k_heads
    if order == "heads, tokens":
        x = normal(11, batch, h, tokens, dim)
        v = x.transpose(1, 2)
    elif order == "tokens, heads":
        v = x = normal(11, batch, tokens, h, dim)
    elif order == "tokens, q k v of each head":
        x = normal(11, batch, tokens, q_heads, 3, dim)
        return x, x[:, :, :, 0], x[:, :, :k_heads, 1]
    else:
        x = normal(11, batch, 3, q_heads, tokens, dim)
        v = x.transpose(2, 3)
        return x, v[:, 0], v[:, 1, :, :k_heads]
    return x, v[:, :, :q_heads], v[:, :, q_heads:q_heads + k_heads]


@pytest.mark.parametrize("order", ["tokens, heads", "heads, tokens", "tokens, q k v of each head",
                                   "q k v, heads, tokens"])
@pytest.mark.parametrize("tokens,D,r", [(1, 64, 64), (37, 64, 64), (37, 80, 30), (9000, 64, 32),
                                        (21, 33, 22)])
def test_packed_buffers_in_place(order, tokens, D, r):
    """q and k in place in a projection's buffer, however it is laid out: what the call out of
    place gives, and nothing else of the buffer is touched."""
    x, q, k = packed(order, 2, tokens, 4, 2, D)
    cos, sin = eb.rotary_table(tokens, r)
    w = normal(12, D)
    before, rest = x.clone(), torch.ones_like(x, dtype=torch.bool)
    for t in (q, k):
        rest.as_strided(t.shape, t.stride(), t.storage_offset()).fill_(False)
    want = eb.rotary(q, k, cos, sin)
    eb.rotary(q, k, cos, sin, out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    want = eb.qk_norm_rotary(q, k, w, w, cos, sin)
    eb.qk_norm_rotary(q, k, w, w, cos, sin, out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    _, fq, fk = packed(order, 2, tokens, 4, 2, D)
    want = eb.qk_norm_rotary_grad(q, k, fq, fk, w, w, cos, sin)
    got = eb.qk_norm_rotary_grad(q, k, fq, fk, w, w, cos, sin, out=(q, k))
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert torch.equal(x[rest], before[rest])
    assert eb.get_device_status() == 0
