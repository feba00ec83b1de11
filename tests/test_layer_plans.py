"""Refusals of the layer operators' plans and executions (heads, matrix
products, epilogue gradients).  CPU: the checks run before any device call,
and the addresses given are never dereferenced."""
import pytest

import broadcast_elementwise_gb300 as eb


def code(fn, *a, **kw):
    with pytest.raises(eb.EbinError) as e:
        fn(*a, **kw)
    return e.value.code


def heads(dtype="bfloat16", q=(2, 4, 5, 64), k=(2, 4, 1, 64), **kw):
    kw.setdefault("table_positions", 16)
    return eb.HeadsPlan(dtype, q, k, **kw)


def test_heads_plan_refusals():
    for dtype in ("int32", "float64", "bool", "uint8"):
        assert code(heads, dtype) == "unsupported_type"
    assert code(heads, norm="rms", weight_dtype="float16") == "unsupported_type"
    for r in (-2, 3, 66):
        assert code(heads, rotary_dim=r) == "invalid_attr"
    assert code(heads, positions="float32") == "invalid_attr"
    for eps in (-1.0, float("nan"), float("inf")):
        assert code(heads, norm="rms", epsilon=eps) == "invalid_attr"
    for shape in ((-1, 4, 5, 64), (2, -4, 5, 64), (2, 4, 5, 0), (2, 4, 5, 1025),
                  (1 << 40, 1 << 20, 5, 64)):
        assert code(heads, q=shape, k=shape[:2] + (1,) + shape[3:], rotary_dim=0) == "invalid_arg"
    assert code(heads, table_positions=-1) == "invalid_arg"
    assert code(heads, q_strides=(-1, 320, 64, 1)) == "invalid_arg"
    assert code(heads, q_strides=(1 << 60, 320, 64, 1)) == "invalid_arg"
    assert code(heads, positions="int32", position_strides=(-1, 1)) == "invalid_arg"
    # an output that overlaps itself; an input may be broadcast
    assert code(heads, q_out_strides=(0, 320, 64, 1)) == "invalid_arg"
    assert code(heads, q_out_strides=(1280, 320, 32, 1)) == "invalid_arg"
    heads(q_strides=(0, 320, 64, 1))
    with pytest.raises(ValueError):
        heads(q_strides=(1280, 320, 64, 2))
    with pytest.raises(ValueError):
        heads(k=(2, 5, 1, 64))


def run(plan, q=0x100000, k=0x200000, cos=0x300000, sin=0x400000, pos=None, qo=0x500000,
        ko=0x600000, wq=None, wk=None):
    eb.execute_heads(plan, q, k, cos, sin, pos, qo, ko, wq, wk, stream=0)


def test_heads_execute_refusals():
    p = heads()
    for missing in ("q", "k", "cos", "sin", "qo", "ko"):
        assert code(run, p, **{missing: None}) == "invalid_arg"
    assert code(run, heads(positions="int32")) == "invalid_arg"
    for off in (dict(q=0x100001), dict(ko=0x600001), dict(cos=0x300002), dict(sin=0x400001)):
        assert code(run, p, **off) == "invalid_arg"                  # off the element size
    assert code(run, heads(positions="int64"), pos=0x700004) == "invalid_arg"
    assert code(run, heads(norm="rms"), wq=0x700001) == "invalid_arg"
    assert code(run, heads(norm="rms", weight_dtype="float32"), wk=0x700002) == "invalid_arg"
    assert code(run, heads(norm="rms", gradient=True)) == "invalid_arg"
    # q is 2560 elements, 5120 bytes
    assert code(run, p, qo=0x100002) == "alias"
    assert code(run, p, qo=0x200000) == "alias"                      # over k
    assert code(run, p, qo=0x300000) == "alias"                      # over the table
    assert code(run, p, ko=0x500000) == "alias"                      # over the other output
    assert code(run, heads(positions="int64"), pos=0x500010) == "alias"
    assert code(run, heads(norm="rms"), wq=0x500010) == "alias"
    # in place with other strides
    other = heads(q_out_strides=(2048, 512, 64, 1))
    assert code(run, other, qo=0x100000) == "alias"
    # views of one buffer that do share elements (k starts inside q's heads)
    packed = heads(**{n + "_strides": (4 * 448, 448, 64, 1) for n in ("q", "k", "q_out", "k_out")})
    assert code(run, packed, k=0x100000 + 2 * 128, qo=0x100000,
                ko=0x100000 + 2 * 128) == "alias"


def test_heads_grad_refusals():
    p = heads(norm="rms", gradient=True)
    assert p.workspace_bytes > 0

    def grad(**kw):
        a = dict(dq=0x100000, dk=0x200000, q=0x300000, k=0x400000, cos=0x500000, sin=0x600000,
                 pos=None, wq=None, wk=None, qo=0x700000, ko=0x800000, dwq=0x900000, dwk=0xA00000,
                 work=0x10000000, size=p.workspace_bytes)
        a.update(kw)
        eb.ebin_heads_grad_execute(p.handle, *[a[n] for n in (
            "dq", "dk", "q", "k", "cos", "sin", "pos", "wq", "wk", "qo", "ko", "dwq", "dwk",
            "work", "size")], 0)

    for missing in ("dq", "dk", "q", "k", "cos", "sin", "qo", "ko", "work"):
        assert code(grad, **{missing: None}) == "invalid_arg"
    assert code(grad, size=p.workspace_bytes - 1) == "invalid_arg"
    assert code(grad, work=0x10000004) == "invalid_arg"
    assert code(grad, dwk=0xA00002) == "invalid_arg"
    assert code(grad, qo=0x300010) == "alias"
    assert code(grad, dwq=0x700000) == "alias"
    assert code(grad, dwq=0xA00010) == "alias"
    assert code(grad, dwk=0x10000000) == "alias"
    assert code(grad, work=0x400000) == "alias"
    with pytest.raises(eb.EbinError):
        eb.execute_heads_grad(heads(), *([None] * 14), stream=0)


def test_rotary_table_refusals():
    def table(positions=4, first=0, cos=0x1000, sin=0x2000, **kw):
        v = dict(rotary_dim=8, scaling=0, base=1e4, factor=2.0, trained_length=64.0,
                 slow_turns=1.0, fast_turns=32.0, amplitude=1.0)
        v.update(kw)
        eb.ebin_rotary_table(eb.ebin_rotary_attrs(**v), first, positions, cos, sin, 0)

    for bad in (dict(rotary_dim=7), dict(rotary_dim=0), dict(scaling=4), dict(base=0.0),
                dict(base=float("nan")), dict(scaling=1, factor=0.5), dict(amplitude=0.0),
                dict(scaling=2, rotary_dim=2), dict(scaling=3, trained_length=0.0),
                dict(scaling=3, slow_turns=32.0)):
        assert code(table, **bad) == "invalid_attr"
    assert code(table, positions=-1) == "invalid_arg"
    assert code(table, first=-1) == "invalid_arg"
    assert code(table, cos=None) == "invalid_arg"
    assert code(table, cos=0x1002) == "invalid_arg"
    assert code(table, sin=0x1010) == "alias"
    table(positions=0, cos=None, sin=None)


def gemm(dtype="bfloat16", m=64, n=96, k=80, **kw):
    return eb.GemmPlan(dtype, m, n, k, **kw)


def test_gemm_plan_refusals():
    for dtype in ("float32", "float64", "int8"):
        assert code(gemm, dtype) == "unsupported_type"
    assert code(gemm, bias="float16") == "unsupported_type"
    for sizes in ((-1, 2, 2), (2, -1, 2), (2, 2, -1), (1 << 31, 2, 2), (2, 2, 1 << 31)):
        assert code(gemm, "bfloat16", *sizes) == "invalid_arg"
    assert code(gemm, lda=79) == "invalid_arg"
    assert code(gemm, trans_b=True, ldb=79) == "invalid_arg"
    assert code(gemm, ldb=95) == "invalid_arg"
    assert code(gemm, ldy=1 << 60) == "invalid_arg"
    with pytest.raises(KeyError):
        gemm(activation="tanh")
    attrs = eb.ebin_gemm_attrs(16, 16, 0, 0, 9, 0, 0, 0, 4, 4, 4, 0, 0, 0, 0, 0)
    assert code(eb.ebin_gemm_plan_create, attrs) == "invalid_attr"
    attrs = eb.ebin_gemm_attrs(16, 16, 2, 0, 0, 0, 0, 0, 4, 4, 4, 0, 0, 0, 0, 0)
    assert code(eb.ebin_gemm_plan_create, attrs) == "invalid_attr"


def test_gemm_workspace():
    """Copies only of operands whose rows are off 16 bytes; rows of whole 128-byte lines."""
    assert gemm().workspace_bytes == 0
    assert gemm(k=81).workspace_bytes == 64 * 128 * 2               # A's rows; B's are 96 wide
    assert gemm(k=81, trans_b=True).workspace_bytes == (64 + 96) * 128 * 2
    assert gemm(m=1, k=81).workspace_bytes == 0                     # one row has no step
    assert gemm(any_alignment=True).workspace_bytes == (64 * 128 + 80 * 128) * 2
    assert gemm(k=0, any_alignment=True).workspace_bytes == 0


def test_gemm_execute_refusals():
    def run(plan, a=0x100000, b=0x200000, bias=None, r=None, y=0x300000, z=None, work=None,
            size=0):
        eb.ebin_gemm_execute(plan.handle, a, b, bias, r, y, z, work, size, 0)

    p = gemm()
    for missing in ("a", "b", "y"):
        assert code(run, p, **{missing: None}) == "invalid_arg"
    assert code(run, gemm(bias="float32")) == "invalid_arg"
    assert code(run, gemm(residual=True)) == "invalid_arg"
    assert code(run, p, a=0x100002) == "invalid_arg"                # off 16 bytes
    assert code(run, p, y=0x300001) == "invalid_arg"                # off the element size
    assert code(run, gemm(bias="float32"), bias=0x400002) == "invalid_arg"
    odd = gemm(k=81)
    assert code(run, odd) == "invalid_arg"                          # no workspace
    assert code(run, odd, work=0x800000, size=odd.workspace_bytes - 1) == "invalid_arg"
    assert code(run, odd, work=0x800008, size=odd.workspace_bytes) == "invalid_arg"
    assert code(run, odd, work=0x100000, size=odd.workspace_bytes) == "alias"
    assert code(run, p, y=0x100010) == "alias"
    assert code(run, p, y=0x200000) == "alias"
    assert code(run, p, z=0x300000) == "alias"
    assert code(run, gemm(residual=True), r=0x300010) == "alias"
    assert code(run, gemm(residual=True, ldy=104), r=0x300000) == "alias"   # another stride
    assert code(run, gemm(bias="bfloat16"), bias=0x300000) == "alias"
    run(gemm(m=0), a=None, b=None, y=None)
    run(gemm(n=0), a=None, b=None, y=None)


def test_epilogue_grad_refusals():
    def plan(dtype="bfloat16", m=16, n=24, activation="silu", bias=True, **kw):
        return eb.EpilogueGradPlan(dtype, m, n, activation=activation, bias=bias, **kw)

    assert code(plan, "float64") == "unsupported_type"
    assert code(plan, m=-1) == "invalid_arg"
    assert code(plan, ld_dz=23) == "invalid_arg"
    p = plan()

    def run(p, dy=0x100000, z=0x200000, dz=0x300000, db=0x400000, work=0x500000, size=None):
        eb.ebin_epilogue_grad_execute(p.handle, dy, z, dz, db, work,
                                      p.workspace_bytes if size is None else size, 0)

    for missing in ("dy", "z", "dz", "db", "work"):
        assert code(run, p, **{missing: None}) == "invalid_arg"
    assert code(run, p, size=p.workspace_bytes - 1) == "invalid_arg"
    assert code(run, p, dy=0x100001) == "invalid_arg"
    assert code(run, p, dz=0x100002) == "alias"
    assert code(run, plan(ld_dz=32), dz=0x100000) == "alias"
    assert code(run, p, db=0x300000) == "alias"
    assert code(run, p, work=0x200000) == "alias"
    assert code(run, p, work=0x400000) == "alias"
    run(plan(n=0), dy=None, z=None, dz=None, db=None, work=None)
