"""Refusals of dropout, of the norms around a block and of several axes' plans, and the words that
dropout draws.  CPU: the checks run before any device call, and the addresses given are
never dereferenced."""
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

import block_ref as ref
import broadcast_elementwise_gb300 as eb

BF16, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")


def code(fn, *a, **kw):
    with pytest.raises(eb.EbinError) as e:
        fn(*a, **kw)
    return e.value.code


# ------------------------------------------------------------------ the words

def test_philox_known_answers():
    """The published test vectors of Philox4x32-10."""
    for counter, key, want in (
            ((0,) * 4, (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
            ((0xffffffff,) * 4, (0xffffffff,) * 2,
             (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
            ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
             (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))):
        got = ref.philox([np.uint64(c) for c in counter], key)
        assert tuple(int(v) for v in got) == want


def test_shares_of_what_is_kept():
    for p in (0.1, 0.5, 0.9):
        m = ref.mask(p, 1, 2, 512, 512)
        # five deviations of a binomial share
        assert abs(float((m == 0).double().mean()) - p) < 5 * (p * (1 - p)) ** 0.5 / 512
        assert abs(float(m.mean()) - 1) < 5 * (p / (1 - p)) ** 0.5 / 512


# ------------------------------------------------------------------ dropout

def drop(dtype="bfloat16", rows=4, n=32, p=0.5, **kw):
    return eb.DropoutPlan(dtype, rows, n, p, **kw)


def test_dropout_plan_refusals():
    for dtype in ("int32", "float64", "bool"):
        assert code(drop, dtype) == "unsupported_type"
    assert code(drop, bias="float16") == "unsupported_type"
    for p in (-0.1, 1.0, 1.5, NAN, 1 - 2.0 ** -40):
        assert code(drop, p=p) == "invalid_attr"
    assert code(drop, residual=True, gradient=True) == "invalid_attr"
    for kw in (dict(rows=-1), dict(n=-1), dict(rows=(1 << 30) + 1), dict(n=(1 << 30) + 1),
               dict(ld_x=31), dict(ld_y=16), dict(ld_residual=1), dict(ld_x=1 << 60)):
        assert code(drop, **kw) == "invalid_arg"
    with pytest.raises(ValueError):
        drop(ld_x=0)
    assert drop(gradient=True).workspace_bytes == 0
    assert drop(gradient=True, bias="float32").workspace_bytes > 0


def test_dropout_execute_refusals():
    def run(plan, x=0x100000, y=0x200000, bias=None, residual=None, word=None):
        eb.execute_dropout(plan, x, y, 1, 2, bias=bias, residual=residual, offset_device=word,
                           stream=0)

    assert code(run, drop(), x=None) == "invalid_arg"
    assert code(run, drop(), y=None) == "invalid_arg"
    assert code(run, drop(bias="float32")) == "invalid_arg"
    assert code(run, drop(residual=True)) == "invalid_arg"
    assert code(run, drop(gradient=True)) == "invalid_arg"
    assert code(run, drop(), x=0x100001) == "invalid_arg"
    assert code(run, drop(), word=0x300004) == "invalid_arg"
    assert code(run, drop(bias="float32"), bias=0x300002) == "invalid_arg"
    assert code(run, drop(), y=0x100002) == "alias"
    assert code(run, drop(ld_y=40), y=0x100000) == "alias"        # in place, another stride
    assert code(run, drop(residual=True), residual=0x200040) == "alias"
    assert code(run, drop(bias="float32"), bias=0x200010) == "alias"
    assert code(run, drop(), word=0x200010) == "alias"

    def grad(plan, dy=0x100000, dx=0x200000, dbias=None, work=None, size=0, word=None):
        eb.ebin_dropout_grad_execute(plan.handle, dy, dx, dbias, work, size, 1, 2, word, 0)

    p = drop(gradient=True, bias="float32")
    good = dict(dbias=0x300000, work=0x400000, size=p.workspace_bytes)
    assert code(grad, drop()) == "invalid_arg"
    for kw in (dict(dbias=None), dict(dbias=0x300002), dict(work=None), dict(work=0x400008),
               dict(size=p.workspace_bytes - 1)):
        assert code(grad, p, **dict(good, **kw)) == "invalid_arg"
    for kw in (dict(dbias=0x100010), dict(work=0x200000), dict(dbias=0x400000),
               dict(word=0x300008), dict(dx=0x100002)):
        assert code(grad, p, **dict(good, **kw)) == "alias"


def test_dropout_columns_of_one_buffer_that_overlap():
    """As test_block_columns_of_one_buffer_that_overlap."""
    p = drop(residual=True, ld_x=80, ld_residual=80, ld_y=80)
    x, res = 0x100000, 0x100000 + 64
    for y in (x + 2, x + 98, x + 160, res - 2, res - 160, res + 320 - 62):
        assert code(eb.execute_dropout, p, x, y, 1, residual=res, stream=0) == "alias"
    p = drop(residual=True, ld_x=80, ld_residual=80, ld_y=84)
    assert code(eb.execute_dropout, p, x, x + 128, 1, residual=res, stream=0) == "alias"
    p = drop(gradient=True, ld_x=80, ld_y=80)
    assert code(eb.execute_dropout_grad, p, x, x + 62, 1, stream=0) == "alias"


# ------------------------------------------------------------------ norms around a block

def block(dtype="bfloat16", rows=4, n=32, **kw):
    return eb.BlockNormPlan(dtype, rows, n, **kw)


def test_block_plan_refusals():
    for dtype in ("int32", "float64", "bool"):
        assert code(block, dtype) == "unsupported_type"
    for name in ("stream_dtype", "weight_dtype", "mod_dtype"):
        assert code(block, **{name: "float16"}) == "unsupported_type"
        block(**{name: "float32"})
    for kw in (dict(epsilon=-1.0), dict(epsilon=NAN), dict(epsilon_post=INF), dict(dropout=1.0),
               dict(dropout=-0.5), dict(stream_scale=INF), dict(branch_scale=NAN),
               dict(branch=False, post="rms"), dict(branch=False, dropout=0.5)):
        assert code(block, **kw) == "invalid_attr"
    for kw in (dict(rows=-1), dict(n=-1), dict(rows=(1 << 30) + 1), dict(n=(1 << 24) + 1),
               dict(gate_rows=3), dict(mod_rows=8), dict(gate_rows=2, mod_rows=4),
               dict(ld_x=31), dict(ld_dz=8), dict(ld_gate=31), dict(ld_y=1 << 60),
               dict(rows=1 << 30, n=1 << 24, gate_rows=1, gradient=True)):
        assert code(block, **kw) == "invalid_arg"
    with pytest.raises(KeyError):
        block(pre="batch")
    for kw in (dict(gate_rows=0), dict(mod_rows=-1), dict(ld_scale=0)):
        with pytest.raises(ValueError):
            block(**kw)
    assert block().workspace_bytes == 0
    assert block(gradient=True).workspace_bytes > 0
    assert code(eb.HeadsPlan, "bfloat16", (1, 2, 3, 4), norm="layer",
                rotary_dim=0) == "invalid_attr"


def test_kernels_that_no_call_reaches_are_not_built():
    """Forward, only 16-bit streams off the vectors go to the kernel that shifts rows."""
    if shutil.which("nm") is None:
        pytest.skip("no nm")
    names = subprocess.run(["nm", "-C", eb.LIB_PATH], capture_output=True, text=True).stdout
    built = set(re.findall(r"void ebin::k_block_unit<(\w+), (\w+), (true|false), (true|false)>\(",
                           names))
    pairs = [("float", "float"), ("__half", "__half"), ("__nv_bfloat16", "__nv_bfloat16"),
             ("__half", "float"), ("__nv_bfloat16", "float")]
    assert built == ({(t, s, layer, "false") for t, s in pairs for layer in ("true", "false")} |
                     {(t, s, "true", "true") for t, s in pairs if s != "float"})


def test_workspace_of_wide_rows():
    """No more than 2^28 sums of 4 bytes, but for a unit a group of all four kinds."""
    for rows in (1, 17, 152, 456, 20000):
        for n in (64, 4096, 8192, 8193, 16384, 40000, 1 << 20, 1 << 24):
            for kw in ({}, dict(gate_rows=rows, mod_rows=rows), dict(gate_rows=1)):
                groups = rows if kw.get("gate_rows") == 1 else 1
                if groups * n // 32 > 2 ** 31 - 1:      # CTAs of the last step: refused
                    continue
                got = block(rows=rows, n=n, gradient=True, post="layer", **kw).workspace_bytes
                assert 0 < got <= 4 * max(1 << 28, 4 * groups * (n + 3)), (rows, n, kw)


def test_block_execute_refusals():
    def run(plan, x=0x100000, y=0x200000, h=0x300000, z=0x400000, **kw):
        eb.execute_block_norm(plan, x, y, h, z, stream=0, **kw)

    p = block()
    assert code(run, p, x=None) == "invalid_arg"
    assert code(run, p, y=None) == "invalid_arg"
    assert code(run, block(gradient=True)) == "invalid_arg"
    assert code(run, block(branch=False), gate=0x500000) == "invalid_arg"
    for kw in (dict(x=0x100001), dict(h=0x300001), dict(z=0x400001), dict(gate=0x500001),
               dict(w_pre=0x500001), dict(scale=0x500001), dict(offset_device=0x500004)):
        assert code(run, p, **kw) == "invalid_arg"
    for kw in (dict(w_post=0x500000), dict(b_post=0x500000)):
        assert code(run, p, **kw) == "invalid_arg"                         # post is none
    for name in ("w_pre", "b_pre", "scale", "shift"):
        assert code(run, block(pre="none"), **{name: 0x500000}) == "invalid_arg"
    assert code(run, block(stream_dtype="float32"), x=0x100002) == "invalid_arg"
    assert code(run, block(weight_dtype="float32"), b_pre=0x500002) == "invalid_arg"
    assert code(run, block(mod_dtype="float32"), gate=0x500002) == "invalid_arg"
    # 256 bytes a matrix
    for kw in (dict(h=0x100002), dict(z=0x100010), dict(z=0x300080), dict(w_pre=0x300000),
               dict(shift=0x400010), dict(gate=0x300010)):
        assert code(run, p, **kw) == "alias"
    assert code(run, block(dropout=0.5), offset_device=0x300000) == "alias"
    assert code(run, block(ld_h=40), h=0x100000) == "alias"            # in place, another stride
    assert code(run, block(stream_dtype="float32"), z=0x100000) == "alias"   # and another type


def test_block_columns_of_one_buffer_that_overlap():
    """Rows of 64 bytes, 160 bytes apart; side by side without sharing a byte they are accepted
    (on the GPU)."""
    p = block(ld_x=80, ld_y=80, ld_h=80, ld_z=80)

    def run(x, y, h, z, plan=p):
        eb.execute_block_norm(plan, x, y, h, z, stream=0)

    x, y = 0x100000, 0x100000 + 64
    for h, z in ((x, x), (x, x + 160), (x, x + 62), (x, y + 2), (x + 98, y), (x + 160 - 62, y),
                 (y, y + 160), (x + 320 - 2, None)):
        assert code(run, x, y, h, z) == "alias", (h - x, z and z - x)
    wide = block(ld_x=80, ld_y=80, ld_h=84, ld_z=80)      # another stride crosses the columns
    assert code(run, x, y, x + 128, None, plan=wide) == "alias"


def test_block_grad_refusals():
    p = block(gradient=True, post="rms")
    good = dict(dz=0x100000, dh=0x110000, h=0x120000, y=0x130000, dx=0x140000, dy=0x150000,
                work=0x10000000, size=p.workspace_bytes, params={}, grads={})

    def grad(plan=p, **kw):
        a = dict(good, **kw)
        params = eb.ebin_block_norm_params(**a["params"])
        eb.ebin_block_norm_grad_execute(plan.handle, a["dz"], a["dh"], a["h"], a["y"], params,
                                        a["dx"], a["dy"], eb.ebin_block_norm_grads(**a["grads"]),
                                        a["work"], a["size"], 0)

    some = dict(grads=dict(w_pre=0x160000))
    assert code(grad, block()) == "invalid_arg"
    for kw in (dict(dz=None), dict(h=None), dict(y=None), dict(dx=0x140001), dict(dy=0x150001),
               dict(grads=dict(w_pre=0x160002)), dict(some, work=None),
               dict(some, work=0x10000008), dict(some, size=p.workspace_bytes - 1)):
        assert code(grad, **kw) == "invalid_arg"
    bare = block(gradient=True, branch=False)
    assert code(grad, bare) == "invalid_arg"                           # dy without a branch
    assert code(grad, bare, dy=None, grads=dict(gate=0x160000)) == "invalid_arg"
    assert code(grad, block(gradient=True), grads=dict(w_post=0x160000)) == "invalid_arg"
    off = block(gradient=True, pre="none")
    for name in ("w_pre", "b_pre", "scale", "shift"):
        assert code(grad, off, grads={name: 0x160000}) == "invalid_arg"
    assert code(grad, block(gradient=True), y=None, grads=dict(gate=0x160000)) == "invalid_arg"
    for kw in (dict(dx=0x100010), dict(dy=0x140000), dict(grads=dict(w_pre=0x140010)),
               dict(grads=dict(w_pre=0x160000, b_pre=0x160010)), dict(some, work=0x130000),
               dict(some, work=0x160000), dict(some, params=dict(w_pre=0x160020))):
        assert code(grad, **kw) == "alias"
    assert code(grad, block(gradient=True, stream_dtype="float32", post="rms"),
                dx=0x100000) == "alias"


@pytest.fixture
def on_cpu(monkeypatch):
    """CPU tensors pass for CUDA ones; launches are recorded, not made."""
    import contextlib
    calls = []
    monkeypatch.setattr(eb, "_same_device", lambda *a: None)
    monkeypatch.setattr(eb, "_launching", lambda *a: contextlib.nullcontext())
    for name in ("execute_block_norm", "execute_block_norm_grad", "execute_dropout",
                 "execute_dropout_grad"):
        monkeypatch.setattr(eb, name, lambda *a, _name=name, **kw: calls.append(_name))
    return calls


def mat(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype)


def test_one_call_forms_check_their_arguments(on_cpu):
    x, y, row = mat(8, 32), mat(8, 32), mat(1, 32)
    for kw in (dict(w_pre=mat(31)), dict(w_pre=mat(64)[::2]), dict(w_pre=mat(32), b_pre=mat(32, dtype=F32)),
               dict(gate=mat(3, 32)), dict(gate=mat(2, 31)), dict(gate=mat(2, 32).t().contiguous().t()),
               dict(scale=mat(2, 32), shift=mat(4, 32)), dict(scale=mat(32), shift=mat(4, 32)),
               dict(gate=mat(32), scale=mat(32, dtype=F32)), dict(out=(mat(8, 32, dtype=F32), None)),
               dict(out=(None, row.expand(8, 32))), dict(gate=row.expand(2, 32)),
               dict(offset_device=torch.zeros(2, dtype=torch.int64)),
               dict(offset_device=torch.zeros(1))):
        with pytest.raises(ValueError):
            eb.block_norm(x, y, **kw)
    for bad in ((mat(8, 33), y), (x, mat(7, 32)), (row.expand(8, 32), y), (mat(8, 8, 32), y)):
        with pytest.raises(ValueError):
            eb.block_norm(*bad)
    for a in ((None, x, x), (y, x, None)):
        with pytest.raises(ValueError):
            eb.block_norm_grad(*a)
    with pytest.raises(ValueError):
        eb.block_norm_grad(None, None, None, y, pre="none")
    with pytest.raises(ValueError):
        eb.block_norm_grad(y, x, x, None, post="rms")
    for kw in (dict(bias=mat(31)), dict(residual=mat(8, 31)), dict(residual=row.expand(8, 32)),
               dict(out=mat(8, 32, dtype=F32)), dict(offset_device=torch.zeros(1))):
        with pytest.raises(ValueError):
            eb.dropout(x, 0.5, 1, **kw)
    with pytest.raises(ValueError):
        eb.dropout(mat(32), 0.5, 1)
    with pytest.raises(ValueError):
        eb.dropout_grad(mat(2, 2, 2), 0.5, 1)
    assert not on_cpu
    h, z = eb.block_norm(x, y, gate=mat(2, 32), scale=mat(4, 32)[::2], shift=mat(2, 96)[:, 32:64])
    assert h.shape == z.shape == x.shape
    eb.block_norm(mat(8, 32, dtype=F32), y, w_pre=mat(32, dtype=F32))
    assert eb.block_norm(x, pre="layer")[0] is None
    assert eb.block_norm(x, y, pre="none")[1] is None
    eb.dropout(x, 0.5, -1, 1 << 80)
    assert len(on_cpu) == 5


def test_one_row_is_a_row_for_all_beside_groups(on_cpu):
    x, y = mat(8, 32), mat(8, 32)
    for kw in (dict(gate=mat(1, 32), scale=mat(4, 32)), dict(gate=mat(2, 32), shift=mat(1, 32)),
               dict(gate=mat(4, 32), scale=mat(1, 32), shift=mat(32)),
               dict(gate=mat(3, 32)[1:2], scale=mat(4, 32), shift=mat(4, 32))):
        eb.block_norm(x, y, **kw)
        grads = eb.block_norm_grad(y, x, x, y, **kw)
        assert all(grads[k].shape == t.shape for k, t in kw.items())
    assert len(on_cpu) == 8
    with pytest.raises(ValueError, match="every 4 rows beside a scale or shift for every 2"):
        eb.block_norm(x, y, gate=mat(2, 32), scale=mat(4, 32))
    with pytest.raises(ValueError, match="same groups"):
        eb.block_norm(x, y, scale=mat(1, 32), shift=mat(4, 32))


def test_a_z_that_there_is_not(on_cpu):
    """Nothing would write it, so it is not handed back as the result."""
    x = mat(8, 32)
    with pytest.raises(ValueError, match="no z"):
        eb.block_norm(x, x, pre="none", out=(None, mat(8, 32)))
    h = mat(8, 32)
    assert eb.block_norm(x, x, pre="none", out=(h, None)) == (h, None)


def test_an_empty_batch_has_no_groups(on_cpu):
    x, none = mat(0, 32), mat(0, 32)
    h, z = eb.block_norm(x, x, gate=none, scale=none, shift=none)
    assert h.shape == z.shape == (0, 32)
    grads = eb.block_norm_grad(x, x, x, x, gate=none, scale=mat(1, 32), shift=mat(32))
    assert [tuple(grads[k].shape) for k in ("gate", "scale", "shift")] == [(0, 32), (1, 32), (32,)]
    assert len(on_cpu) == 2
    for gate in (none, mat(3, 32)):
        with pytest.raises(ValueError, match="groups dividing the rows"):
            eb.block_norm(mat(8, 32), mat(8, 32), gate=gate)


# ------------------------------------------------------------------ several axes

def axes(sections=(8, 12, 12), order="blocks", **kw):
    kw.setdefault("table_positions", 16)
    kw.setdefault("positions", "int32")
    return eb.HeadsPlan("bfloat16", (2, 4, 5, 64), (2, 4, 1, 64), axes=sections, axes_order=order,
                        **kw)


def test_axes_plan_refusals():
    for sections in ((8, 12, 11), (33,), (0, 0, 0), (40, -8), (16, 16, 1)):
        assert code(axes, sections) == "invalid_attr"
    assert code(axes, positions=None) == "invalid_attr"
    assert code(axes, rotary_dim=0) == "invalid_attr"
    assert code(axes, norm="layer") == "invalid_attr"
    assert code(axes, table_positions=1 << 31) == "invalid_arg"
    assert code(axes, position_strides=(-1, 4, 1)) == "invalid_arg"
    assert code(axes, position_strides=(1 << 60, 4, 1)) == "invalid_arg"
    for sections in ((), (1, 1, 1, 1, 28)):
        with pytest.raises(ValueError):
            axes(sections)
    with pytest.raises(ValueError):
        axes(position_strides=(4, 1))
    with pytest.raises(KeyError):
        axes(order="mixed")
    axes((0, 32, 0, 0), "dealt", norm="rms", gradient=True)
    a = eb.ebin_heads_attrs()
    assert code(eb.ebin_heads_plan_create_axes, a, eb.ebin_rotary_axes()) == "unsupported_type"


def test_axes_execute_refusals():
    p = axes()

    def run(q=0x100000, k=0x200000, cos=0x300000, sin=0x400000, pos=0x700000, qo=0x500000,
            ko=0x600000):
        eb.execute_heads(p, q, k, cos, sin, pos, qo, ko, stream=0)

    assert code(run, pos=None) == "invalid_arg"
    assert code(run, pos=0x700002) == "invalid_arg"
    # three axes of 8 positions, 96 bytes, behind one another
    assert code(run, pos=0x500000 - 92) == "alias"


def test_axes_table_refusals():
    def table(rotary_dim=64, sections=(8, 12, 12), order=0, count=None, scaling=0):
        x = eb.ebin_rotary_axes(len(sections) if count is None else count, order)
        for i, s in enumerate(sections):
            x.sections[i] = s
        v = eb.ebin_rotary_attrs(rotary_dim, scaling, 1e4, 2.0, 64.0, 1.0, 32.0, 1.0)
        eb.ebin_rotary_table_axes(v, x, 0, 4, 0x1000, 0x1000, 0)

    for kw in (dict(rotary_dim=62), dict(sections=(8, 12, -12)), dict(order=2), dict(order=-1),
               dict(count=0), dict(count=5), dict(scaling=2), dict(rotary_dim=2048,
                                                                   sections=(1024,))):
        assert code(table, **kw) == "invalid_attr"
    assert code(table) == "alias"          # both tables at one address


def test_axes_positions_of_the_one_call_forms(on_cpu, monkeypatch):
    monkeypatch.setattr(eb, "execute_heads", lambda *a, **kw: on_cpu.append(a))
    q, cos = mat(2, 3, 4, 8), torch.zeros(3, 4)
    at = torch.zeros(2, 2, 3, dtype=torch.int32)
    eb.rotary(q, None, cos, cos, at, axes=(2, 2))
    eb.rotary(q, None, cos, cos, at[:, 0].long(), axes=(2, 2))
    assert len(on_cpu) == 2
    for bad in (None, at[0, 0], at[:, :1], at.float(), torch.zeros(3, 2, 3, dtype=torch.int32)):
        with pytest.raises(ValueError):
            eb.rotary(q, None, cos, cos, bad, axes=(2, 2))
