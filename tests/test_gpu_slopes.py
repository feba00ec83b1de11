"""Derivatives of the epilogue's activations far out and at infinities, in every type and on
both of the gradient's paths (vectors of columns, single ones)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

import broadcast_elementwise_gb300 as eb  # noqa: E402
import layer_ref as ref  # noqa: E402

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
KINDS = ["relu", "gelu", "gelu_tanh", "silu"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("n", [16, 13])
def test_far_out_and_at_infinities(kind, dtype, n):
    """The slope is 0 or 1 from |z| = 100 on (the nearest that a kernel comes to it in 32
    bits, 2^-24 or 2^-149 off, is lost in every type's rounding but binary32's: 1e-6), up to an
    infinite z; a NaN stays one."""
    big = float(torch.finfo(dtype).max)
    far = [100.0, 6e4, big, math.inf]
    z = torch.tensor([far * 2 + [-v for v in far] * 2] * 3, device="cuda", dtype=dtype)[:, :n]
    z = z.contiguous()
    dy = torch.full_like(z, 0.75)
    want = torch.where(z > 0, dy, torch.zeros_like(dy))
    dz, db = eb.gemm_epilogue_grad(dy, z, activation=kind)
    assert ((dz - want).abs() <= 1e-6).all(), (dz, want)
    assert ((db - want.float().sum(0)).abs() <= 1e-5).all()
    z[1, 5] = math.nan
    dz, db = eb.gemm_epilogue_grad(dy, z, activation=kind)
    assert dz[1, 5].isnan() and db[5].isnan()
    assert int(dz.isnan().sum()) == 1 and int(db.isnan().sum()) == 1


@pytest.mark.parametrize("kind", KINDS)
def test_the_gradient_of_a_stored_overflow(kind):
    """A binary16 pre-activation past 65504 is stored as an infinity; its gradient is 0 or dy."""
    k, n = 64, 136
    x = torch.full((4, k), 200.0, dtype=F16, device="cuda")
    x[1::2] *= -1
    w = torch.full((n, k), 20.0, dtype=F16, device="cuda")
    z = torch.empty(4, n, dtype=F16, device="cuda")
    y = eb.gemm(x, w, trans_b=True, activation=kind, preact=z)
    assert z.isinf().all()
    assert (y[1::2] == 0).all() and (y[::2] == math.inf).all()
    dy = torch.full_like(z, 0.5)
    dz, db = eb.gemm_epilogue_grad(dy, z, activation=kind)
    assert (dz[::2] == 0.5).all() and (dz[1::2] == 0).all() and (db == 1.0).all()
    assert eb.gemm(dz, w).isfinite().all()
