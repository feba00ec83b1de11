"""The activations and their slopes on 16-bit data, held to their own size: an error bound
relative to the result, down to the tails that a bound in units of 1 cannot see.

Bound: the type's rounding, and 6e-5 of the value: 2.6e-5 of the normal distribution's fit;
the exponential's argument, of at most 130 in powers of 2, formed in four binary32 roundings
(130 * 4 * 2^-24 * ln 2 = 2.2e-5, met only at the far end); 16 roundings of 2^-23 beside them.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

import broadcast_elementwise_gb300 as eb  # noqa: E402
import layer_ref as ref  # noqa: E402

F16, BF16 = torch.float16, torch.bfloat16
KINDS = ["gelu", "gelu_tanh", "silu"]
RELATIVE = 6e-5


def every(dtype, lowest):
    """Every value of the type in [lowest, 0), as one column."""
    bits = torch.arange(1, 1 << 15, dtype=torch.int32)
    z = (bits - (1 << 15)).to(torch.int16).view(dtype)      # the sign bit set
    z = z[z.isfinite() & (z >= lowest) & (z < 0)]
    return z.reshape(-1, 1).cuda()


def check(got, want, scale, what):
    bound = ref.ROUND[got.dtype] * want.abs() + 1.01 * RELATIVE * scale + ref.TINY[got.dtype]
    # what the exponential cannot hold in 32 bits, and the kernels' arithmetic keeps as 0
    bound = bound + 200 * 2.0 ** -126
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    assert not bad.any(), (what, int(bad.sum()), float((off / bound).max()))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("kind", KINDS)
def test_the_value_of_every_negative(kind, dtype):
    lowest = -8.5 if kind == "gelu_tanh" else -13.0
    z = every(dtype, lowest)
    one = torch.ones(1, 8, dtype=dtype, device="cuda")
    y = eb.gemm(z, one, activation=kind)           # k = 1: z itself is the pre-activation
    want = ref.act(z.double(), kind).expand(-1, 8)
    check(y, want, want.abs(), kind)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("columns", [8, 1])
def test_the_slope_of_every_negative(kind, dtype, columns):
    """The slope is a difference: its bound goes by the two terms' sizes."""
    lowest = -8.5 if kind == "gelu_tanh" else -13.0
    z = every(dtype, lowest).expand(-1, columns).contiguous()
    dz, _ = eb.gemm_epilogue_grad(torch.ones_like(z), z, activation=kind, bias=False)
    zz = z.double()
    want = ref.act_slope(zz, kind)
    value = ref.act(zz, kind) / zz                 # the term without z's slope
    check(dz, want, value.abs() + (want - value).abs(), kind)


def test_a_form_with_an_absolute_bound_is_caught():
    """7.1.26 of the Handbook itself (error 7.5e-8 of 1) does not pass."""
    z = every(BF16, -13.0).double()
    a = -z / 2 ** 0.5
    t = 1 / (1 + 0.3275911 * a)
    c = (0.254829592, -0.284496736, 1.421413741, -1.453152027, 1.061405429)
    phi = 0.5 * sum(k * t ** (i + 1) for i, k in enumerate(c)) * (-a * a).exp()
    want = ref.act(z, "gelu")
    assert ((phi - want / z).abs() < 7.6e-8).all()
    with pytest.raises(AssertionError):
        check((z * phi).to(BF16), want, want.abs(), "7.1.26")
