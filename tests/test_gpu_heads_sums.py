"""The head norms' weight gradients on the GPU within a bound that goes by the additions made
(heads_sums.py), so that an item or a CTA's part left out shows at every size."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import broadcast_elementwise_gb300 as eb  # noqa: E402
import heads_sums as sums  # noqa: E402
import test_gpu_heads as heads  # noqa: E402

MORE = [(1, 3001, 9, 4, 33, 22, "half", "dense"), (2, 2049, 6, 2, 520, 520, "half", "dense"),
        (1, 5000, 3, 1, 192, 192, "half", "odd"), (5, 1, 32, 8, 128, 128, "half", "packed")]


@pytest.mark.parametrize("dtype,wdtype", [(heads.BF16, heads.BF16), (heads.F16, heads.F32),
                                          (heads.F32, heads.F32)])
@pytest.mark.parametrize("shape", heads.MANY + MORE + heads.SHAPES[3:14], ids=str)
def test_weight_gradients(shape, dtype, wdtype):
    B, S, Hq, Hk, D, r, layout, how = shape
    g = heads.gen(12)
    q, k = heads.views(g, B, S, Hq, Hk, D, dtype, how)
    dq, dk = heads.views(g, B, S, Hq, Hk, D, dtype, how)
    wq, wk = ((1 + 0.3 * heads.normal(g, D)).to(wdtype) for _ in range(2))
    cos, sin = heads.tables(S + 3, r)
    at = torch.randint(0, S + 3, (B, S), generator=g, device="cuda")
    eps = 1e-5
    got = eb.qk_norm_rotary_grad(dq, dk, q, k, wq, wk, cos, sin, at, epsilon=eps, layout=layout)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    c, s = heads.rows(cos, at), heads.rows(sin, at)
    for x, d, dw, H in ((q, dq, got[2], Hq), (k, dk, got[3], Hk)):
        t, size = sums.terms(d.double(), x.double(), c, s, layout, eps)
        want, bound = t.sum((0, 1, 2)), sums.bound(t, size, H / (Hq + Hk), sms)
        off = (dw.double() - want).abs()
        assert sums.outside(dw, want, bound) == 0, float((off / bound).max())
        # and the bound would see the last item missing
        item = t.reshape(-1, D)[-min(H, 4):].sum(0)
        assert int((item.abs() > 2 * bound).sum()) > 0.3 * D
    assert eb.get_device_status() == 0
