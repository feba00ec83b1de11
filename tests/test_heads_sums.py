"""The bound on the head norms' weight gradients, on the CPU: at sizes where groups walk many
items it rejects a sum of nothing, one with an item left out and one without a CTA's part,
and accepts a plain binary32 sum."""
import pytest
import torch

import heads_sums as sums
import layer_ref as ref

# k heads of the sizes at which groups of lanes walk several items each
SIZES = [(2, 4096, 8, 128, 128, "half"), (1, 9001, 5, 96, 46, "half"),
         (3, 4099, 3, 80, 40, "interleaved"), (1, 12001, 9, 64, 32, "half")]


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_the_bound_sees_what_is_missing(size):
    B, S, H, D, r, layout = size
    g = torch.Generator().manual_seed(1)
    x, dy = (torch.randn(B, S, H, D, generator=g) for _ in range(2))
    cos, sin = (c[torch.arange(S)].expand(B, S, -1) for c in ref.table(S, r))
    t, s = sums.terms(dy.double(), x.double(), cos, sin, layout, 1e-5)
    want, b = t.sum((0, 1, 2)), sums.bound(t, s, 0.2, 152)
    assert (b < 1e-3 * want.abs().max()).all()
    rows = t.reshape(-1, D)
    plain = torch.zeros(D)
    for part in rows.float().split(512):                   # a binary32 sum in parts
        plain = plain + part.sum(0)
    assert sums.outside(plain, want, b) == 0
    item = rows[:min(H, 4)].sum(0)
    cta = rows[::max(1, rows.shape[0] // 60)].sum(0)
    assert sums.outside(torch.zeros(D), want, b) > 0.9 * D
    assert sums.outside((want - item).float(), want, b) > 0.5 * D
    assert sums.outside((want - cta).float(), want, b) > 0.9 * D
    assert sums.outside((want + item).float(), want, b) > 0.5 * D      # an item taken twice
