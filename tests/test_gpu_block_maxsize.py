"""The norms around a block and dropout where elements lie past 2^31 of a buffer: the rows on
either side of that, the first and the last, against the 64-bit form, and the parameters'
gradients, whose sums take in all rows.

Bounds as in test_gpu_block_norm; of a sum over rows a unit of at least 152 adds its rows one after
another and the units follow in 32 strands: rows / 152 + 512 additions at most."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import block_ref as ref  # noqa: E402
import broadcast_elementwise_gb300 as eb  # noqa: E402
import layer_ref  # noqa: E402
from test_gpu_block_norm import BF16, normal, steps  # noqa: E402

WALL = 1 << 31


def rows_of_interest(rows, ld):
    at = WALL // ld
    return torch.tensor(sorted({r for s in (0, at - 4, rows - 8) for r in range(s, s + 8)
                                if 0 <= r < rows}), device="cuda")


def make(seed, rows, n, ld, dtype=BF16):
    """Rows `ld` apart in one buffer."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = torch.empty((rows - 1) * ld + n, dtype=dtype, device="cuda")
    for i in range(0, t.numel(), 1 << 28):
        t[i:i + (1 << 28)].normal_(generator=g)
    return torch.as_strided(t, (rows, n), (ld, 1))


@pytest.mark.parametrize("rows,n,ld", [(270000, 8192, 8192), (270001, 8191, 8191),
                                       (1050000, 2048, 2056), (7, 4096, (1 << 29) + 8),
                                       (70000, 40000, 40000)])
def test_block(rows, n, ld):
    post, pre = "rms", "layer"
    x, y = make(1, rows, n, ld), make(2, rows, n, ld)
    p = {"w_pre": 1 + 0.3 * normal(3, n), "w_post": 1 + 0.3 * normal(4, n)}
    kw = dict(post=post, pre=pre, epsilon=1e-5, epsilon_post=1e-5, **p)
    h, z = eb.block_norm(x, y, out=(make(5, rows, n, ld), None), **kw)
    at = rows_of_interest(rows, ld)
    eps = float(torch.tensor(1e-5))
    want = ref.block(x[at], y[at], post, pre, eps, eps, 1.0, 1.0, 1.0, **p)
    layer_ref.check(h[at], *want[0], steps(n), "h")
    layer_ref.check(z[at], *want[1], steps(n), "z")
    del h, z
    dz, dh = y, x      # another use of the same numbers
    got = eb.block_norm_grad(dz, dh, x, y, **kw)
    want = ref.block_grad(dz[at], dh[at], x[at], y[at], post, pre, eps, eps, 1.0, 1.0, 1.0, **p)
    layer_ref.check(got["x"][at], *want["x"], steps(n), "dx")
    layer_ref.check(got["y"][at], *want["y"], steps(n), "dy")
    sums = {k: [0.0, 0.0] for k in p}
    step = (1 << 27) // n
    for r in range(0, rows, step):
        s = slice(r, r + step)
        part = ref.block_grad(dz[s], dh[s], x[s], y[s], post, pre, eps, eps, 1.0, 1.0, 1.0, **p)
        for k, v in sums.items():
            v[0], v[1] = v[0] + part[k][0], v[1] + part[k][1]
    for k, v in sums.items():
        layer_ref.check(got[k], *v, steps(n) + rows / 152 + 512, "d" + k)


@pytest.mark.parametrize("rows,n,ld", [(270000, 8192, 8192), (270001, 8191, 8191),
                                       (7, 4096, (1 << 29) + 8), (3, 1 << 30, 1 << 30)])
def test_dropout(rows, n, ld):
    p, seed, offset = 0.3, 2 ** 63 + 5, 2 ** 35
    x = make(1, rows, n, ld)
    y = eb.dropout(x, p, seed, offset)
    at = rows_of_interest(rows, ld)
    cols = np.unique(np.concatenate([np.arange(min(n, 4096)), np.arange(max(0, n - 4096), n)]))
    quads = np.unique(cols // 4).astype(np.uint64)
    row = at.cpu().numpy().astype(np.uint64)
    c0, c1 = np.meshgrid(quads, row)
    full = np.ones_like(c0)
    w = ref.philox([c0, c1, full * np.uint64(offset & 0xFFFFFFFF), full * np.uint64(offset >> 32)],
                   [seed & 0xFFFFFFFF, seed >> 32])
    words = np.stack(w, -1).reshape(len(row), -1)
    place = {int(q): i for i, q in enumerate(quads)}
    pick = np.array([4 * place[int(c) // 4] + int(c) % 4 for c in cols])
    keep = torch.from_numpy(words[:, pick] >= np.uint64(ref.bound(p))).cuda()
    m = keep.double() / (1.0 - ref.bound(p) / 2.0 ** 32)
    index = torch.from_numpy(cols.astype(np.int64)).cuda()
    xs, ys = x[at][:, index], y[at][:, index]
    layer_ref.check(ys, m * xs.double(), m * xs.double().abs(), 2, "dropout")
    assert (ys[~keep] == 0).all()
