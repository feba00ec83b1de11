"""What the one-call forms of the layer operators check and pass on, on the CPU:
tensors stand in for device ones, and the launches are recorded."""
import pytest
import torch

import broadcast_elementwise_gb300 as eb

BF16 = torch.bfloat16


@pytest.fixture
def recorded(monkeypatch):
    """CPU tensors pass for CUDA ones; launches are recorded, not made."""
    calls = []
    monkeypatch.setattr(eb, "_same_device", lambda *a: None)
    for name in ("execute_gemm", "execute_epilogue_grad", "execute_heads", "execute_heads_grad"):
        monkeypatch.setattr(eb, name, lambda *a, _name=name, **kw: calls.append((_name, a, kw)))
    return calls


def mat(*shape):
    return torch.zeros(shape, dtype=BF16)


# ------------------------------------------------------------------ rows that lie on one another

def test_a_matrix_keeps_its_row_stride():
    for t, ld in ((mat(5, 8), 8), (mat(5, 24)[:, 8:16], 24), (mat(1, 8), 8), (mat(0, 8), 8),
                  (mat(5, 1), 1), (mat(5, 7)[:, 2:3], 7), (mat(1, 8).expand(1, 8), 8)):
        assert eb._matrix("here", t, None, BF16, t.device) == ld


EXPANDED = [mat(1, 16).expand(8, 16),              # strides (0, 1)
            mat().expand(8, 1),                    # (0, 0): the gradient of a sum, [m, 1]
            mat(64).as_strided((8, 16), (5, 1)),   # rows that overlap
            mat(64).as_strided((8, 1), (0, 1))]


@pytest.mark.parametrize("t", EXPANDED, ids=lambda t: str(tuple(t.stride())))
def test_overlapping_rows_are_refused(t):
    with pytest.raises(ValueError, match="rows"):
        eb._matrix("here", t, None, BF16, t.device)


def test_expanded_operands_of_a_product_are_refused(recorded):
    a, b, row = mat(8, 32), mat(32, 16), mat(1, 16)
    for kw in (dict(residual=row.expand(8, 16)), dict(out=row.expand(8, 16)),
               dict(preact=row.expand(8, 16))):
        with pytest.raises(ValueError, match="rows"):
            eb.gemm(a, b, **kw)
    with pytest.raises(ValueError, match="rows"):
        eb.gemm(mat(1, 32).expand(8, 32), b)
    with pytest.raises(ValueError, match="rows"):
        eb.gemm(a, mat(1, 16).expand(32, 16))
    with pytest.raises(ValueError, match="rows"):
        eb.gemm(a, mat(1, 32).expand(16, 32), trans_b=True)
    for dy in (row.expand(8, 16), mat().expand(8, 1)):
        with pytest.raises(ValueError, match="rows"):
            eb.gemm_epilogue_grad(dy)
    dense = mat(8, 16)
    with pytest.raises(ValueError, match="rows"):
        eb.gemm_epilogue_grad(dense, row.expand(8, 16), activation="silu")
    with pytest.raises(ValueError, match="rows"):
        eb.gemm_epilogue_grad(dense, out=row.expand(8, 16))
    assert not recorded


def test_a_row_stride_of_zero_is_no_plan():
    """None means dense rows; 0, which a broadcast tensor's stride() gives, does not."""
    for name in ("lda", "ldb", "ldy", "ld_residual", "ld_preact"):
        with pytest.raises(ValueError, match=name):
            eb.GemmPlan(BF16, 8, 16, 32, **{name: 0})
        eb.GemmPlan(BF16, 8, 16, 32, **{name: 32})
    for name in ("ld_dy", "ld_z", "ld_dz"):
        with pytest.raises(ValueError, match=name):
            eb.EpilogueGradPlan(BF16, 8, 16, **{name: 0})
        eb.EpilogueGradPlan(BF16, 8, 16, **{name: 16})
