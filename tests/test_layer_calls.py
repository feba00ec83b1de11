"""What the one-call forms of the layer operators check and pass on, on the CPU:
tensors stand in for device ones, and the launches are recorded."""
import contextlib
import itertools
import random
import types

import pytest
import torch

import broadcast_elementwise_gb300 as eb

BF16 = torch.bfloat16
needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                                  reason="the addresses would be launched on")


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


# ------------------------------------------------------------------ the stream of what a call allocates

HANDLE = 0x5EA0


@pytest.fixture
def streams(monkeypatch, recorded):
    """Each allocation's size and the address of the stream that was current for it, beside
    the launches (CPU tensors, no device)."""
    seen = types.SimpleNamespace(now=0, blocks=[], launches=recorded)

    class Stream:
        def __init__(self, handle, device=None):
            self.cuda_stream, self.device = handle, torch.device("cpu")

    @contextlib.contextmanager
    def on(stream):
        before, seen.now = seen.now, stream.cuda_stream
        try:
            yield
        finally:
            seen.now = before

    empty = torch.empty

    def recorded_empty(*a, **kw):
        kw["device"] = "cpu"
        t = empty(*a, **kw)
        seen.blocks.append((t.nbytes, seen.now))
        return t

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch, "empty", recorded_empty)
    monkeypatch.setattr(eb, "_stream", lambda s: s if isinstance(s, int) else
                        seen.now if s is None else s.cuda_stream)
    monkeypatch.setattr(eb, "ebin_rotary_table", lambda *a: seen.launches.append(("table", a, {})))
    seen.Stream = Stream
    return seen


def calls_with_memory():
    """Each one-call form, and how many blocks it allocates."""
    x, g = mat(2, 3, 4, 8), mat(2, 3, 2, 8)
    cos = torch.zeros(3, 4)
    return [("gemm", 2, lambda s: eb.gemm(mat(8, 33), mat(33, 16), stream=s)),
            ("gemm into out", 1, lambda s: eb.gemm(mat(8, 33), mat(33, 16), out=mat(8, 16), stream=s)),
            ("gemm_epilogue_grad", 3, lambda s: eb.gemm_epilogue_grad(mat(8, 16), stream=s)),
            ("rotary", 2, lambda s: eb.rotary(x, g, cos, cos, stream=s)),
            ("qk_norm_rotary", 2, lambda s: eb.qk_norm_rotary(x, g, None, None, cos, cos, stream=s)),
            ("qk_norm_rotary_grad", 5,
             lambda s: eb.qk_norm_rotary_grad(x, g, x, g, None, None, cos, cos, stream=s)),
            ("rotary_table", 2, lambda s: eb.rotary_table(4, 8, stream=s))]


@pytest.mark.parametrize("i", range(7), ids=[c[0] for c in calls_with_memory()])
@pytest.mark.parametrize("how", ["stream", "address"])
def test_memory_belongs_to_the_launch_stream(streams, monkeypatch, i, how):
    """A workspace dropped at return must be handed out again in the order of the stream
    that its kernel runs on; no block may come from another stream's pending work."""
    monkeypatch.setattr(torch, "empty_like", lambda t, **kw: torch.empty(t.shape, dtype=t.dtype))
    _, blocks, call = calls_with_memory()[i]
    call(streams.Stream(HANDLE) if how == "stream" else HANDLE)
    assert len(streams.blocks) == blocks and len(streams.launches) == 1
    assert {at for _, at in streams.blocks} == {HANDLE}, streams.blocks
    streams.blocks.clear()
    call(None)
    assert {at for _, at in streams.blocks} == {0}
    assert streams.now == 0


class OnDevice(torch.Tensor):
    """A CPU tensor that passes for a CUDA one and notes which stream its copy was made on."""
    is_cuda = True
    seen = None

    def contiguous(self):
        self.seen.blocks.append((self.nbytes, self.seen.now))
        return torch.Tensor.contiguous(self)


@pytest.mark.parametrize("how", ["stream", "address"])
def test_binary_memory_belongs_to_the_launch_stream(streams, monkeypatch, how):
    monkeypatch.setattr(eb, "execute", lambda *a: streams.launches.append(a))
    monkeypatch.setattr(OnDevice, "seen", streams)
    x = torch.zeros(2, 4, 3).as_subclass(OnDevice)
    block = torch.zeros(4, 4).as_subclass(OnDevice)       # a copied parameter block
    for handle in (HANDLE, 0):
        streams.blocks.clear()
        s = None if not handle else streams.Stream(HANDLE) if how == "stream" else HANDLE
        out = eb.binary("BatchNormalization", x, block, epsilon=1e-5, stream=s)
        assert out.shape == x.shape and len(streams.blocks) == 2
        assert {at for _, at in streams.blocks} == {handle}
    assert len(streams.launches) == 2


def test_a_stream_of_another_device_is_refused(streams):
    s = streams.Stream(HANDLE)
    s.device = torch.device("cuda", 1)
    with pytest.raises(ValueError, match="cuda:1"):
        eb._launching(torch.device("cuda", 0), s)


# ------------------------------------------------------------------ tables

def test_a_rotation_needs_its_tables_length():
    for kw in (dict(), dict(rotary_dim=4), dict(norm="rms")):
        with pytest.raises(ValueError, match="table_positions"):
            eb.HeadsPlan(BF16, (1, 2, 3, 8), **kw)
    eb.HeadsPlan(BF16, (1, 2, 3, 8), norm="rms", rotary_dim=0)
    eb.HeadsPlan(BF16, (1, 2, 3, 8), table_positions=0)


@needs_no_gpu
def test_an_empty_table_may_be_null():
    """Without a row there is nothing to read: the call gets as far as the device."""
    for rows, code in ((0, "cuda"), (1, "invalid_arg")):
        plan = eb.HeadsPlan(BF16, (1, 2, 3, 8), table_positions=rows)
        with pytest.raises(eb.EbinError) as e:
            eb.execute_heads(plan, 0x100000, None, None, None, None, 0x200000, None, stream=0)
        assert e.value.code == code


# ------------------------------------------------------------------ views of one buffer

def outcome(fn, *a, **kw):
    """The status of a call that cannot succeed here: "cuda" once nothing is refused."""
    with pytest.raises(eb.EbinError) as e:
        fn(*a, **kw)
    return e.value.code


def in_place(q, k):
    """Rotate views q and k (CPU tensors for their shapes, strides and addresses) in place."""
    plan = eb.HeadsPlan(q.dtype, q.shape, k.shape, table_positions=16, q_strides=q.stride(),
                        k_strides=k.stride(), q_out_strides=q.stride(), k_out_strides=k.stride())
    at = 1 << 40      # far from the tables
    base = min(q.data_ptr(), k.data_ptr())
    q, k = (at + t.data_ptr() - base for t in (q, k))
    return outcome(eb.execute_heads, plan, q, k, 0x100000, 0x200000, None, q, k, stream=0)


def packed(order, batch, tokens, q_heads, k_heads, dim):
    """q and k of one projection, its buffer laid out in the given order."""
    h = q_heads + 2 * k_heads
    if order == "tokens, heads":
        x = mat(batch, tokens, h, dim)
    elif order == "heads, tokens":
        x = mat(batch, h, tokens, dim).transpose(1, 2)
    elif order == "tokens, q k v of each head":
        x = mat(batch, tokens, q_heads, 3, dim)
        return x[:, :, :, 0], x[:, :, :k_heads, 1]
    else:                                    # q, k, v of a sequence one after another
        x = mat(batch, 3, q_heads, tokens, dim).transpose(2, 3)
        return x[:, 0], x[:, 1, :, :k_heads]
    return x[:, :, :q_heads], x[:, :, q_heads:q_heads + k_heads]


@needs_no_gpu
@pytest.mark.parametrize("order", ["tokens, heads", "heads, tokens", "tokens, q k v of each head",
                                   "q k v, heads, tokens"])
@pytest.mark.parametrize("sizes", [(1, 5, 4, 2, 8), (2, 5, 4, 2, 8), (3, 1, 4, 4, 8),
                                   (2, 4096, 32, 8, 128), (7, 3, 1, 1, 2)], ids=str)
def test_packed_views_in_place_share_nothing(order, sizes):
    q, k = packed(order, *sizes)
    assert in_place(q, k) == "cuda"


@needs_no_gpu
def test_views_that_share_are_refused():
    q, k = packed("heads, tokens", 2, 5, 4, 2, 8)
    x = mat(2, 8, 5, 8).transpose(1, 2)
    assert in_place(x[:, :, :4], x[:, :, 3:5]) == "alias"
    assert in_place(x[:, :, ::2], x[:, :, 1::2]) == "cuda"
    assert in_place(x[:, :, ::2], x[:, :, 2:4]) == "alias"
    y = mat(2, 5, 4, 20)
    assert in_place(y[..., :8], y[..., 8:16]) == "cuda"
    assert in_place(y[..., :8], y[..., 7:15]) == "alias"


def starts(batch, tokens, heads, strides, first):
    return [first + b * strides[0] + t * strides[1] + h * strides[2]
            for b, t, h in itertools.product(range(batch), range(tokens), range(heads))]


@needs_no_gpu
def test_overlap_against_every_element():
    """Random views against the sets of their elements: an accepted pair shares none, and
    a refused one does (these are too small for the search to give up)."""
    rng = random.Random(5)
    seen = {"alias": 0, "cuda": 0}
    while min(seen.values()) < 300 or sum(seen.values()) < 2000:
        batch, tokens, dim = rng.randint(1, 3), rng.randint(1, 4), rng.choice([1, 2, 4])
        heads = rng.randint(1, 3), rng.randint(1, 3)
        views = []
        for h in heads:
            n = [batch, tokens, h]
            order = rng.sample(range(3), 3)
            strides, step = [0] * 3, dim * rng.randint(1, 4)
            for i in order:
                strides[i] = step
                step = step * n[i] + rng.choice([0, 0, dim, 3])
            views.append((h, strides))
        if rng.random() < 0.5:                # the same steps, as views of one buffer have
            views[1] = (heads[1], views[0][1])
        d = rng.randint(-40, 40)
        rows = [starts(batch, tokens, h, st, f) for (h, st), f in zip(views, (0, d))]
        try:
            q, k = ((batch, tokens, h, dim) for h in heads)
            st = [tuple(s) + (1,) for _, s in views]
            plan = eb.HeadsPlan("bfloat16", q, k, rotary_dim=0, q_strides=st[0], k_strides=st[1],
                                q_out_strides=st[0], k_out_strides=st[1])
        except eb.EbinError as e:             # an output that overlaps itself
            assert e.code == "invalid_arg"
            continue
        at = 1 << 40
        got = outcome(eb.execute_heads, plan, at, at + 2 * d, None, None, None, at, at + 2 * d,
                      stream=0)
        elements = [{r + j for r in rr for j in range(dim)} for rr in rows]
        assert got == ("alias" if elements[0] & elements[1] else "cuda"), (views, d, dim)
        seen[got] += 1


# ------------------------------------------------------------------ the current stream

def test_the_current_stream_without_torch_internals(monkeypatch):
    """The address comes from torch's public call where its parts are missing, take other
    arguments or disagree with it; and from the parts where they do not."""
    now = types.SimpleNamespace(cuda_stream=HANDLE)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: now)
    parts = {"_cuda_getDevice": lambda: 0, "_cuda_getCurrentRawStream": lambda d: HANDLE + d}
    for broken in (dict(_cuda_getDevice=None), dict(_cuda_getCurrentRawStream=None),
                   dict(_cuda_getCurrentRawStream=lambda: HANDLE),
                   dict(_cuda_getDevice=lambda: 1), dict()):
        for name, fn in {**parts, **broken}.items():
            if fn is None:
                monkeypatch.delattr(torch._C, name, raising=False)
            else:
                monkeypatch.setattr(torch._C, name, fn, raising=False)
        monkeypatch.setattr(eb, "_current", None)
        now.cuda_stream = HANDLE
        assert eb._stream(None) == HANDLE
        now.cuda_stream = HANDLE + 8
        assert eb._stream(None) == (HANDLE + 8 if broken else HANDLE)
    assert eb._stream(7) == 7 and eb._stream(now) == HANDLE + 8
