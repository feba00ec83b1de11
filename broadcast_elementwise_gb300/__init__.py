"""GB300-native ONNX broadcast binary elementwise engine: Python binding.

A thin ctypes binding of ``libebin.so``, whose C ABI (``include/ebin.h``) is
the product's boundary.  The ``ebin_*`` functions here have the C names and
only marshal arguments; every step of the path (descriptor checks, planning,
the plan cache, validation and the elementwise kernels) runs in the library.
PyTorch is used for device memory and streams only.

Importing this package loads the library and fails loudly if it is missing:
there is no CPU or eager fallback.

Typical use::

    import torch, broadcast_elementwise_gb300 as eb
    y = eb.binary("Add", x, b)                   # allocates y, runs on the current stream

    desc = eb.Descriptor("Mod", "float32", fmod=0, opset=28)
    plan = eb.Plan(desc, a.shape, b.shape)
    eb.execute(plan, a, b, out)

What a transformer layer needs around its attention::

    cos, sin = eb.rotary_table(8192, 128)
    qkv = eb.gemm(x, w, bias, trans_b=True)      # x [rows, k], w [n, k]
    q, k, v = qkv.view(batch, tokens, -1, 128).split([32, 8, 8], dim=2)
    eb.qk_norm_rotary(q, k, wq, wk, cos, sin, positions, out=(q, k))
"""
from __future__ import annotations

import ctypes
import os
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libebin.so")

OPS = {"Add": 0, "Sub": 1, "Mul": 2, "Div": 3, "Mod": 4, "Pow": 5,
       "Equal": 6, "Less": 7, "Greater": 8, "LessOrEqual": 9, "GreaterOrEqual": 10,
       "And": 11, "Or": 12, "Xor": 13,
       "BitwiseAnd": 14, "BitwiseOr": 15, "BitwiseXor": 16,
       "BitShift": 17, "PRelu": 18, "BatchNormalization": 19, "Clip": 20,
       "Max": 21, "Min": 22, "RSub": 23, "RDiv": 24, "BiasPRelu": 25, "MulAdd": 26,
       "BiasPReluBN": 27}
DTYPES = {"float32": 1, "uint8": 2, "int8": 3, "uint16": 4, "int16": 5, "int32": 6, "int64": 7,
          "bool": 9, "float16": 10, "float64": 11, "uint32": 12, "uint64": 13, "bfloat16": 16}
DTYPE_NAMES = {v: k for k, v in DTYPES.items()}
ITEMSIZE = {"float32": 4, "uint8": 1, "int32": 4, "int64": 8, "bool": 1, "float16": 2,
            "uint32": 4, "bfloat16": 2, "int8": 1, "int16": 2, "uint16": 2, "uint64": 8,
            "float64": 8}
FAMILIES = {"auto": -1, "empty": 0, "contiguous": 1, "left_scalar": 2, "right_scalar": 3,
            "repeated_block": 4, "inner_vector_outer": 5, "general_strided": 6}
FAMILY_NAMES = {v: k for k, v in FAMILIES.items()}
STATUS = {0: "ok", 1: "invalid_arg", 2: "unsupported_op", 3: "unsupported_type",
          4: "invalid_attr", 5: "incompatible_shapes", 6: "rank_too_large", 7: "alias",
          8: "cuda", 9: "family"}
DEVICE_DIV_BY_ZERO = 0x1
DEVICE_SHIFT_RANGE = 0x2
DEVICE_POSITION_RANGE = 0x4
DEVICE_WAIT_LIMIT = 0x8
NORMS = {"none": 0, "rms": 1}
LAYOUTS = {"half": 0, "interleaved": 1}
SCALINGS = {"none": 0, "linear": 1, "base": 2, "by_parts": 3}
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
MAX_RANK = 8
PLAN_CACHE_CAPACITY = 8


class EbinError(RuntimeError):
    """A non-OK status returned by the C ABI; ``.code`` holds its name."""

    def __init__(self, status: int, where: str):
        self.status = status
        self.code = STATUS.get(status, "unknown")
        super().__init__("%s: %s" % (where, self.code))


class ebin_attrs(ctypes.Structure):
    _fields_ = [("fmod", ctypes.c_int32), ("direction", ctypes.c_int32),
                ("epsilon", ctypes.c_float), ("clip_has_min", ctypes.c_int32),
                ("clip_has_max", ctypes.c_int32), ("with_scalar", ctypes.c_int32),
                ("scalar_b", ctypes.c_float)]


class ebin_rotary_attrs(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("trained_length", ctypes.c_double), ("slow_turns", ctypes.c_double),
                ("fast_turns", ctypes.c_double), ("amplitude", ctypes.c_double)]


class ebin_heads_view(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("token", ctypes.c_int64), ("head", ctypes.c_int64)]


class ebin_heads_attrs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("dtype_w", ctypes.c_int), ("norm", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("gradient", ctypes.c_int32),
                ("epsilon", ctypes.c_float), ("batch", ctypes.c_int64),
                ("tokens", ctypes.c_int64), ("q_heads", ctypes.c_int32),
                ("k_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("rotary_dim", ctypes.c_int32), ("position_type", ctypes.c_int32),
                ("position_strides", ctypes.c_int64 * 2), ("table_positions", ctypes.c_int64),
                ("q", ebin_heads_view), ("k", ebin_heads_view), ("dq", ebin_heads_view),
                ("dk", ebin_heads_view), ("q_out", ebin_heads_view),
                ("k_out", ebin_heads_view)]


class ebin_gemm_attrs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("dtype_bias", ctypes.c_int), ("trans_a", ctypes.c_int32),
                ("trans_b", ctypes.c_int32), ("activation", ctypes.c_int32),
                ("has_bias", ctypes.c_int32), ("has_residual", ctypes.c_int32),
                ("any_alignment", ctypes.c_int32), ("m", ctypes.c_int64), ("n", ctypes.c_int64),
                ("k", ctypes.c_int64), ("lda", ctypes.c_int64), ("ldb", ctypes.c_int64),
                ("ldy", ctypes.c_int64), ("ld_residual", ctypes.c_int64),
                ("ld_preact", ctypes.c_int64)]


class ebin_epilogue_grad_attrs(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("activation", ctypes.c_int32),
                ("has_bias", ctypes.c_int32), ("m", ctypes.c_int64), ("n", ctypes.c_int64),
                ("ld_dy", ctypes.c_int64), ("ld_z", ctypes.c_int64), ("ld_dz", ctypes.c_int64)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError("libebin.so is not built (%s); run __graft_entry__.build() or "
                          "python broadcast_elementwise_gb300/_build.py" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    p_i64 = ctypes.POINTER(ctypes.c_int64)
    sigs = {
        "ebin_descriptor_create": (i32, [i32, i32, ctypes.POINTER(ebin_attrs), i32, i32,
                                         ctypes.POINTER(vp)]),
        "ebin_descriptor_output_dtype": (i32, [vp, ctypes.POINTER(ctypes.c_int)]),
        "ebin_descriptor_id": (i32, [vp, ctypes.POINTER(ctypes.c_uint64)]),
        "ebin_descriptor_destroy": (None, [vp]),
        "ebin_plan_create": (i32, [vp, p_i64, i32, p_i64, i32, ctypes.POINTER(vp)]),
        "ebin_plan_create_forced": (i32, [vp, p_i64, i32, p_i64, i32, i32, ctypes.POINTER(vp)]),
        "ebin_plan_create3": (i32, [vp, p_i64, i32, p_i64, i32, p_i64, i32, ctypes.POINTER(vp)]),
        "ebin_plan_create_strided": (i32, [vp, p_i64, p_i64, i32, p_i64, p_i64, i32, i32,
                                           ctypes.POINTER(vp)]),
        "ebin_plan_create3_forced": (i32, [vp, p_i64, i32, p_i64, i32, p_i64, i32, i32,
                                           ctypes.POINTER(vp)]),
        "ebin_execute3": (i32, [vp, vp, vp, vp, vp, vp]),
        "ebin_plan_output_shape": (i32, [vp, p_i64, ctypes.POINTER(ctypes.c_int)]),
        "ebin_plan_numel": (i32, [vp, p_i64]),
        "ebin_plan_family": (i32, [vp, ctypes.POINTER(ctypes.c_int)]),
        "ebin_plan_geometry": (i32, [vp, ctypes.POINTER(ctypes.c_int), p_i64, p_i64, p_i64]),
        "ebin_plan_release": (None, [vp]),
        "ebin_plan_cache_stats": (i32, [ctypes.POINTER(ctypes.c_uint64),
                                        ctypes.POINTER(ctypes.c_uint64),
                                        ctypes.POINTER(ctypes.c_int)]),
        "ebin_plan_cache_clear": (None, []),
        "ebin_execute": (i32, [vp, vp, vp, vp, vp]),
        "ebin_execute_host": (i32, [vp, vp, vp, vp, vp, vp, vp, vp]),
        "ebin_execute_mapped": (i32, [vp, vp, vp, vp, vp]),
        "ebin_execute3_mapped": (i32, [vp, vp, vp, vp, vp, vp]),
        "ebin_get_device_status": (i32, [vp, ctypes.POINTER(ctypes.c_uint32)]),
        "ebin_execute_noalloc": (i32, [vp, vp, vp, vp, vp, i32, ctypes.POINTER(ctypes.c_uint32)]),
        "ebin_noalloc_read_status": (i32, [i32, vp, ctypes.POINTER(ctypes.c_uint32)]),
        "ebin_rotary_table": (i32, [ctypes.POINTER(ebin_rotary_attrs), i64, i64, vp, vp, vp]),
        "ebin_heads_plan_create": (i32, [ctypes.POINTER(ebin_heads_attrs), ctypes.POINTER(vp)]),
        "ebin_heads_plan_workspace": (i32, [vp, ctypes.POINTER(ctypes.c_size_t)]),
        "ebin_heads_plan_release": (None, [vp]),
        "ebin_heads_execute": (i32, [vp] * 11),
        "ebin_heads_grad_execute": (i32, [vp] * 15 + [ctypes.c_size_t, vp]),
        "ebin_gemm_plan_create": (i32, [ctypes.POINTER(ebin_gemm_attrs), ctypes.POINTER(vp)]),
        "ebin_gemm_plan_workspace": (i32, [vp, ctypes.POINTER(ctypes.c_size_t)]),
        "ebin_gemm_plan_release": (None, [vp]),
        "ebin_gemm_execute": (i32, [vp] * 8 + [ctypes.c_size_t, vp]),
        "ebin_epilogue_grad_plan_create": (i32, [ctypes.POINTER(ebin_epilogue_grad_attrs),
                                                 ctypes.POINTER(vp)]),
        "ebin_epilogue_grad_plan_workspace": (i32, [vp, ctypes.POINTER(ctypes.c_size_t)]),
        "ebin_epilogue_grad_plan_release": (None, [vp]),
        "ebin_epilogue_grad_execute": (i32, [vp] * 6 + [ctypes.c_size_t, vp]),
        "ebin_launch_count": (ctypes.c_uint64, []),
        "ebin_dtype_size": (ctypes.c_size_t, [i32]),
        "ebin_status_string": (ctypes.c_char_p, [i32]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


def _check(status: int, where: str):
    if status != 0:
        raise EbinError(status, where)


def _shape(shape):
    dims = [int(d) for d in shape]
    arr = (ctypes.c_int64 * max(1, len(dims)))(*dims)
    return arr, len(dims)


def _ptr(x) -> int | None:
    """Device address of a tensor (or an int address, or None)."""
    if x is None or isinstance(x, int):
        return x
    return x.data_ptr()


_current = None     # () -> the address of torch's current stream


def _ptrs(*xs):
    """_ptr of each argument, in one call (a launch-bound path passes many)."""
    return [x if x is None or isinstance(x, int) else x.data_ptr() for x in xs]


def _current_stream():
    """A function that gives the address of torch.cuda.current_stream(): by torch's own
    parts of that call, without its Stream object (3.0 -> 0.2 us), where this version
    has them and they agree with it, else by the call itself."""
    import torch
    now = torch.cuda.current_stream().cuda_stream     # initialises CUDA, or says why it cannot
    try:
        device, raw = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        if raw(device()) == now:
            return lambda: raw(device())
    except (AttributeError, TypeError):
        pass
    return lambda: torch.cuda.current_stream().cuda_stream


def _stream(stream) -> int | None:
    if stream is None:
        global _current
        if _current is None:
            _current = _current_stream()
        return _current()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ----------------------------------------------------------------- the C ABI, by name

def ebin_descriptor_create(op, opset, attrs, dtype_a, dtype_b) -> int:
    out = ctypes.c_void_p()
    _check(lib.ebin_descriptor_create(op, opset, ctypes.byref(attrs) if attrs else None,
                                      dtype_a, dtype_b, ctypes.byref(out)),
           "ebin_descriptor_create")
    return out.value


def ebin_descriptor_output_dtype(desc) -> int:
    v = ctypes.c_int()
    _check(lib.ebin_descriptor_output_dtype(desc, ctypes.byref(v)), "ebin_descriptor_output_dtype")
    return v.value


def ebin_descriptor_id(desc) -> int:
    v = ctypes.c_uint64()
    _check(lib.ebin_descriptor_id(desc, ctypes.byref(v)), "ebin_descriptor_id")
    return v.value


def ebin_descriptor_destroy(desc) -> None:
    lib.ebin_descriptor_destroy(desc)


def ebin_plan_create(desc, shape_a, shape_b) -> int:
    sa, ra = _shape(shape_a)
    sb, rb = _shape(shape_b)
    out = ctypes.c_void_p()
    _check(lib.ebin_plan_create(desc, sa, ra, sb, rb, ctypes.byref(out)), "ebin_plan_create")
    return out.value


def ebin_plan_create_forced(desc, shape_a, shape_b, family) -> int:
    sa, ra = _shape(shape_a)
    sb, rb = _shape(shape_b)
    out = ctypes.c_void_p()
    _check(lib.ebin_plan_create_forced(desc, sa, ra, sb, rb, family, ctypes.byref(out)),
           "ebin_plan_create_forced")
    return out.value


def ebin_plan_create_strided(desc, shape_a, strides_a, shape_b, strides_b, family=-1) -> int:
    """Marshal ebin_plan_create_strided (strides None = dense)."""
    sa, ra = _shape(shape_a)
    sb, rb = _shape(shape_b)
    ta = _shape(strides_a)[0] if strides_a is not None else None
    tb = _shape(strides_b)[0] if strides_b is not None else None
    out = ctypes.c_void_p()
    _check(lib.ebin_plan_create_strided(desc, sa, ta, ra, sb, tb, rb, family, ctypes.byref(out)),
           "ebin_plan_create_strided")
    return out.value


def ebin_plan_create3(desc, shape_a, shape_b, shape_c, family=None) -> int:
    """Marshal ebin_plan_create3 (family None) or ebin_plan_create3_forced."""
    sa, ra = _shape(shape_a)
    sb, rb = _shape(shape_b)
    sc, rc = _shape(shape_c)
    out = ctypes.c_void_p()
    if family is None:
        _check(lib.ebin_plan_create3(desc, sa, ra, sb, rb, sc, rc, ctypes.byref(out)),
               "ebin_plan_create3")
    else:
        _check(lib.ebin_plan_create3_forced(desc, sa, ra, sb, rb, sc, rc, family,
                                            ctypes.byref(out)), "ebin_plan_create3_forced")
    return out.value


def ebin_plan_output_shape(plan) -> tuple:
    shape = (ctypes.c_int64 * MAX_RANK)()
    rank = ctypes.c_int()
    _check(lib.ebin_plan_output_shape(plan, shape, ctypes.byref(rank)), "ebin_plan_output_shape")
    return tuple(shape[i] for i in range(rank.value))


def ebin_plan_numel(plan) -> int:
    v = ctypes.c_int64()
    _check(lib.ebin_plan_numel(plan, ctypes.byref(v)), "ebin_plan_numel")
    return v.value


def ebin_plan_family(plan) -> int:
    v = ctypes.c_int()
    _check(lib.ebin_plan_family(plan, ctypes.byref(v)), "ebin_plan_family")
    return v.value


def ebin_plan_geometry(plan):
    rank = ctypes.c_int()
    n, sa, sb = ((ctypes.c_int64 * MAX_RANK)() for _ in range(3))
    _check(lib.ebin_plan_geometry(plan, ctypes.byref(rank), n, sa, sb), "ebin_plan_geometry")
    r = rank.value
    return [n[i] for i in range(r)], [sa[i] for i in range(r)], [sb[i] for i in range(r)]


def ebin_plan_release(plan) -> None:
    lib.ebin_plan_release(plan)


def ebin_plan_cache_stats():
    h, m, s = ctypes.c_uint64(), ctypes.c_uint64(), ctypes.c_int()
    _check(lib.ebin_plan_cache_stats(ctypes.byref(h), ctypes.byref(m), ctypes.byref(s)),
           "ebin_plan_cache_stats")
    return h.value, m.value, s.value


def ebin_plan_cache_clear() -> None:
    lib.ebin_plan_cache_clear()


def ebin_execute(plan, A, B, out, stream) -> None:
    _check(lib.ebin_execute(plan, A, B, out, stream), "ebin_execute")


def ebin_execute3(plan, A, B, C, out, stream) -> None:
    _check(lib.ebin_execute3(plan, A, B, C, out, stream), "ebin_execute3")


def ebin_execute_host(plan, host_a, host_b, host_out, dev_a, dev_b, dev_out, stream) -> None:
    _check(lib.ebin_execute_host(plan, host_a, host_b, host_out, dev_a, dev_b, dev_out, stream),
           "ebin_execute_host")


def ebin_execute_mapped(plan, host_a, host_b, host_out, stream) -> None:
    _check(lib.ebin_execute_mapped(plan, host_a, host_b, host_out, stream), "ebin_execute_mapped")


def ebin_execute3_mapped(plan, host_a, host_b, host_c, host_out, stream) -> None:
    _check(lib.ebin_execute3_mapped(plan, host_a, host_b, host_c, host_out, stream),
           "ebin_execute3_mapped")


def ebin_execute_noalloc(plan, A, B, out, stream, status_slot, want_status=True):
    """Marshal ebin_execute_noalloc; returns the status bits (0 when not requested)."""
    bits = ctypes.c_uint32(0)
    _check(lib.ebin_execute_noalloc(plan, A, B, out, stream, int(status_slot),
                                    ctypes.byref(bits) if want_status else None),
           "ebin_execute_noalloc")
    return bits.value


NOALLOC_STATUS_SLOTS = 64


def ebin_noalloc_read_status(status_slot, stream) -> int:
    """Marshal ebin_noalloc_read_status; returns the slot's status bits."""
    v = ctypes.c_uint32(0)
    _check(lib.ebin_noalloc_read_status(int(status_slot), stream, ctypes.byref(v)),
           "ebin_noalloc_read_status")
    return v.value


def ebin_get_device_status(stream) -> int:
    v = ctypes.c_uint32()
    _check(lib.ebin_get_device_status(stream, ctypes.byref(v)), "ebin_get_device_status")
    return v.value


def ebin_rotary_table(attrs, first_position, positions, cos, sin, stream) -> None:
    _check(lib.ebin_rotary_table(ctypes.byref(attrs), int(first_position), int(positions), cos,
                                 sin, stream), "ebin_rotary_table")


def ebin_heads_plan_create(attrs) -> int:
    out = ctypes.c_void_p()
    _check(lib.ebin_heads_plan_create(ctypes.byref(attrs), ctypes.byref(out)),
           "ebin_heads_plan_create")
    return out.value


def ebin_heads_plan_workspace(plan) -> int:
    v = ctypes.c_size_t()
    _check(lib.ebin_heads_plan_workspace(plan, ctypes.byref(v)), "ebin_heads_plan_workspace")
    return v.value


def ebin_heads_plan_release(plan) -> None:
    lib.ebin_heads_plan_release(plan)


def ebin_heads_execute(plan, q, k, cos, sin, positions, wq, wk, q_out, k_out, stream) -> None:
    st = lib.ebin_heads_execute(plan, q, k, cos, sin, positions, wq, wk, q_out, k_out, stream)
    if st:
        raise EbinError(st, "ebin_heads_execute")


def ebin_heads_grad_execute(plan, dq, dk, q, k, cos, sin, positions, wq, wk, dq_out, dk_out, dwq,
                            dwk, workspace, workspace_bytes, stream) -> None:
    st = lib.ebin_heads_grad_execute(plan, dq, dk, q, k, cos, sin, positions, wq, wk, dq_out,
                                     dk_out, dwq, dwk, workspace, workspace_bytes, stream)
    if st:
        raise EbinError(st, "ebin_heads_grad_execute")


def ebin_gemm_plan_create(attrs) -> int:
    out = ctypes.c_void_p()
    _check(lib.ebin_gemm_plan_create(ctypes.byref(attrs), ctypes.byref(out)),
           "ebin_gemm_plan_create")
    return out.value


def ebin_gemm_plan_workspace(plan) -> int:
    v = ctypes.c_size_t()
    _check(lib.ebin_gemm_plan_workspace(plan, ctypes.byref(v)), "ebin_gemm_plan_workspace")
    return v.value


def ebin_gemm_plan_release(plan) -> None:
    lib.ebin_gemm_plan_release(plan)


def ebin_gemm_execute(plan, A, B, bias, residual, Y, preact, workspace, workspace_bytes,
                      stream) -> None:
    st = lib.ebin_gemm_execute(plan, A, B, bias, residual, Y, preact, workspace, workspace_bytes,
                               stream)
    if st:
        raise EbinError(st, "ebin_gemm_execute")


def ebin_epilogue_grad_plan_create(attrs) -> int:
    out = ctypes.c_void_p()
    _check(lib.ebin_epilogue_grad_plan_create(ctypes.byref(attrs), ctypes.byref(out)),
           "ebin_epilogue_grad_plan_create")
    return out.value


def ebin_epilogue_grad_plan_workspace(plan) -> int:
    v = ctypes.c_size_t()
    _check(lib.ebin_epilogue_grad_plan_workspace(plan, ctypes.byref(v)),
           "ebin_epilogue_grad_plan_workspace")
    return v.value


def ebin_epilogue_grad_plan_release(plan) -> None:
    lib.ebin_epilogue_grad_plan_release(plan)


def ebin_epilogue_grad_execute(plan, dy, z, dz, dbias, workspace, workspace_bytes, stream) -> None:
    st = lib.ebin_epilogue_grad_execute(plan, dy, z, dz, dbias, workspace, workspace_bytes, stream)
    if st:
        raise EbinError(st, "ebin_epilogue_grad_execute")


def ebin_launch_count() -> int:
    return int(lib.ebin_launch_count())


def ebin_dtype_size(dtype) -> int:
    return int(lib.ebin_dtype_size(dtype))


def ebin_status_string(status) -> str:
    return lib.ebin_status_string(status).decode()


# ----------------------------------------------------------------- thin object wrappers

def _dtype_code(dtype) -> int:
    if isinstance(dtype, int):
        return dtype
    if isinstance(dtype, str):
        return DTYPES[dtype]
    return DTYPES[torch_dtype_name(dtype)]


def torch_dtype_name(t) -> str:
    import torch
    table = {torch.float32: "float32", torch.float16: "float16", torch.bfloat16: "bfloat16",
             torch.int32: "int32", torch.int64: "int64", torch.uint8: "uint8",
             torch.bool: "bool", torch.uint32: "uint32", torch.int8: "int8",
             torch.int16: "int16", torch.uint16: "uint16", torch.uint64: "uint64",
             torch.float64: "float64"}
    return table[t]


def torch_dtype(name: str):
    import torch
    return {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16,
            "int32": torch.int32, "int64": torch.int64, "uint8": torch.uint8,
            "bool": torch.bool, "uint32": torch.uint32, "int8": torch.int8,
            "int16": torch.int16, "uint16": torch.uint16, "uint64": torch.uint64,
            "float64": torch.float64}[name]


class Descriptor:
    """Owns an ebin descriptor (operator, opset, attributes, element type)."""

    def __init__(self, op: str, dtype, *, opset: int = 28, fmod: int = 0, direction: int = 0,
                 epsilon: float = 1e-5, has_min: bool = True, has_max: bool = True,
                 scalar_b: float | None = None, dtype_b=None):
        """``scalar_b`` given: ncnn binaryop's with_scalar, B is that value.
        ``dtype_b``: B's type where it may differ from A's (Pow's exponent;
        a float32 parameter block of BatchNormalization, BiasPRelu or
        BiasPReluBN beside float16, bfloat16 or float64 x)."""
        self.op = op
        self.dtype = DTYPE_NAMES[_dtype_code(dtype)]
        self.dtype_b = self.dtype if dtype_b is None else DTYPE_NAMES[_dtype_code(dtype_b)]
        self.with_scalar = scalar_b is not None
        attrs = ebin_attrs(int(fmod), int(direction), float(epsilon), int(bool(has_min)),
                           int(bool(has_max)), int(self.with_scalar),
                           float(scalar_b) if self.with_scalar else 0.0)
        code = _dtype_code(dtype)
        code_b = code if dtype_b is None else _dtype_code(dtype_b)
        self.handle = ebin_descriptor_create(OPS[op], int(opset), attrs, code, code_b)
        self.out_dtype = DTYPE_NAMES[ebin_descriptor_output_dtype(self.handle)]
        self.id = ebin_descriptor_id(self.handle)

    def close(self):
        if self.handle:
            ebin_descriptor_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Plan:
    """Holds one plan reference for (descriptor, shape_a, shape_b)."""

    def __init__(self, desc: Descriptor, shape_a, shape_b, family: str | None = None,
                 strides_a=None, strides_b=None):
        """strides_a / strides_b: element strides of strided input views (None = dense)."""
        self.desc = desc
        self.shape_a = tuple(int(d) for d in shape_a)
        self.shape_b = tuple(int(d) for d in shape_b)
        if strides_a is not None or strides_b is not None:
            self.handle = ebin_plan_create_strided(
                desc.handle, self.shape_a, strides_a, self.shape_b, strides_b,
                -1 if family is None else FAMILIES[family])
        elif family is None:
            self.handle = ebin_plan_create(desc.handle, self.shape_a, self.shape_b)
        else:
            self.handle = ebin_plan_create_forced(desc.handle, self.shape_a, self.shape_b,
                                                  FAMILIES[family])
        self.output_shape = ebin_plan_output_shape(self.handle)
        self.numel = ebin_plan_numel(self.handle)
        self.family = FAMILY_NAMES[ebin_plan_family(self.handle)]

    def geometry(self):
        return ebin_plan_geometry(self.handle)

    def close(self):
        if self.handle:
            ebin_plan_release(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Plan3(Plan):
    """Holds one three-input plan reference (MulAdd) for (descriptor, shapes A, B, C)."""

    def __init__(self, desc: Descriptor, shape_a, shape_b, shape_c, family: str | None = None):
        self.desc = desc
        self.shape_a = tuple(int(d) for d in shape_a)
        self.shape_b = tuple(int(d) for d in shape_b)
        self.shape_c = tuple(int(d) for d in shape_c)
        self.handle = ebin_plan_create3(desc.handle, self.shape_a, self.shape_b, self.shape_c,
                                        None if family is None else FAMILIES[family])
        self.output_shape = ebin_plan_output_shape(self.handle)
        self.numel = ebin_plan_numel(self.handle)
        self.family = FAMILY_NAMES[ebin_plan_family(self.handle)]


def execute3(plan: Plan3, A, B, C, out, stream=None) -> None:
    """Enqueue a three-input plan on device buffers (torch tensors or int addresses)."""
    ebin_execute3(plan.handle, _ptr(A), _ptr(B), _ptr(C), _ptr(out), _stream(stream))


def execute(plan: Plan, A, B, out, stream=None) -> None:
    """Enqueue the plan on device buffers (torch tensors or int addresses)."""
    ebin_execute(plan.handle, _ptr(A), _ptr(B), _ptr(out), _stream(stream))


def execute_mapped(plan: Plan, A, B, out, stream=None) -> None:
    """Enqueue the plan on pinned host buffers, read and written in place by the
    kernel (torch pinned tensors or int addresses)."""
    ebin_execute_mapped(plan.handle, _ptr(A), _ptr(B), _ptr(out), _stream(stream))


def execute3_mapped(plan: Plan3, A, B, C, out, stream=None) -> None:
    """Enqueue a three-input plan on pinned host buffers, in place."""
    ebin_execute3_mapped(plan.handle, _ptr(A), _ptr(B), _ptr(C), _ptr(out), _stream(stream))


def get_device_status(stream=None) -> int:
    return ebin_get_device_status(_stream(stream))


_descriptors: dict = {}


def _attr_key(v):
    """Cache key of an attribute value: floats by bit pattern (-0.0 is not 0.0,
    and a NaN matches itself)."""
    return ("f", struct.pack("<d", v)) if isinstance(v, float) else v


def descriptor(op: str, dtype, **attrs) -> Descriptor:
    """A process-wide Descriptor per (op, dtype, attributes), so plans stay cached."""
    key = (op, _dtype_code(dtype), tuple(sorted((k, _attr_key(v)) for k, v in attrs.items())))
    d = _descriptors.get(key)
    if d is None:
        d = _descriptors[key] = Descriptor(op, dtype, **attrs)
    return d


def _launching(device, stream):
    """The context of a one-call form: its device and, with ``stream``, that stream as
    torch's current one.  What torch allocates inside then belongs to the stream
    that uses it: a workspace dropped at return is handed out again in that
    stream's order, and no block is taken over that another stream still uses."""
    import torch
    if stream is None:
        return torch.cuda.device(device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_stream(stream), device)
    elif device.index not in (None, stream.device.index):
        raise ValueError("the tensors are on %s and the stream on %s" % (device, stream.device))
    return torch.cuda.stream(stream)


def binary(op: str, a, b, out=None, *, stream=None, **attrs):
    """One-shot call: returns ``out`` (allocated if None).

    On torch CUDA tensors, inputs that are not contiguous run as strided views
    (no copy), except a BatchNormalization / Clip / BiasPRelu / BiasPReluBN
    parameter block, which is copied.  On pinned CPU tensors (contiguous),
    the kernel reads and writes host memory in place (ebin_execute_mapped;
    ``out`` is allocated pinned); synchronise ``stream`` before reading it.
    With ``stream`` what the call allocates on the device is that stream's memory.
    """
    if (b is not None and op in ("BatchNormalization", "BiasPRelu", "BiasPReluBN")
            and b.dtype != a.dtype and "dtype_b" not in attrs):
        attrs["dtype_b"] = b.dtype      # a float32 parameter block beside 16-bit or float64 x
    desc = descriptor(op, a.dtype, **attrs)
    plain_b = op not in ("BatchNormalization", "Clip", "BiasPRelu", "BiasPReluBN")
    if b is not None and b.dtype != torch_dtype(desc.dtype_b):
        raise ValueError("binary: B is %s; %s on %s takes B of %s"
                         % (b.dtype, op, desc.dtype, desc.dtype_b))
    if not a.is_cuda:
        if not a.is_pinned() or (b is not None and not b.is_pinned()):
            raise ValueError("binary: CPU tensors must be pinned (tensor.pin_memory())")
        if not a.is_contiguous() or (b is not None and not b.is_contiguous()):
            raise ValueError("binary: pinned CPU tensors must be contiguous")
        plan = Plan(desc, a.shape, b.shape if b is not None else (2,))
        out = _output(out, plan, desc, None)
        execute_mapped(plan, a, b, out, stream)
        return out
    if b is not None and b.device != a.device:
        raise ValueError("binary: A is on %s and B on %s" % (a.device, b.device))
    with _launching(a.device, stream):
        if b is not None and not plain_b:
            b = b.contiguous()
        ta = None if a.is_contiguous() else tuple(a.stride())
        tb = None if (b is None or b.is_contiguous()) else tuple(b.stride())
        plan = Plan(desc, a.shape, b.shape if b is not None else (2,), strides_a=ta, strides_b=tb)
        out = _output(out, plan, desc, a.device)
        execute(plan, a, b, out, stream)
    return out


def _output(out, plan, desc, device):
    """The output tensor of binary(): allocated when None (pinned host memory
    when device is None), else checked to be what the kernel writes: the
    output's type and shape, contiguous, on that device (or pinned)."""
    import torch
    want = torch_dtype(desc.out_dtype)
    if out is None:
        if device is None:
            return torch.empty(plan.output_shape, dtype=want).pin_memory()
        return torch.empty(plan.output_shape, dtype=want, device=device)
    if out.dtype != want or tuple(out.shape) != tuple(plan.output_shape):
        raise ValueError("binary: out is %s %s; the result is %s %s"
                         % (out.dtype, tuple(out.shape), desc.out_dtype, tuple(plan.output_shape)))
    if not out.is_contiguous():
        raise ValueError("binary: out must be contiguous")
    if device is None and (out.is_cuda or not out.is_pinned()):
        raise ValueError("binary: out must be a pinned CPU tensor, as the inputs are")
    if device is not None and out.device != device:
        raise ValueError("binary: A is on %s and out on %s" % (device, out.device))
    return out


# ----------------------------------------------------------------- heads: rotary positions, norms
#
# In the one-call forms below ``stream=s`` does what calling them under
# torch.cuda.stream(s) does: the inputs are ready in s's order, and what the call
# allocates, its results among it, is s's memory.

def rotary_table(positions: int, rotary_dim: int, *, base: float = 10000.0,
                 scaling: str = "none", factor: float = 1.0, trained_length: float = 0.0,
                 slow_turns: float = 1.0, fast_turns: float = 32.0, amplitude: float = 1.0,
                 first_position: int = 0, device="cuda", stream=None):
    """(cos, sin), float32 [positions, rotary_dim / 2], formed in binary64 on the
    device.  scaling, for contexts longer than the trained one: "linear" divides
    every frequency by factor, "base" stretches the base, "by_parts" divides
    what turns fewer than slow_turns times within trained_length, keeps what
    turns more than fast_turns times and blends between."""
    import torch
    attrs = ebin_rotary_attrs(int(rotary_dim), SCALINGS[scaling], float(base), float(factor),
                              float(trained_length), float(slow_turns), float(fast_turns),
                              float(amplitude))
    with _launching(torch.device(device), stream):
        cos = torch.empty(int(positions), int(rotary_dim) // 2, device="cuda")
        sin = torch.empty_like(cos)
        ebin_rotary_table(attrs, first_position, positions, _ptr(cos), _ptr(sin), _stream(stream))
    return cos, sin


def _heads_view(shape, strides, what):
    """The (batch, token, head) strides of a [batch, tokens, heads, head_dim] view."""
    if strides is None:
        n = [int(d) for d in shape]
        return ebin_heads_view(n[1] * n[2] * n[3], n[2] * n[3], n[3])
    st = [int(v) for v in strides]
    if len(st) != 4 or (st[3] != 1 and int(shape[3]) > 1):
        raise ValueError("%s: the last dimension of a heads view is dense (strides %s)"
                         % (what, tuple(st)))
    return ebin_heads_view(st[0], st[1], st[2])


class HeadsPlan:
    """A plan of the operators on heads: rotary positions (norm "none") or the
    RMS norm of each head and the rotation (norm "rms"), forward or gradient.

    Shapes are [batch, tokens, heads, head_dim]; strides (None = dense) are the
    views' element strides, as ``tensor.stride()`` gives them.  ``k_shape`` None
    leaves k out.  ``positions``: None (token t is at position t), torch.int32
    or torch.int64: the type of a [batch, tokens] tensor of positions, its
    element strides ``position_strides``.  ``rotary_dim`` None rotates whole heads;
    a rotation needs ``table_positions``, the rows of its tables.  Run with
    execute_heads, or, for norm "rms" with gradient=True, execute_heads_grad.
    """

    def __init__(self, dtype, q_shape, k_shape=None, *, norm: str = "none", epsilon: float = 1e-6,
                 weight_dtype=None, layout: str = "half", rotary_dim: int | None = None,
                 gradient: bool = False, positions=None, position_strides=None,
                 table_positions: int | None = None, q_strides=None, k_strides=None, dq_strides=None,
                 dk_strides=None, q_out_strides=None, k_out_strides=None):
        q_shape = tuple(int(d) for d in q_shape)
        k_shape = (q_shape[0], q_shape[1], 0, q_shape[3]) if k_shape is None else \
            tuple(int(d) for d in k_shape)
        if len(q_shape) != 4 or len(k_shape) != 4:
            raise ValueError("HeadsPlan: shapes are [batch, tokens, heads, head_dim]")
        if (q_shape[0], q_shape[1], q_shape[3]) != (k_shape[0], k_shape[1], k_shape[3]):
            raise ValueError("HeadsPlan: q is %s and k %s; they differ in heads only"
                             % (q_shape, k_shape))
        code = _dtype_code(dtype)
        a = ebin_heads_attrs()
        a.dtype = code
        a.dtype_w = code if weight_dtype is None else _dtype_code(weight_dtype)
        a.norm, a.layout = NORMS[norm], LAYOUTS[layout]
        a.gradient, a.epsilon = int(bool(gradient)), float(epsilon)
        a.batch, a.tokens, a.q_heads, a.head_dim = q_shape
        a.k_heads = k_shape[2]
        a.rotary_dim = q_shape[3] if rotary_dim is None else int(rotary_dim)
        if a.rotary_dim > 0 and table_positions is None:
            raise ValueError("HeadsPlan: a rotation of %d elements needs table_positions "
                             "(rotary_dim=0: no rotation)" % a.rotary_dim)
        a.position_type = 0 if positions is None else _dtype_code(positions)
        ps = (q_shape[1], 1) if position_strides is None else position_strides
        a.position_strides = (ctypes.c_int64 * 2)(int(ps[0]), int(ps[1]))
        a.table_positions = int(table_positions or 0)
        for name, shape, st in (("q", q_shape, q_strides), ("k", k_shape, k_strides),
                                ("dq", q_shape, dq_strides), ("dk", k_shape, dk_strides),
                                ("q_out", q_shape, q_out_strides),
                                ("k_out", k_shape, k_out_strides)):
            setattr(a, name, _heads_view(shape, st, name))
        self.q_shape, self.k_shape = q_shape, k_shape
        self.handle = ebin_heads_plan_create(a)
        self.workspace_bytes = ebin_heads_plan_workspace(self.handle)

    def close(self):
        if self.handle:
            ebin_heads_plan_release(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def execute_heads(plan: HeadsPlan, q, k, cos, sin, positions, q_out, k_out, wq=None, wk=None,
                  stream=None) -> None:
    """Enqueue a rotation (either direction) or a norm with rotation on device
    buffers laid out as the plan says (torch tensors or int addresses)."""
    st = lib.ebin_heads_execute(plan.handle, *_ptrs(q, k, cos, sin, positions, wq, wk, q_out,
                                                    k_out), _stream(stream))
    if st:
        raise EbinError(st, "ebin_heads_execute")


def execute_heads_grad(plan: HeadsPlan, dq, dk, q, k, cos, sin, positions, wq, wk, dq_out, dk_out,
                       dwq, dwk, workspace, stream=None) -> None:
    """Enqueue the gradient of norm and rotation; ``workspace``: a uint8 device
    tensor of at least plan.workspace_bytes."""
    ebin_heads_grad_execute(plan.handle, *_ptrs(dq, dk, q, k, cos, sin, positions, wq, wk, dq_out,
                                                dk_out, dwq, dwk, workspace),
                            _bytes_of(workspace), _stream(stream))


def _bytes_of(t) -> int:
    return 0 if t is None else t.nbytes


def _same_device(where, first, *others):
    """ValueError unless every tensor (None is passed over) is on the first one's CUDA device."""
    if not first.is_cuda:
        raise ValueError("%s: tensors must be on a CUDA device" % where)
    for t in others:
        if t is not None and t.device != first.device:
            raise ValueError("%s: tensors are on %s and %s" % (where, first.device, t.device))


def _heads_inputs(where, q, k, cos, sin, positions):
    """The checks of the one-shot calls; returns the plan's keywords for the table and positions."""
    import torch
    _same_device(where, q, k, cos, sin, positions)
    if q.dim() != 4 or (k is not None and k.dim() != 4):
        raise ValueError("%s: q and k are [batch, tokens, heads, head_dim]" % where)
    if k is not None and k.dtype != q.dtype:
        raise ValueError("%s: q is %s and k %s" % (where, q.dtype, k.dtype))
    kw = {"rotary_dim": 0}
    if cos is not None or sin is not None:
        if cos is None or sin is None or cos.dim() != 2 or cos.shape != sin.shape:
            raise ValueError("%s: cos and sin are two [positions, rotary_dim / 2] tables" % where)
        for t in (cos, sin):
            if t.dtype != torch.float32 or not t.is_contiguous():
                raise ValueError("%s: cos and sin are contiguous float32" % where)
        kw = {"rotary_dim": 2 * cos.shape[1], "table_positions": cos.shape[0]}
    if positions is not None:
        if positions.dim() == 1:
            positions = positions.expand(q.shape[0], -1)
        if tuple(positions.shape) != tuple(q.shape[:2]) or \
                positions.dtype not in (torch.int32, torch.int64):
            raise ValueError("%s: positions are int32 or int64 [tokens] or [batch, tokens]" % where)
        kw.update(positions=positions.dtype, position_strides=positions.stride())
    return kw, positions


def _heads_out(where, x, out):
    import torch
    if x is None:
        return None
    if out is None:
        return torch.empty(x.shape, dtype=x.dtype, device=x.device)
    if out.dtype != x.dtype or out.shape != x.shape or out.device != x.device:
        raise ValueError("%s: an output is %s %s on %s; the result is %s %s on %s"
                         % (where, out.dtype, tuple(out.shape), out.device, x.dtype,
                            tuple(x.shape), x.device))
    return out


def _run_heads(where, q, k, cos, sin, positions, out, wq, wk, stream, **kw):
    more, positions = _heads_inputs(where, q, k, cos, sin, positions)
    _same_device(where, q, wq, wk)
    qo, ko = (None, None) if out is None else out
    with _launching(q.device, stream):
        qo, ko = _heads_out(where, q, qo), _heads_out(where, k, ko)
        plan = HeadsPlan(q.dtype, q.shape, None if k is None else k.shape, q_strides=q.stride(),
                         k_strides=None if k is None else k.stride(), q_out_strides=qo.stride(),
                         k_out_strides=None if k is None else ko.stride(), **more, **kw)
        execute_heads(plan, q, k, cos, sin, positions, qo, ko, wq, wk, stream)
    return qo, ko


def rotary(q, k, cos, sin, positions=None, *, layout: str = "half", gradient: bool = False,
           out=None, stream=None):
    """Rotary positions of q and k (either may be a strided view; k may be None):
    returns (q_out, k_out), new tensors or ``out``, which may be (q, k) itself.
    ``gradient``: q and k are the incoming gradients, rotated back."""
    return _run_heads("rotary", q, k, cos, sin, positions, out, None, None, stream,
                      layout=layout, gradient=gradient)


def _norm_weights(where, q, wq, wk):
    """The common type of the norm weights (None where there is none)."""
    kinds = {w.dtype for w in (wq, wk) if w is not None}
    for w in (wq, wk):
        if w is not None and (tuple(w.shape) != (q.shape[-1],) or not w.is_contiguous()):
            raise ValueError("%s: a norm weight is a contiguous [head_dim] tensor" % where)
    if len(kinds) > 1:
        raise ValueError("%s: wq and wk have one type" % where)
    return kinds.pop() if kinds else None


def qk_norm_rotary(q, k, wq, wk, cos=None, sin=None, positions=None, *, epsilon: float = 1e-6,
                   layout: str = "half", out=None, stream=None):
    """The RMS norm of each head of q and k, times its weight (None = 1), and
    the rotation (cos None = norm only) in one pass; returns (q_out, k_out)."""
    wd = _norm_weights("qk_norm_rotary", q, wq, wk)
    return _run_heads("qk_norm_rotary", q, k, cos, sin, positions, out, wq, wk, stream,
                      norm="rms", epsilon=epsilon, layout=layout, weight_dtype=wd)


def qk_norm_rotary_grad(dq, dk, q, k, wq, wk, cos=None, sin=None, positions=None, *,
                        epsilon: float = 1e-6, layout: str = "half", out=None, stream=None):
    """The gradient of qk_norm_rotary: (dq, dk, dwq, dwk) for the incoming
    gradients dq, dk and the forward inputs q, k; dwq and dwk are float32
    (dk and dwk None without k)."""
    import torch
    where = "qk_norm_rotary_grad"
    wd = _norm_weights(where, q, wq, wk)
    more, positions = _heads_inputs(where, q, k, cos, sin, positions)
    _same_device(where, q, dq, dk, wq, wk)
    for g, x in ((dq, q), (dk, k)):
        if (g is None) != (x is None) or (g is not None and
                                          (g.shape != x.shape or g.dtype != x.dtype)):
            raise ValueError("%s: a gradient has its input's shape and type" % where)
    qo, ko = (None, None) if out is None else out
    st = (lambda t: None if t is None else t.stride())
    with _launching(q.device, stream):
        qo, ko = _heads_out(where, q, qo), _heads_out(where, k, ko)
        plan = HeadsPlan(q.dtype, q.shape, None if k is None else k.shape, norm="rms",
                         epsilon=epsilon, layout=layout, weight_dtype=wd, gradient=True,
                         q_strides=st(q), k_strides=st(k), dq_strides=st(dq), dk_strides=st(dk),
                         q_out_strides=st(qo), k_out_strides=st(ko), **more)
        dwq = torch.empty(q.shape[-1], device=q.device)
        dwk = None if k is None else torch.empty(q.shape[-1], device=q.device)
        work = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device=q.device)
        execute_heads_grad(plan, dq, dk, q, k, cos, sin, positions, wq, wk, qo, ko, dwq, dwk,
                           work, stream)
    return qo, ko, dwq, dwk


# ----------------------------------------------------------------- matrix products

class GemmPlan:
    """A plan of y = act(op(A) op(B) + bias) + residual: op(A) [m, k], op(B)
    [k, n]; a transposed operand is stored [k, m] or [n, k].  ``bias``: None, or
    the bias's type (the operands' or float32); strides between stored rows in
    elements (None = dense); any_alignment: A and B may start off 16 bytes."""

    def __init__(self, dtype, m: int, n: int, k: int, *, trans_a: bool = False,
                 trans_b: bool = False, bias=None, activation: str = "none",
                 residual: bool = False, any_alignment: bool = False, lda=None, ldb=None,
                 ldy=None, ld_residual=None, ld_preact=None):
        code = _dtype_code(dtype)
        a = ebin_gemm_attrs(code, code if bias is None else _dtype_code(bias), int(bool(trans_a)),
                            int(bool(trans_b)), ACTIVATIONS[activation], int(bias is not None),
                            int(bool(residual)), int(bool(any_alignment)), int(m), int(n), int(k),
                            *_row_strides("GemmPlan", lda=lda, ldb=ldb, ldy=ldy,
                                          ld_residual=ld_residual, ld_preact=ld_preact))
        self.handle = ebin_gemm_plan_create(a)
        self.workspace_bytes = ebin_gemm_plan_workspace(self.handle)

    def close(self):
        if self.handle:
            ebin_gemm_plan_release(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def execute_gemm(plan: GemmPlan, A, B, y, *, bias=None, residual=None, preact=None,
                 workspace=None, stream=None) -> None:
    """Enqueue a product on device buffers laid out as the plan says (torch
    tensors or int addresses); ``workspace``: a uint8 device tensor of at least
    plan.workspace_bytes (None where that is 0)."""
    st = lib.ebin_gemm_execute(plan.handle, *_ptrs(A, B, bias, residual, y, preact, workspace),
                               _bytes_of(workspace), _stream(stream))
    if st:
        raise EbinError(st, "ebin_gemm_execute")


class EpilogueGradPlan:
    """A plan of dz = dy act'(z) and, with bias=True, dbias = its sum over rows."""

    def __init__(self, dtype, m: int, n: int, *, activation: str = "none", bias: bool = False,
                 ld_dy=None, ld_z=None, ld_dz=None):
        a = ebin_epilogue_grad_attrs(_dtype_code(dtype), ACTIVATIONS[activation], int(bool(bias)),
                                     int(m), int(n),
                                     *_row_strides("EpilogueGradPlan", ld_dy=ld_dy, ld_z=ld_z,
                                                   ld_dz=ld_dz))
        self.handle = ebin_epilogue_grad_plan_create(a)
        self.workspace_bytes = ebin_epilogue_grad_plan_workspace(self.handle)

    def close(self):
        if self.handle:
            ebin_epilogue_grad_plan_release(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def execute_epilogue_grad(plan: EpilogueGradPlan, dy, z, dz, dbias=None, workspace=None,
                          stream=None) -> None:
    """Enqueue an epilogue's gradient on device buffers laid out as the plan says."""
    st = lib.ebin_epilogue_grad_execute(plan.handle, *_ptrs(dy, z, dz, dbias, workspace),
                                        _bytes_of(workspace), _stream(stream))
    if st:
        raise EbinError(st, "ebin_epilogue_grad_execute")


def _matrix(where, t, shape, dtype, device):
    """Row stride of a [rows, columns] tensor whose rows are dense; ValueError otherwise."""
    if t.dim() != 2 or (shape is not None and tuple(t.shape) != tuple(shape)):
        raise ValueError("%s: a matrix is %s, wanted %s" % (where, tuple(t.shape), shape))
    if t.dtype != dtype or t.device != device:
        raise ValueError("%s: a matrix is %s on %s, wanted %s on %s"
                         % (where, t.dtype, t.device, dtype, device))
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("%s: a matrix's rows are dense (strides %s)" % (where, t.stride()))
    width = max(1, t.shape[1])
    step = t.stride(0) if t.shape[0] > 1 else width
    if step < width:
        raise ValueError("%s: a matrix's rows lie apart (strides %s); pass an expanded tensor's "
                         "copy" % (where, t.stride()))
    return step


def _row_strides(where, **strides):
    """The ABI's row strides, where 0 stands for dense rows: None gives that, and
    0 itself, the stride of a broadcast tensor, is refused."""
    for name, v in strides.items():
        if v is not None and int(v) == 0:
            raise ValueError("%s: %s is 0; rows lie apart, and None means dense" % (where, name))
    return [0 if v is None else int(v) for v in strides.values()]


def gemm(a, b, bias=None, residual=None, *, trans_a: bool = False, trans_b: bool = False,
         activation: str = "none", out=None, preact=None, stream=None):
    """y = act(op(a) op(b) + bias) + residual on 16-bit CUDA tensors, in one
    call; a and b are matrices whose rows are dense and lie apart (a row stride
    is fine, an expanded tensor is not), transposed where trans_a / trans_b say
    so.  ``out`` may be ``residual``.
    ``preact``: a tensor that receives the pre-activation, which the gradient
    reads (gemm_epilogue_grad)."""
    import torch
    where = "gemm"
    _same_device(where, a, b, bias, residual, out, preact)
    if a.dim() != 2 or b.dim() != 2:
        raise ValueError("gemm: a and b are matrices")
    m, k = (a.shape[1], a.shape[0]) if trans_a else a.shape
    kb, n = (b.shape[1], b.shape[0]) if trans_b else b.shape
    if kb != k:
        raise ValueError("gemm: op(a) is [%d, %d] and op(b) [%d, %d]" % (m, k, kb, n))
    lda = _matrix(where, a, None, a.dtype, a.device)
    ldb = _matrix(where, b, None, a.dtype, a.device)
    if bias is not None and (tuple(bias.shape) != (n,) or not bias.is_contiguous()):
        raise ValueError("gemm: the bias is a contiguous [%d] tensor" % n)
    ld = [None if t is None else _matrix(where, t, (m, n), a.dtype, a.device)
          for t in (out, residual, preact)]
    with _launching(a.device, stream):
        if out is None:
            out = torch.empty(m, n, dtype=a.dtype, device=a.device)
        plan = GemmPlan(a.dtype, m, n, k, trans_a=trans_a, trans_b=trans_b,
                        bias=None if bias is None else bias.dtype, activation=activation,
                        residual=residual is not None, lda=lda, ldb=ldb, ldy=ld[0],
                        ld_residual=ld[1], ld_preact=ld[2],
                        any_alignment=a.data_ptr() % 16 != 0 or b.data_ptr() % 16 != 0)
        work = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device=a.device)
        execute_gemm(plan, a, b, out, bias=bias, residual=residual, preact=preact,
                     workspace=work, stream=stream)
    return out


def gemm_epilogue_grad(dy, z=None, *, activation: str = "none", bias: bool = True, out=None,
                       stream=None):
    """(dz, dbias) of a product's epilogue for the incoming gradient dy and the
    pre-activation z ([m, n] matrices; z is not read without an activation);
    dbias is float32 (None with bias=False).  ``out`` may be dy or z."""
    import torch
    where = "gemm_epilogue_grad"
    _same_device(where, dy, z, out)
    if activation != "none" and z is None:
        raise ValueError("gemm_epilogue_grad: %s needs z" % activation)
    shape = tuple(dy.shape)
    ld = [None if t is None else _matrix(where, t, shape, dy.dtype, dy.device)
          for t in (dy, z, out)]
    with _launching(dy.device, stream):
        if out is None:
            out = torch.empty(dy.shape, dtype=dy.dtype, device=dy.device)
        plan = EpilogueGradPlan(dy.dtype, shape[0], shape[1], activation=activation, bias=bias,
                                ld_dy=ld[0], ld_z=ld[1], ld_dz=ld[2])
        dbias = torch.empty(shape[1], device=dy.device) if bias else None
        work = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device=dy.device)
        execute_epilogue_grad(plan, dy, z, out, dbias, work, stream)
    return out, dbias
