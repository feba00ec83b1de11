"""CPU check of the copies that bring rows off the vectors to shared memory: nothing outside
the tensor is read, and every element is where its lane reads it, whatever the widths,
strides and first addresses.

The kernel's schedule (csrc/ebin_block_copy.h) is compiled here and drives a model of a
chunk's buffer; schedules that do less must be caught.
"""
import ctypes
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "broadcast_elementwise_gb300", "csrc")
# bytes of an element, columns of a lane's piece: 16-bit rows, 32-bit rows, 16-bit beside 32-bit
KINDS = [(2, 8), (4, 4), (2, 4)]


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("copies") / "libcopies.so")
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I" + CSRC,
                           os.path.join(HERE, "row_copies.cpp"), "-o", so])
    fn = ctypes.CDLL(so).row_copies
    i64 = ctypes.c_int64
    fn.argtypes = [ctypes.c_int, ctypes.c_int, i64, i64, i64, ctypes.c_size_t, ctypes.c_int,
                   ctypes.POINTER(i64), ctypes.POINTER(i64)]

    def run(size, columns, rule=0, widths=(1, 2, 3, 5, 8, 31, 77, 129, 256, 257, 515, 1021)):
        outside = missing = 0
        for n in widths:
            for rows in (1, 2, 5, 9, 17, 40):
                for ld in (n, n + 1, n + 24):
                    for off in range(0, 16, size):
                        o, m = i64(), i64()
                        fn(size, columns, rows, n, ld, 4096 + off, rule, ctypes.byref(o),
                           ctypes.byref(m))
                        outside, missing = outside + o.value, missing + m.value
        return outside, missing

    return run


@pytest.mark.parametrize("size,columns", KINDS)
def test_copies_stay_within_the_tensor(check, size, columns):
    assert check(size, columns) == (0, 0)


@pytest.mark.parametrize("size,columns", KINDS)
def test_whole_vectors_are_caught(check, size, columns):
    outside, missing = check(size, columns, 1)
    assert outside > 1000 and missing == 0


def test_the_first_and_last_row_alone_are_caught(check):
    """Rows of a few bytes: a vector of the third row begins before the first one."""
    assert check(2, 8, 2, widths=(1, 2, 3))[0] > 100
