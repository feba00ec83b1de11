"""CPU check of how a matrix product winds down when a wait inside it runs out: whatever
the warps had done, on one CTA or a pair, no operand copy may still be on its way when
shared memory is left, and every wait ends once the copies have landed.

The kernel's schedule (csrc/ebin_gemm_drain.h) is compiled here and drives a model of
the stage barriers over random walks that stop anywhere; schedules that do less must
be caught.
"""
import ctypes
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "broadcast_elementwise_gb300", "csrc")


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("drain") / "libdrain.so")
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I" + CSRC,
                           os.path.join(HERE, "drain_schedule.cpp"), "-o", so])
    fn = ctypes.CDLL(so).drain_check
    fn.restype = ctypes.c_int
    fn.argtypes = [ctypes.c_uint64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                   ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]

    def run(ctas, rule, walks=20000):
        stuck, uneven = ctypes.c_int(), ctypes.c_int()
        left = fn(7, walks, ctas, rule, ctypes.byref(stuck), ctypes.byref(uneven))
        return left, stuck.value, uneven.value

    return run


@pytest.mark.parametrize("ctas", [1, 2])
def test_nothing_is_left_on_its_way(check, ctas):
    left, stuck, uneven = check(ctas, 0)
    assert (left, stuck) == (0, 0)
    assert ctas == 1 or uneven > 1000      # pairs that stopped at different steps were met


@pytest.mark.parametrize("ctas", [1, 2])
def test_a_drain_by_the_copying_warp_alone_is_caught(check, ctas):
    """The wait that ran out may be another warp's: the copies it had issued stay open."""
    assert check(ctas, 1)[0] > 1000


def test_plain_waits_are_caught_on_a_pair(check):
    """The leader's own steps alone: a peer that is ahead leaves copies open, one that is
    behind leaves waits that never end."""
    left, stuck, _ = check(2, 2)
    assert left > 100 and stuck > 100
    assert check(1, 2)[:2] == (0, 0)
