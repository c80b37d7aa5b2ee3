"""What the decode operators' self-test refuses, before the library touches CUDA,
and what the other entry points load of them."""
import ctypes
import os
import subprocess

import pytest

import mixture_experts_layer_12_gb300 as moe
from mixture_experts_layer_12_gb300 import build as moe_build, decode


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return decode._lib()


SHAPE = dict(T=4, H=128, F=256, E=8, k=2)


@pytest.mark.parametrize("kw,group,limit_ns,code", [
    (dict(T=65), 0, 10 ** 6, moe.MOE_ERR_UNSUPPORTED), (dict(), 48, 10 ** 6, moe.MOE_ERR_UNSUPPORTED),
    (dict(F=160), 64, 10 ** 6, moe.MOE_ERR_UNSUPPORTED), (dict(), 0, 999, moe.MOE_ERR_INVALID_ARG),
    (dict(), 64, 10 ** 9 + 1, moe.MOE_ERR_INVALID_ARG),
])
def test_wait_selftest_refuses(lib, kw, group, limit_ns, code):
    s = moe.make_shape(**{**SHAPE, **kw})
    good = [ctypes.c_void_p(0x1000 * (i + 1)) for i in range(15)]
    assert lib.moed_selftest_wait_timeout(ctypes.byref(s), group, *good, 1 << 40, limit_ns, None) == code


def test_wait_selftest_refuses_null_and_small_buffers(lib):
    s = moe.make_shape(**SHAPE)
    need = lib.moed_workspace_size(ctypes.byref(s))
    good = [ctypes.c_void_p(0x1000 * (i + 1)) for i in range(15)]
    for i in range(15):
        if i == 2:
            continue  # the bias may be null
        args = list(good)
        args[i] = None
        assert lib.moed_selftest_wait_timeout(ctypes.byref(s), 64, *args, need, 10 ** 6, None) == \
            moe.MOE_ERR_INVALID_ARG, i
    assert lib.moed_selftest_wait_timeout(ctypes.byref(s), 0, *good, need - 1, 10 ** 6, None) == \
        moe.MOE_ERR_INVALID_ARG


def test_other_entry_points_do_not_load_the_decode_kernels(lib):
    """What sets a device up for moe.h's calls refers to nothing of the decode
    operators: their kernels' code is loaded by their own first call."""
    objs = [s.replace(".cu", ".o") for s in moe_build.SOURCES if not s.startswith(("decode", "q4"))]
    assert "api.o" in objs
    for o in objs:
        path = os.path.join(moe_build.BUILD_DIR, o)
        syms = subprocess.run(["nm", "-u", path], capture_output=True, text=True, check=True).stdout
        assert "decode" not in syms and "q4" not in syms, o


@pytest.mark.parametrize("name", ["w_router", "w1", "w2", "bias", "q4", "E", "F", "H", "k", "act", "capacity_factor",
                                  "gating"])
def test_what_a_layer_was_made_with_cannot_be_set(name):
    """It would hold for batch sizes not seen yet and be ignored for the others."""
    with pytest.raises(AttributeError):
        setattr(object.__new__(moe.MoEDecodeLayer), name, 1)
