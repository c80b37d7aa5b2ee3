"""The decode operators' C ABI and binding without a GPU: the header's
symbols, what the calls refuse (all before the library touches CUDA), the
workspace sizes, the 4-bit layout's shape rules, and the reference the GPU
tests use, against brute force."""
import copy
import ctypes
import os
import pickle
import re

import pytest
import torch

import decode_reference as ref
import mixture_experts_layer_12_gb300 as moe
from mixture_experts_layer_12_gb300 import build as moe_build, decode

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return decode._lib()


def test_exports_match_header(lib):
    with open(os.path.join(ROOT, "include", "moe_decode.h")) as f:
        decl = set(re.findall(r"MOE_API\s+[\w\s\*]+?\b(moed_\w+)\s*\(", f.read()))
    assert decl == set(moe.DECODE_EXPORTS)
    import subprocess
    out = subprocess.run(["nm", "-D", "--defined-only", moe.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    assert {w.split()[-1] for w in out.splitlines() if w.split()[-1].startswith("moed_")} == decl


def test_header_limits_match_the_binding():
    with open(os.path.join(ROOT, "include", "moe_decode.h")) as f:
        src = f.read()
    assert f"#define MOED_MAX_TOKENS {moe.MOED_MAX_TOKENS}\n" in src
    assert f"#define MOED_MAX_ROWS {moe.MOED_MAX_ROWS}\n" in src


SHAPE = dict(T=4, H=128, F=256, E=8, k=2)


@pytest.mark.parametrize("kw,code", [
    (dict(T=65), moe.MOE_ERR_UNSUPPORTED), (dict(T=-1), moe.MOE_ERR_INVALID_ARG),
    (dict(E=0), moe.MOE_ERR_UNSUPPORTED), (dict(E=257), moe.MOE_ERR_UNSUPPORTED),
    (dict(k=0), moe.MOE_ERR_UNSUPPORTED), (dict(k=9, E=16), moe.MOE_ERR_UNSUPPORTED),
    (dict(k=5, E=4), moe.MOE_ERR_UNSUPPORTED), (dict(H=100), moe.MOE_ERR_UNSUPPORTED),
    (dict(F=4), moe.MOE_ERR_UNSUPPORTED), (dict(gating=3), moe.MOE_ERR_INVALID_ARG),
])
def test_layer_refuses_bad_shapes(lib, kw, code):
    s = moe.make_shape(**{**SHAPE, **kw})
    assert lib.moed_workspace_size(ctypes.byref(s)) == 0
    assert lib.moed_forward(ctypes.byref(s), *([None] * 13), 0, None) == code
    assert lib.moed_forward_q4(ctypes.byref(s), 32, *([None] * 15), 0, None) == code
    assert lib.moe_last_error_string()


@pytest.mark.parametrize("kw,group", [(dict(H=96), 64), (dict(F=160), 64), (dict(), 16), (dict(), 0),
                                      (dict(), 256), (dict(H=64), 128)])
def test_q4_layer_refuses_bad_groups(lib, kw, group):
    s = moe.make_shape(**{**SHAPE, **kw})
    assert lib.moed_forward_q4(ctypes.byref(s), group, *([None] * 15), 0, None) == moe.MOE_ERR_UNSUPPORTED


def test_layer_refuses_null_misaligned_and_small_buffers(lib):
    s = moe.make_shape(**SHAPE)
    need = lib.moed_workspace_size(ctypes.byref(s))
    P = ctypes.c_void_p
    good = [P(0x1000 * (i + 1)) for i in range(13)]
    calls = 0
    for i in range(13):
        for bad in (P(None), P(0x1008)):
            if i == 2 and bad.value is None:
                continue  # the bias may be null
            args = list(good)
            args[i] = bad
            assert lib.moed_forward(ctypes.byref(s), *args, need, None) == moe.MOE_ERR_INVALID_ARG, i
            calls += 1
    assert calls == 25
    assert lib.moed_forward(ctypes.byref(s), *good, need - 1, None) == moe.MOE_ERR_INVALID_ARG
    assert b"moed_workspace_size" in lib.moe_last_error_string()
    assert lib.moed_forward(None, *good, need, None) == moe.MOE_ERR_INVALID_ARG
    good = [P(0x1000 * (i + 1)) for i in range(15)]
    for i in range(15):
        if i == 2:
            continue
        args = list(good)
        args[i] = P(None)
        assert lib.moed_forward_q4(ctypes.byref(s), 64, *args, need, None) == moe.MOE_ERR_INVALID_ARG, i


@pytest.mark.parametrize("kw,code", [
    (dict(rows=513), moe.MOE_ERR_UNSUPPORTED), (dict(rows=-1), moe.MOE_ERR_INVALID_ARG),
    (dict(K=96), moe.MOE_ERR_UNSUPPORTED), (dict(K=0), moe.MOE_ERR_UNSUPPORTED),
    (dict(N=12), moe.MOE_ERR_UNSUPPORTED), (dict(N=0), moe.MOE_ERR_UNSUPPORTED),
    (dict(E=0), moe.MOE_ERR_UNSUPPORTED), (dict(E=257), moe.MOE_ERR_UNSUPPORTED),
    (dict(group=48), moe.MOE_ERR_UNSUPPORTED), (dict(n_segments=0), moe.MOE_ERR_INVALID_ARG),
    (dict(n_segments=257), moe.MOE_ERR_INVALID_ARG),
])
def test_matvec_refuses(lib, kw, code):
    a = {**dict(rows=3, K=128, N=64, E=4, group=64, n_segments=4), **kw}
    P = ctypes.c_void_p
    ptrs = [P(0x1000 * (i + 1)) for i in range(6)]
    assert lib.moed_matvec_q4(*a.values(), *ptrs, 1 << 40, None) == code


def test_matvec_refuses_null_misaligned_and_small_buffers(lib):
    P = ctypes.c_void_p
    need = lib.moed_matvec_q4_workspace_size(3, 4, 128, 64)
    assert need > 0 and lib.moed_matvec_q4_workspace_size(513, 4, 128, 64) == 0
    good = [P(0x1000 * (i + 1)) for i in range(6)]
    for i in range(6):
        for bad in (P(None), P(0x1008)):
            args = list(good)
            args[i] = bad
            assert lib.moed_matvec_q4(3, 128, 64, 4, 64, 4, *args, need, None) == moe.MOE_ERR_INVALID_ARG
    assert lib.moed_matvec_q4(3, 128, 64, 4, 64, 4, *good, need - 1, None) == moe.MOE_ERR_INVALID_ARG


def test_matvec_refuses_a_y_that_overlaps_x(lib):
    P = ctypes.c_void_p
    need = lib.moed_matvec_q4_workspace_size(3, 1, 128, 64)
    x, nx, ny = 0x10000, 3 * 128 * 2, 3 * 64 * 2
    for y in (x, x + nx - 16, x - ny + 16):
        rc = lib.moed_matvec_q4(3, 128, 64, 1, 64, 1, P(x), P(0x1000), P(0x2000), None, P(y), P(0x3000), need, None)
        assert rc == moe.MOE_ERR_INVALID_ARG and b"overlaps" in lib.moe_last_error_string()


def test_a_copied_q4weights_has_addresses_of_its_own():
    w = moe.Q4Weights(torch.zeros(2, 16, 8, dtype=torch.int32), torch.ones(2, 4, 8, dtype=torch.bfloat16))
    for c in (copy.deepcopy(w), pickle.loads(pickle.dumps(w))):
        assert c._args == (c.codes.data_ptr(), c.scales.data_ptr())
        assert not set(c._args) & set(w._args)
        assert (c.E, c.K, c.N, c.group) == (2, 128, 8, 32) and torch.equal(c.scales, w.scales)


def test_conversions_refuse(lib):
    P = ctypes.c_void_p
    good = [P(0x1000 * (i + 1)) for i in range(3)]
    for fn in (lib.moed_quantize_q4, lib.moed_dequantize_q4):
        for dims in ((0, 128, 64, 64), (4, 96, 64, 64), (4, 128, 60, 64), (4, 128, 64, 100), (4, 0, 64, 32),
                     (4, 128, -8, 32), (256, 1 << 24, 1 << 24, 32)):
            assert fn(*dims, *good, None) == moe.MOE_ERR_UNSUPPORTED, dims
        for i in range(3):
            for bad in (P(None), P(0x1008)):
                args = list(good)
                args[i] = bad
                assert fn(4, 128, 64, 64, *args, None) == moe.MOE_ERR_INVALID_ARG


def test_workspace_grows_with_the_call(lib):
    size = lambda **kw: moe.moed_workspace_size(moe.make_shape(**{**SHAPE, **kw}))  # noqa: E731
    assert size(T=0) > moe.MOE_WS_MIN_BYTES
    assert size(T=1) <= size(T=8) < size(T=9) < size(T=64, k=8)
    # holds h and the fp32 expert outputs of T*k rows
    assert size(T=64, k=8, H=4096, F=14336) >= 512 * (4096 * 4 + 14336 * 2)


def test_q4_weights_shapes():
    c, s = torch.zeros(2, 16, 24, dtype=torch.int32), torch.zeros(2, 2, 24, dtype=torch.bfloat16)
    w = moe.Q4Weights(c, s)
    assert (w.E, w.K, w.N, w.group) == (2, 128, 24, 64)
    assert moe.Q4Weights(c[0], s[0]).E == 1
    with pytest.raises(TypeError):
        moe.Q4Weights(c.long(), s)
    with pytest.raises(TypeError):
        moe.Q4Weights(c, s.float())
    for bad in (s[:, :, :16], s[:1], torch.zeros(2, 8, 24, dtype=torch.bfloat16),
                torch.zeros(2, 3, 24, dtype=torch.bfloat16), s[0]):
        with pytest.raises(ValueError):
            moe.Q4Weights(c, bad)
    with pytest.raises(ValueError, match="contiguous"):
        moe.Q4Weights(c.transpose(1, 2).contiguous().transpose(1, 2), s)


def test_layer_object_refuses_mismatched_weights(lib):
    bf = dict(dtype=torch.bfloat16)
    wr, w1, w2 = torch.zeros(128, 8, **bf), torch.zeros(8, 128, 256, **bf), torch.zeros(8, 256, 128, **bf)
    for args, kw in (((wr, w1, w2[:, :, :64]), {}), ((wr, w1, w2), dict(act="swiglu")),
                     ((wr[:, :4], w1, w2), {}), ((wr, w1[0], w2), {}), ((wr, w1, w2[0]), {})):
        with pytest.raises(ValueError):
            moe.MoEDecodeLayer(*args, 2, **kw)
    q = moe.Q4Weights(torch.zeros(8, 16, 256, dtype=torch.int32), torch.zeros(8, 1, 256, **bf))
    with pytest.raises(TypeError):
        moe.MoEDecodeLayer(wr, q, w2, 2)
    with pytest.raises(ValueError, match="CUDA"):
        moe.MoEDecodeLayer(wr, w1, w2, 2)
    with pytest.raises(ValueError):
        moe.quantize_q4(torch.zeros(100, 64, **bf), 32)
    with pytest.raises(ValueError):
        moe.quantize_q4(torch.zeros(128, 64, **bf), 16)
    with pytest.raises(ValueError):
        moe.matvec_q4(torch.zeros(2, 64, **bf), q)


def test_reference_packs_and_unpacks():
    g = torch.Generator().manual_seed(3)
    c = torch.randint(0, 16, (2, 64, 5), generator=g)
    words = ref.pack_codes(c)
    assert words.dtype == torch.int32 and torch.equal(ref.unpack_codes(words), c)
    # nibble i of word r is row 8 r + i
    for e, r, n in ((0, 0, 0), (1, 7, 4), (0, 3, 2)):
        v = int(words[e, r, n]) & 0xFFFFFFFF
        assert [(v >> (4 * i)) & 15 for i in range(8)] == c[e, 8 * r:8 * r + 8, n].tolist()


def test_reference_dispatch_is_the_counting_sort():
    import oracle
    g = torch.Generator().manual_seed(4)
    ids = torch.stack([torch.randperm(6, generator=g)[:3] for _ in range(17)])
    for cf in (None, 0.6):
        cap = ref.capacity(17, 3, 6, cf)
        want = oracle.dispatch(ids.int().numpy(), 6, cf)
        for got, w in zip(ref.dispatch(ids, 6, cap), want):
            assert (got.numpy() == w).all()
