"""The training operators' C ABI and binding without a GPU: the header's symbols,
what the calls refuse (all before the library touches CUDA), workspace sizes, and
the reference the GPU tests use, against differences and brute force."""
import ctypes
import os
import re

import pytest
import torch

import mixture_experts_layer_12_gb300 as moe
import train_reference as ref
from mixture_experts_layer_12_gb300 import build as moe_build, train

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return train._lib()


def test_exports_match_header(lib):
    with open(os.path.join(ROOT, "include", "moe_train.h")) as f:
        decl = set(re.findall(r"MOE_API\s+[\w\s\*]+?\b(moet_\w+)\s*\(", f.read()))
    assert decl == set(moe.TRAIN_EXPORTS)
    import subprocess
    out = subprocess.run(["nm", "-D", "--defined-only", moe.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    assert {w.split()[-1] for w in out.splitlines() if w.split()[-1].startswith("moet_")} == decl


# name -> (arguments between the shape and the pointers, pointers before status, which may be null)
CALLS = {
    "moet_expert_ffn": ((16,), 7, {6}), "moet_expert_ffn_backward": ((16,), 10, {2}),
    "moet_router_probs": ((), 4, {2}), "moet_route_backward": ((), 9, {4, 8}),
    "moet_forward": ((16,), 17, {2, 13, 14, 15, 16}), "moet_backward": ((16,), 19, {2, 12, 13, 16}),
}
SHAPE = dict(T=4, H=128, F=256, E=8, k=2)


def size_of(lib, name, s, bits=16):
    fn = getattr(lib, name + "_workspace_size")
    return fn(ctypes.byref(s), bits) if name == "moet_backward" else fn(ctypes.byref(s))


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), moe.MOE_ERR_INVALID_ARG), (dict(E=0), moe.MOE_ERR_UNSUPPORTED),
    (dict(E=257), moe.MOE_ERR_UNSUPPORTED), (dict(k=0), moe.MOE_ERR_UNSUPPORTED),
    (dict(k=9, E=16), moe.MOE_ERR_UNSUPPORTED), (dict(H=100), moe.MOE_ERR_UNSUPPORTED),
    (dict(gating=3), moe.MOE_ERR_INVALID_ARG), (dict(T=1 << 23, k=4), moe.MOE_ERR_UNSUPPORTED)])
def test_bad_shapes_are_refused(lib, name, kw, code):
    s = moe.make_shape(**{**SHAPE, **kw})
    mid, n, _ = CALLS[name]
    assert size_of(lib, name, s) == 0
    assert getattr(lib, name)(ctypes.byref(s), *mid, *([P(0x1000)] * n), P(0x1000), P(0x1000), 1 << 50, None) == code
    assert lib.moe_last_error_string()


@pytest.mark.parametrize("name", list(CALLS) + ["moet_dispatch_rows_backward", "moet_combine_backward"])
def test_widths_past_the_limits_are_refused(lib, name):
    mid, n, _ = CALLS.get(name, ((), {"moet_dispatch_rows_backward": 3}.get(name, 6), None))
    rest = [P(0x1000), P(0x1000), 1 << 62] if name in CALLS else []
    ffn = "ffn" in name or name in ("moet_forward", "moet_backward")
    for kw in (dict(H=(1 << 25) + 8), dict(H=2 ** 31 - 8)) + ((dict(F=(1 << 29) + 8), dict(F=2 ** 31 - 8)) if ffn else ()):
        s = moe.make_shape(**{**SHAPE, **kw})
        if name in CALLS:
            assert size_of(lib, name, s) == 0
        assert getattr(lib, name)(ctypes.byref(s), *mid, *([P(0x1000)] * n), *rest, None) == moe.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("name", list(CALLS))
def test_null_misaligned_and_small_buffers_are_refused(lib, name):
    mid, n, optional = CALLS[name]
    s = moe.make_shape(**SHAPE)
    need = size_of(lib, name, s)
    fn = getattr(lib, name)
    good = [P(0x1000 * (i + 1)) for i in range(n + 2)]
    for i in range(n + 2):
        for bad in (P(None), P(0x1008)):
            if i in optional:
                continue
            args = list(good)
            args[i] = bad
            assert fn(ctypes.byref(s), *mid, *args, need, None) == moe.MOE_ERR_INVALID_ARG, (i, bad)
    assert fn(ctypes.byref(s), *mid, *good, need - 1, None) == moe.MOE_ERR_INVALID_ARG
    assert b"_workspace_size" in lib.moe_last_error_string()
    assert fn(None, *mid, *good, need, None) == moe.MOE_ERR_INVALID_ARG
    if mid:
        assert fn(ctypes.byref(s), 4, *good, need, None) == moe.MOE_ERR_INVALID_ARG


def test_what_8_bits_and_the_softmax_over_all_need(lib):
    s = moe.make_shape(**SHAPE)
    need = size_of(lib, "moet_backward", s, 8)
    assert need > size_of(lib, "moet_backward", s, 16) and size_of(lib, "moet_backward", s, 4) == 0
    # positions of the scales of z and of x (and of x's codes)
    for name, at in (("moet_expert_ffn", (6,)), ("moet_expert_ffn_backward", (2,)), ("moet_forward", (13, 14, 15)),
                     ("moet_backward", (2, 12))):
        _, n, _ = CALLS[name]
        good = [P(0x1000 * (i + 1)) for i in range(n + 2)]
        for i in at:
            args = list(good)
            args[i] = P(None)
            assert getattr(lib, name)(ctypes.byref(s), 8, *args, 1 << 40, None) == moe.MOE_ERR_INVALID_ARG, (name, i)
    s1 = moe.make_shape(**SHAPE, gating=1)
    for name, i in (("moet_forward", 16), ("moet_backward", 13), ("moet_route_backward", 4)):
        mid, n, _ = CALLS[name]
        args = [P(0x1000 * (j + 1)) for j in range(n + 2)]
        args[i] = P(None)
        assert getattr(lib, name)(ctypes.byref(s1), *mid, *args, 1 << 40, None) == moe.MOE_ERR_INVALID_ARG, name


@pytest.mark.parametrize("rows,cols,code", [(-1, 8, moe.MOE_ERR_INVALID_ARG), (4, 12, moe.MOE_ERR_UNSUPPORTED),
                                            (4, 0, moe.MOE_ERR_UNSUPPORTED), (1 << 43, 8, moe.MOE_ERR_UNSUPPORTED),
                                            (4, -8, moe.MOE_ERR_INVALID_ARG)])
def test_a8_refuses(lib, rows, cols, code):
    for fn in (lib.moet_quantize_a8, lib.moet_dequantize_a8):
        assert fn(rows, cols, P(0x1000), P(0x2000), P(0x3000), None) == code
        assert fn(0, 8, None, None, None, None) == moe.MOE_OK
        for i in range(3):
            for bad in (P(None), P(0x1008)):
                args = [P(0x1000), P(0x2000), P(0x3000)]
                args[i] = bad
                assert fn(4, 8, *args, None) == moe.MOE_ERR_INVALID_ARG


def test_rows_refuse(lib):
    s = moe.make_shape(4, 128, 8, 8, 2)
    for fn, n in ((lib.moet_dispatch_rows_backward, 3), (lib.moet_combine_backward, 6)):
        for i in range(n):
            for bad in (P(None), P(0x1008)):
                args = [P(0x1000 * (j + 1)) for j in range(n)]
                args[i] = bad
                assert fn(ctypes.byref(s), *args, None) == moe.MOE_ERR_INVALID_ARG
        assert fn(ctypes.byref(moe.make_shape(4, 100, 8, 8, 2)), *([P(0x1000)] * n), None) == moe.MOE_ERR_UNSUPPORTED
        assert fn(ctypes.byref(moe.make_shape(0, 128, 8, 8, 2)), *([None] * n), None) == moe.MOE_OK


# name -> (pointers written, pointers read) with their bytes, in the order of the arguments; sizes for SHAPE, kept in
# 8 bits, softmax over all, n = T k
def buffers(name, bits):
    T, H, F, E, k = (SHAPE[v] for v in "THFEk")
    n = T * k
    z, zs = n * F * bits // 8, n * F // 32 if bits == 8 else 0
    x8, xs = (T * H, T * H // 32) if bits == 8 else (0, 0)
    w1 = w2 = 2 * E * H * F
    wr, p, th, nh, off = 2 * H * E, 4 * T * E, 2 * T * H, 2 * n * H, 4 * (E + 1)
    r, w = "r", "w"  # read, written
    return {
        "moet_dispatch_rows_backward": [(r, nh), (r, 4 * n), (w, th)],
        "moet_combine_backward": [(r, th), (r, nh), (r, 4 * n), (r, 4 * n), (w, nh), (w, 4 * n)],
        "moet_expert_ffn": [(r, nh), (r, w1), (r, w2), (r, off), (w, nh), (w, z), (w, zs)],
        "moet_expert_ffn_backward": [(r, nh), (r, z), (r, zs), (r, w1), (r, w2), (r, off), (r, nh), (w, nh), (w, w1),
                                     (w, w2)],
        "moet_router_probs": [(r, th), (r, wr), (r, 4 * E), (w, p)],
        "moet_route_backward": [(r, th), (r, wr), (r, 4 * n), (r, 4 * n), (r, p), (r, 4 * n), (w, th), (w, wr),
                                (w, 4 * E)],
        "moet_forward": [(r, th), (r, wr), (r, 4 * E), (r, w1), (r, w2), (w, th), (w, 4 * n), (w, 4 * n), (w, 4 * E),
                         (w, off), (w, 4 * n), (w, 4 * n), (w, z), (w, zs), (w, x8), (w, xs), (w, p)],
        "moet_backward": [(r, th), (r, T * H * bits // 8), (r, xs), (r, wr), (r, w1), (r, w2), (r, 4 * n), (r, 4 * n),
                          (r, off), (r, 4 * n), (r, 4 * n), (r, z), (r, zs), (r, p), (w, th), (w, wr), (w, 4 * E),
                          (w, w1), (w, w2)],
    }[name]


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses, of which some calls are not refused")
@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("name", ["moet_dispatch_rows_backward", "moet_combine_backward", *CALLS])
def test_outputs_that_overlap_are_refused(lib, name, bits):
    """Every output, the status block and the workspace one 16-byte piece into the
    front or the end of every other buffer of the call; side by side they pass on
    to the device, of which there is none."""
    s = moe.make_shape(**SHAPE, gating=1)
    bufs = buffers(name, bits)
    mid = (bits,) if name in CALLS and CALLS[name][0] else ()
    tail = []
    if name in CALLS:
        need = size_of(lib, name, s, bits)
        bufs = bufs + [("w", moe.MOE_WS_MIN_BYTES), ("w", need)]
        tail = [need]
    step = 1 << 30
    at = [step * (i + 1) for i in range(len(bufs))]

    def call(addresses):
        return getattr(lib, name)(ctypes.byref(s), *mid, *[P(a) for a in addresses], *tail, None)

    assert call(at) == moe.MOE_ERR_CUDA
    for i, (kind, size) in enumerate(bufs):
        if kind == "r" or size == 0:
            continue
        for j, (_, other) in enumerate(bufs):
            if i == j or other == 0:
                continue
            up = [-(-v // 16) * 16 for v in (other, size)]  # whole 16-byte pieces
            for d, code in ((up[0] - 16, moe.MOE_ERR_INVALID_ARG), (16 - up[1], moe.MOE_ERR_INVALID_ARG),
                            (up[0], moe.MOE_ERR_CUDA), (-up[1], moe.MOE_ERR_CUDA)):
                a = list(at)
                a[i] = at[j] + d
                assert call(a) == code, (i, j, d)
                if code == moe.MOE_ERR_INVALID_ARG:
                    assert b"overlaps" in lib.moe_last_error_string()
    for i, (kind, _) in enumerate(bufs):  # inputs may be one another's
        for j, (other, _) in enumerate(bufs):
            if kind == other == "r":
                a = list(at)
                a[i] = a[j]
                assert call(a) == moe.MOE_ERR_CUDA


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses, of which some calls are not refused")
def test_a8_outputs_that_overlap_are_refused(lib):
    rows, cols = 4, 40  # 320 bytes of bf16, 160 of codes, 8 of scales
    a, b, c = 1 << 30, 1 << 31, 1 << 32
    q, d = lib.moet_quantize_a8, lib.moet_dequantize_a8
    for fn, args in ((q, (a, b, c)), (q, (a, a + 320, a + 480)), (q, (a, a - 160, a - 176)), (d, (a, b, c)),
                     (d, (a, a, b)), (d, (a, a + 160, a + 176)), (d, (a, a - 16, a - 336))):
        assert fn(rows, cols, *[P(v) for v in args], None) == moe.MOE_ERR_CUDA, args
    for fn, args in ((q, (a, a, c)), (q, (a, a + 304, c)), (q, (a, a - 144, c)), (q, (a, b, a + 16)),
                     (q, (a, b, b + 144)), (d, (a, b, a)), (d, (a, b, b - 304)), (d, (a, b, b)), (d, (a, b, a + 144))):
        assert fn(rows, cols, *[P(v) for v in args], None) == moe.MOE_ERR_INVALID_ARG, args
        assert b"overlaps" in lib.moe_last_error_string()


def test_workspaces_hold_what_a_call_needs(lib):
    s = moe.make_shape(4096, 4096, 14336, 8, 2)
    n, pad = 8192, 8192 + 8 * 15
    assert size_of(lib, "moet_backward", s) >= 2 * pad * (2 * 4096 + 2 * 14336) + 4 * n * 4096
    assert size_of(lib, "moet_expert_ffn", s) >= 2 * n * 14336


def test_a8_tensor_checks_shapes():
    c = torch.zeros(3, 40, dtype=torch.int8)
    moe.A8Tensor(c, torch.zeros(3, 2, dtype=torch.uint8))
    for bad in (torch.zeros(3, 1, dtype=torch.uint8), torch.zeros(2, 2, dtype=torch.uint8)):
        with pytest.raises(ValueError):
            moe.A8Tensor(c, bad)
    with pytest.raises(TypeError):
        moe.A8Tensor(c.int(), torch.zeros(3, 2, dtype=torch.uint8))
    with pytest.raises(TypeError):
        moe.A8Tensor(c, torch.zeros(3, 2))


def test_binding_refuses_host_tensors_and_wrong_shapes():
    bf = torch.bfloat16
    x = torch.zeros(4, 16, dtype=bf)
    slot = torch.zeros(4, 2, dtype=torch.int32)
    w1, w2 = torch.zeros(2, 16, 8, dtype=bf), torch.zeros(2, 8, 16, dtype=bf)
    o = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match=r"dxp must be \[T \* k, H\]"):
        moe.dispatch_rows_backward(x, slot)
    with pytest.raises(ValueError, match="w1 must be"):
        moe.expert_ffn(x, w1, w2, o, act="swiglu")
    with pytest.raises(ValueError, match="xp must be"):
        moe.expert_ffn_backward(x[:, :8], x, w1, w2, o, x)
    with pytest.raises(ValueError, match="x must be"):
        moe.route_backward(x, torch.zeros(8, 4, dtype=bf), slot, torch.zeros(4, 2), torch.zeros(4, 2))
    if not torch.cuda.is_available():
        return
    with pytest.raises(ValueError, match="CUDA"):
        moe.quantize_a8(x)


@pytest.mark.skipif(torch.cuda.is_available(), reason="host tensors, which the calls would pass on")
def test_kept_tensors_that_were_replaced_are_checked(lib, monkeypatch):
    """The sizes of what a Saved or an A8Tensor holds are checked by the calls that
    read them, not only when it is made: smaller ones would be read past their end."""
    monkeypatch.setattr(train, "_here", lambda: (-1, None))  # host tensors pass for tensors of this device
    bf, i8, u8 = torch.bfloat16, torch.int8, torch.uint8
    q = moe.A8Tensor(torch.zeros(6, 64, dtype=i8), torch.zeros(6, 2, dtype=u8))
    q.scales = q.scales[:3]
    with pytest.raises(ValueError, match="scales must be"):
        moe.dequantize_a8(q)
    w1, w2, o = torch.zeros(2, 32, 64, dtype=bf), torch.zeros(2, 64, 32, dtype=bf), torch.zeros(3, dtype=torch.int32)
    rows = torch.zeros(6, 32, dtype=bf)
    with pytest.raises(ValueError, match="z.scales must be"):
        moe.expert_ffn_backward(rows, q, w1, w2, o, rows)

    layer = object.__new__(moe.MoETrainLayer)
    layer.E, layer.F, layer.H, layer.k, layer.act, layer.capacity_factor, layer.gating = 2, 64, 32, 2, "gelu", None, 1
    layer.w_router, layer.w1, layer.w2, layer.bias = torch.zeros(32, 2, dtype=bf), w1, w2, None
    layer.status = torch.zeros(256, dtype=u8)

    def saved(bits):
        v = moe.Saved()
        v.call, v._stream = layer._call(3), None
        v.x = rows[:3] if bits == 16 else moe.A8Tensor(torch.zeros(3, 32, dtype=i8), torch.zeros(3, 1, dtype=u8))
        v.z = torch.zeros(6, 64, dtype=bf) if bits == 16 else moe.A8Tensor(torch.zeros(6, 64, dtype=i8),
                                                                            torch.zeros(6, 2, dtype=u8))
        v.probs = torch.zeros(3, 2)
        v._block = torch.zeros(64, dtype=torch.int32)
        v.versions = layer._versions(v)
        return v

    dy = rows[3:]
    for bits in (16, 8):
        v = saved(bits)
        v.z = v.z[:5] if bits == 16 else moe.A8Tensor(v.z.codes[:5], v.z.scales[:5])
        with pytest.raises(ValueError, match="z(.codes)? must be"):
            layer.backward(v, dy)
        v = saved(bits)
        v.probs = v.probs[:2]
        with pytest.raises(ValueError, match="probs must be"):
            layer.backward(v, dy)
        v = saved(bits)
        v.z = saved(24 - bits).z
        with pytest.raises(ValueError, match="bits"):
            layer.backward(v, dy)
        with pytest.raises(moe.MoEError) as e:  # what was kept goes on to the library, which finds no device
            layer.backward(saved(bits), dy)
        assert e.value.code == moe.MOE_ERR_CUDA
    v = saved(8)
    v.x.scales = v.x.scales[:2]
    with pytest.raises(ValueError, match="x.scales must be"):
        layer.backward(v, dy)


def test_sizes_past_32_bits_are_refused(monkeypatch):
    """Not cut to their lower 32 bits (4 rows, 8 columns)."""
    monkeypatch.setattr(train, "_here", lambda: (-1, None))  # tensors without memory, on no device
    new = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device="meta")  # noqa: E731
    many = (1 << 32) + 4
    for kw in (dict(T=many), dict(H=1 << 31), dict(F=1 << 32), dict(E=(1 << 32) + 8), dict(k=(1 << 32) + 2)):
        with pytest.raises(ValueError, match="32 bits"):
            moe.make_shape(**{**SHAPE, **kw})
    with pytest.raises(ValueError, match=r"2\^31"):
        moe.quantize_a8(new(1, (1 << 32) + 8))
    with pytest.raises(ValueError, match=r"2\^31"):
        moe.dequantize_a8(moe.A8Tensor(new((1 << 32) + 8, dtype=torch.int8), new((1 << 27) + 1, dtype=torch.uint8)))
    with pytest.raises(ValueError, match="32 bits"):
        moe.dispatch_rows_backward(new(many, 8), new(many, 1, dtype=torch.int32))
    with pytest.raises(ValueError, match="32 bits"):
        moe.expert_ffn(new(many, 8), new(1, 8, 8), new(1, 8, 8), new(2, dtype=torch.int32))


# ------------------------------------------------------ the tests' reference --

@pytest.mark.parametrize("gating", [0, 1, 2])
@pytest.mark.parametrize("act", ["gelu", "swiglu"])
def test_reference_gradients_match_differences(act, gating):
    """Directional derivatives of sum(y dy) by central differences with step h:
    off by h^2 times a third derivative (below 1e4 at these sizes: 1e-8) and by
    2^-52 |f| / h (1e-9)."""
    g = torch.Generator().manual_seed(5)
    T, H, F, E, k = 9, 16, 24, 5, 3
    gated = act == "swiglu"
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, wr, b = rnd(T, H), rnd(H, E) / 4, rnd(E)
    w1, w2, dy = rnd(E, H, (2 if gated else 1) * F) / 4, rnd(E, F, H) / 5, rnd(T, H)
    lg = x @ wr + b
    ids = torch.topk(lg, k, dim=1).indices
    counts, offsets, perm, slot = ref.dispatch(ids, E, ref.capacity(T, k, E, 0.8))
    assert (slot < 0).any()
    n = int(offsets[-1])
    z = torch.cat([x[perm[int(offsets[e]):int(offsets[e + 1])] // k] @ w1[e] for e in range(E)])
    z = z.view(n, 2, F) if gated else z
    r = ref.layer_backward(x, z, wr, w1, w2, ids, ref.gate(lg, ids, gating), torch.softmax(lg, 1), offsets, perm, slot,
                           dy, gating, gated)
    h = 1e-6
    args = dict(x=x, wr=wr, b=b, w1=w1, w2=w2)
    for name, key in (("x", "dx"), ("wr", "dw_router"), ("b", "dbias"), ("w1", "dw1"), ("w2", "dw2")):
        for _ in range(3):
            d = rnd(*args[name].shape)
            f = [float((ref.layer(*[a + s * h * d if n2 == name else a for n2, a in args.items()], ids, slot, gating,
                                  gated) * dy).sum()) for s in (1, -1)]
            want = (f[0] - f[1]) / (2 * h)
            got = float((r[key][0] * d).sum())
            assert abs(got - want) <= 1e-7 * (1 + abs(want)) * 10, (name, got, want)


def test_reference_8_bits_by_brute_force():
    v = torch.tensor([[127.0, 63.5, 0.5, 1.5, -127.0] + [0.0] * 27, [127.5] * 32, [0.0] * 32, [2.0 ** -130] * 32])
    b = ref.a8_scales(v)
    assert b[:, 0].tolist() == [127, 128, 1, 1]
    assert ref.a8_codes(v, b)[0, :5].tolist() == [127, 64, 0, 2, -127]
    assert ref.a8_codes(v, b)[1, 0] == 64 and ref.a8_codes(v, b)[3, 0] == 0
    x = torch.randn(50, 72, generator=torch.Generator().manual_seed(1)).bfloat16()
    b = ref.a8_scales(x)
    q = ref.a8_codes(x, b)
    assert int(q.abs().max()) <= 127
    s = torch.exp2((b - 127).double()).repeat_interleave(32, 1)[:, :72]
    assert ((ref.a8_values(q, b) - x.double()).abs() <= s / 2).all()
    m = torch.nn.functional.pad(x.double().abs(), (0, 24)).view(50, 3, 32).amax(2)
    assert (m > 127 * torch.exp2((b - 128).double())).all()  # no smaller scale would do
