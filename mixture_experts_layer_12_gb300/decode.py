"""Decode operators of the MoE layer: Python binding of include/moe_decode.h.

The whole layer for a few tokens in two kernels (:class:`MoEDecodeLayer`,
:func:`moed_forward`), with bf16 experts or with 4-bit ones and group scales
(:class:`Q4Weights`), grouped 4-bit matrix-vector products
(:func:`matvec_q4`), and the conversions between bf16 and 4 bits
(:func:`quantize_q4`, :func:`dequantize_q4`).  The ``moed_*`` functions mirror
the C entry points name for name; the others allocate what they return.
As in the rest of the package every step runs in the library's CUDA kernels.
"""
from __future__ import annotations

import ctypes
import threading

import torch

from . import (_BF, _F32, _I32, _args, _check, _forward_specs, _ptr, _stream, _ws, MOE_ERR_UNSUPPORTED,
               MOE_GATE_TOPK_SOFTMAX, RoutingBuffers, check_tensor, load_library, make_shape, moe_shape)

MOED_MAX_TOKENS = 64
MOED_MAX_ROWS = 512

# Every symbol include/moe_decode.h declares.
DECODE_EXPORTS = ("moed_workspace_size", "moed_forward", "moed_forward_q4",
                  "moed_matvec_q4_workspace_size", "moed_matvec_q4", "moed_quantize_q4",
                  "moed_dequantize_q4", "moed_selftest_wait_timeout")

_sig_lock = threading.Lock()
_sig_lib = None


def _lib():
    """The library with the decode entry points' signatures set."""
    global _sig_lib
    if _sig_lib is not None:
        return _sig_lib
    lib = load_library()
    with _sig_lock:
        P, S, I, Z = ctypes.c_void_p, ctypes.POINTER(moe_shape), ctypes.c_int32, ctypes.c_size_t
        sig = {
            "moed_workspace_size": ([S], Z),
            "moed_forward": ([S] + [P] * 13 + [Z, P], ctypes.c_int),
            "moed_forward_q4": ([S, I] + [P] * 15 + [Z, P], ctypes.c_int),
            "moed_selftest_wait_timeout": ([S, I] + [P] * 15 + [Z, ctypes.c_uint64, P], ctypes.c_int),
            "moed_matvec_q4_workspace_size": ([I] * 4, Z),
            "moed_matvec_q4": ([I] * 6 + [P] * 6 + [Z, P], ctypes.c_int),
            "moed_quantize_q4": ([I] * 4 + [P] * 4, ctypes.c_int),
            "moed_dequantize_q4": ([I] * 4 + [P] * 4, ctypes.c_int),
        }
        for name, (args, res) in sig.items():
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, res
        _sig_lib = lib
    return lib


# ------------------------------------------------------------ C ABI names --

def moed_workspace_size(shape: moe_shape) -> int:
    n = int(_lib().moed_workspace_size(ctypes.byref(shape)))
    if n == 0:
        _check(MOE_ERR_UNSUPPORTED)
    return n


def moed_forward(shape, x, w_router, b_router, w1, w2, y, ids, weights, counts, offsets, perm, slot,
                 ws, stream=None):
    p = _args(shape, *_forward_specs(x, w_router, b_router, w1, w2, y, ids, weights, counts, offsets,
                                     perm, slot))
    _check(_lib().moed_forward(ctypes.byref(shape), *p, *_ws(ws), _stream(stream)))


def _q4_ptrs(w, E, K, N, name):
    """(codes, scales) pointers of `w` checked against W [E, K, N] and the
    current device."""
    if (w.E, w.K, w.N) != (E, K, N):
        raise ValueError(f"{name} is [{w.E}, {w.K}, {w.N}]; the shape needs [{E}, {K}, {N}]")
    return (_ptr(w.codes, _I32, f"{name}.codes", E * (K // 8) * N),
            _ptr(w.scales, _BF, f"{name}.scales", E * (K // w.group) * N))


def _q4_layer_ptrs(shape, w1, w2):
    """(w1, w1_scales, w2, w2_scales) pointers of a layer's :class:`Q4Weights`."""
    if w1.group != w2.group:
        raise ValueError(f"w1 has groups of {w1.group} rows, w2 of {w2.group}")
    f1 = 2 * shape.F if shape.expert_act else shape.F
    return _q4_ptrs(w1, shape.E, shape.H, f1, "w1") + _q4_ptrs(w2, shape.E, shape.F, shape.H, "w2")


def moed_forward_q4(shape, x, w_router, b_router, w1, w2, y, ids, weights, counts, offsets, perm, slot,
                    ws, stream=None):
    """moed_forward with w1, w2 as :class:`Q4Weights` of one group size."""
    q = _q4_layer_ptrs(shape, w1, w2)
    specs = _forward_specs(x, w_router, b_router, None, None, y, ids, weights, counts, offsets, perm, slot)
    p = _args(shape, *specs)
    _check(_lib().moed_forward_q4(ctypes.byref(shape), w1.group, *p[:3], *q, *p[5:], *_ws(ws),
                                  _stream(stream)))


def moed_selftest_wait_timeout(shape, x, w_router, b_router, w1, w2, y, ids, weights, counts, offsets, perm,
                               slot, ws, limit_ns: int, stream=None):
    """The layer (w1, w2 tensors or :class:`Q4Weights`) with waits that run out."""
    q4 = isinstance(w1, Q4Weights)
    specs = _forward_specs(x, w_router, b_router, None if q4 else w1, None if q4 else w2, y, ids, weights,
                           counts, offsets, perm, slot)
    p = _args(shape, *specs)
    q = _q4_layer_ptrs(shape, w1, w2) if q4 else (p[3], None, p[4], None)
    _check(_lib().moed_selftest_wait_timeout(ctypes.byref(shape), w1.group if q4 else 0, *p[:3], *q, *p[5:],
                                             *_ws(ws), int(limit_ns), _stream(stream)))


def moed_matvec_q4_workspace_size(rows: int, n_segments: int, K: int, N: int) -> int:
    n = int(_lib().moed_matvec_q4_workspace_size(rows, n_segments, K, N))
    if n == 0:
        _check(MOE_ERR_UNSUPPORTED)
    return n


def moed_matvec_q4(x, w, seg_offsets, y, ws, stream=None):
    """y[r] = x[r] W[i % E] for the rows r of segment i; w a :class:`Q4Weights`;
    seg_offsets None: one segment, all rows."""
    rows = x.shape[0]
    n_segments = 1 if seg_offsets is None else seg_offsets.numel() - 1
    c, s = _q4_ptrs(w, w.E, w.K, w.N, "w")
    _check(_lib().moed_matvec_q4(
        rows, w.K, w.N, w.E, w.group, n_segments, _ptr(x, _BF, "x", rows * w.K), c, s,
        _ptr(seg_offsets, _I32, "seg_offsets", n_segments + 1), _ptr(y, _BF, "y", rows * w.N), *_ws(ws),
        _stream(stream)))


def moed_quantize_q4(w, codes, scales, group: int, stream=None):
    E, K, N = w.shape
    g = int(group) if int(group) > 0 else 1
    _check(_lib().moed_quantize_q4(E, K, N, int(group), _ptr(w, _BF, "w", E * K * N),
                                   _ptr(codes, _I32, "codes", E * (K // 8) * N),
                                   _ptr(scales, _BF, "scales", E * (K // g) * N), _stream(stream)))


def moed_dequantize_q4(w, out, stream=None):
    """out[e, kk, n] = bf16((c - 8) * scale) of a :class:`Q4Weights`."""
    c, s = _q4_ptrs(w, w.E, w.K, w.N, "w")
    _check(_lib().moed_dequantize_q4(w.E, w.K, w.N, w.group, c, s, _ptr(out, _BF, "out", w.E * w.K * w.N),
                                     _stream(stream)))


# --------------------------------------------------------------- helpers --

class Q4Weights:
    """W [E, K, N] in 4 bits with group scales (layout: include/moe_decode.h).

    codes [E, K/8, N] int32, scales [E, K/group, N] bf16; without the leading
    E they describe one matrix (E = 1).  The group size follows from the
    shapes."""

    __slots__ = ("_codes", "_scales", "E", "K", "N", "group", "_device", "_args")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        if codes.dtype != _I32 or scales.dtype != _BF:
            raise TypeError(f"codes must be int32 and scales bfloat16, got {codes.dtype} and {scales.dtype}")
        if codes.dim() == 2 and scales.dim() == 2:
            codes, scales = codes.unsqueeze(0), scales.unsqueeze(0)
        if codes.dim() != 3 or scales.dim() != 3:
            raise ValueError("codes must be [E, K/8, N] and scales [E, K/group, N]")
        E, K8, N = codes.shape
        if scales.shape[0] != E or scales.shape[2] != N or scales.shape[1] == 0 or K8 * 8 % scales.shape[1]:
            raise ValueError(f"scales {tuple(scales.shape)} do not match codes {tuple(codes.shape)}")
        group = K8 * 8 // scales.shape[1]
        if group not in (32, 64, 128):
            raise ValueError(f"groups of {group} rows: 32, 64 or 128 are supported")
        if not (codes.is_contiguous() and scales.is_contiguous()):
            raise ValueError("codes and scales must be contiguous")
        dev = codes.get_device()
        self._set(codes, scales, E, K8 * 8, N, group, dev if scales.get_device() == dev else -1)

    def _set(self, codes, scales, E, K, N, group, dev):
        self._codes, self._scales = codes, scales
        self.E, self.K, self.N, self.group = E, K, N, group
        # what the calls below pass for them
        self._device = dev
        self._args = (codes.data_ptr(), scales.data_ptr())

    def __reduce__(self):  # a copy has addresses of its own
        return Q4Weights, (self._codes, self._scales)

    # fixed for the object's life: the calls use their addresses
    codes = property(lambda self: self._codes)
    scales = property(lambda self: self._scales)


def _on(stream):
    """`stream` (a torch stream or a raw handle) as the current stream."""
    if isinstance(stream, torch.cuda.Stream):
        return torch.cuda.stream(stream)
    return torch.cuda.stream(torch.cuda.ExternalStream(int(stream)))


def _here():
    """(current device, its current stream's handle)."""
    dev = torch.cuda.current_device()
    return dev, torch._C._cuda_getCurrentRawStream(dev)


def _addr(t: torch.Tensor, dtype, name: str, numel: int, dev: int) -> int:
    """Address of `t` after the binding's checks (see check_tensor)."""
    if not (t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and t.numel() >= numel):
        check_tensor(t, dtype, name, numel, dev)
    return t.data_ptr()


def _q4_here(w: Q4Weights, dev: int):
    if w._device != dev:
        raise ValueError(f"the 4-bit weights' codes are on {w.codes.device} and their scales on "
                         f"{w.scales.device}, the current device is cuda:{dev}")
    if (w._codes.data_ptr(), w._scales.data_ptr()) != w._args:
        raise ValueError("the 4-bit weights' tensors were given other memory")
    return w._args


def quantize_q4(w: torch.Tensor, group: int = 128, stream=None) -> Q4Weights:
    """bf16 w [E, K, N] or [K, N] -> :class:`Q4Weights`."""
    if stream is not None:
        with _on(stream):
            return quantize_q4(w, group)
    if w.dim() not in (2, 3):
        raise ValueError(f"w must be [E, K, N] or [K, N], got {tuple(w.shape)}")
    E, K, N = w.shape if w.dim() == 3 else (1, *w.shape)
    if group not in (32, 64, 128) or K % group:
        raise ValueError(f"group = {group}: need 32, 64 or 128, dividing K = {K}")
    dev, raw = _here()
    src = _addr(w, _BF, "w", E * K * N, dev)
    codes = torch.empty((E, K // 8, N), dtype=_I32, device=w.device)
    scales = torch.empty((E, K // group, N), dtype=_BF, device=w.device)
    q = Q4Weights.__new__(Q4Weights)  # of tensors that need no checks
    q._set(codes, scales, E, K, N, group, dev)
    rc = (_sig_lib or _lib()).moed_quantize_q4(E, K, N, group, src, *q._args, raw)
    if rc:
        _check(rc)
    return q


def dequantize_q4(w: Q4Weights, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The bf16 matrices [E, K, N] that `w` stands for."""
    if stream is not None:
        with _on(stream):
            return dequantize_q4(w, out)
    dev, raw = _here()
    q = _q4_here(w, dev)
    E, K, N = w.E, w.K, w.N
    if out is None:
        out = torch.empty((E, K, N), dtype=_BF, device=w._codes.device)
        dst = out.data_ptr()
    else:
        dst = _addr(out, _BF, "out", E * K * N, dev)
    rc = (_sig_lib or _lib()).moed_dequantize_q4(E, K, N, w.group, *q, dst, raw)
    if rc:
        _check(rc)
    return out


# Workspaces of matvec_q4: one per stream, grown as needed.  Calls on one
# stream run one after the other and may share it, if the two kernels of a call
# are enqueued together (the lock); a call that is captured into a CUDA graph
# gets its own.
_matvec_bytes: dict = {}
_matvec_ws: dict = {}
_enqueue = threading.Lock()


def _matvec_workspace(rows: int, n_segments: int, K: int, N: int, dev: int, raw: int) -> torch.Tensor:
    n = _matvec_bytes.get((rows, n_segments))
    if n is None:
        n = _matvec_bytes[rows, n_segments] = moed_matvec_q4_workspace_size(rows, n_segments, K, N)
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(n, dtype=torch.uint8, device=dev)
    ws = _matvec_ws.get((dev, raw))
    if ws is None or ws.numel() < n:
        ws = _matvec_ws[dev, raw] = torch.empty(n, dtype=torch.uint8, device=dev)
    return ws


def matvec_q4(x: torch.Tensor, w: Q4Weights, seg_offsets: torch.Tensor | None = None,
              out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[r] = x[r] W[i % E] for the rows r of segment i (rows [seg_offsets[i],
    seg_offsets[i+1]) of x); without seg_offsets all rows use a single matrix.
    Rows of y outside every segment are not written."""
    if stream is not None:
        with _on(stream):
            return matvec_q4(x, w, seg_offsets, out)
    E, K, N = w.E, w.K, w.N
    if x.dim() != 2 or x.shape[1] != K:
        raise ValueError(f"x must be [rows, {K}], got {tuple(x.shape)}")
    rows = x.shape[0]
    dev, raw = _here()
    if seg_offsets is None:
        if E != 1:
            raise ValueError(f"seg_offsets is needed with {E} matrices")
        n_segments, seg = 1, None
    else:
        if seg_offsets.dim() != 1 or seg_offsets.numel() < 2:
            raise ValueError("seg_offsets must be [n_segments + 1]")
        n_segments = seg_offsets.numel() - 1
        seg = _addr(seg_offsets, _I32, "seg_offsets", n_segments + 1, dev)
    q = _q4_here(w, dev)
    src = _addr(x, _BF, "x", rows * K, dev)
    if out is None:
        out = torch.empty((rows, N), dtype=_BF, device=x.device)
        dst = out.data_ptr()
    else:
        dst = _addr(out, _BF, "out", rows * N, dev)
    with _enqueue:
        ws = _matvec_workspace(rows, n_segments, K, N, dev, raw)
        rc = (_sig_lib or _lib()).moed_matvec_q4(rows, K, N, E, w.group, n_segments, src, *q, seg, dst, ws.data_ptr(),
                                                 ws.numel(), raw)
    if rc:
        _check(rc)
    return out


class _Buffers:
    """Routing outputs of the calls with T tokens on one stream, their workspace
    (`ws`, or a new one) and the call's arguments that stay the same."""

    def __init__(self, layer, T: int, stream: int, ws: torch.Tensor | None):
        shape = layer._shape(T)
        dev = layer.w_router.device
        need = moed_workspace_size(shape)
        self.ws = ws if ws is not None and ws.numel() >= need else torch.empty(need, dtype=torch.uint8, device=dev)
        n, i32 = T * layer.k, dict(dtype=_I32, device=dev)
        self.routing = r = RoutingBuffers(
            ids=torch.empty(T, layer.k, **i32), weights=torch.empty(T, layer.k, dtype=_F32, device=dev),
            counts=torch.empty(layer.E, **i32), offsets=torch.empty(layer.E + 1, **i32),
            perm=torch.empty(n, **i32), slot=torch.empty(T, layer.k, **i32))
        self.shape = shape
        self.head = (ctypes.byref(shape),) + ((layer.w1.group,) if layer.q4 else ())
        self.tail = tuple(ctypes.c_void_p(t.data_ptr()) for t in
                          (r.ids, r.weights, r.counts, r.offsets, r.perm, r.slot, self.ws)) + \
            (ctypes.c_size_t(self.ws.numel()), ctypes.c_void_p(stream))


class MoEDecodeLayer:
    """A layer's weights for decode steps of at most MOED_MAX_TOKENS tokens:
    w1 / w2 as bf16 tensors ([E, H, F] or [E, H, 2F] for "swiglu", [E, F, H])
    or as :class:`Q4Weights`.  Calling it runs moed_forward(_q4) on the current
    stream (or `stream`) and returns a new y [T, H].  What it was made with
    cannot be set later.

    ``routing`` and ``ws`` are those of the last call; the next call with as
    many tokens on the same stream writes the routing again, and the next call
    on the same stream the workspace.  Calls on different streams have buffers
    of their own, and so has every call that is captured into a CUDA graph, so
    they may overlap."""

    def __init__(self, w_router, w1, w2, k: int, bias=None, capacity_factor=None,
                 gating: int = MOE_GATE_TOPK_SOFTMAX, act: str = "gelu"):
        self._q4 = isinstance(w1, Q4Weights)
        if self.q4 != isinstance(w2, Q4Weights):
            raise TypeError("w1 and w2 must both be tensors or both Q4Weights")
        if not self.q4 and w2.dim() != 3:
            raise ValueError(f"w2 must be [E, F, H], got {tuple(w2.shape)}")
        self._E, self._F, self._H = (w2.E, w2.K, w2.N) if self.q4 else w2.shape
        self._k, self._act = int(k), act
        self._capacity_factor, self._gating = capacity_factor, int(gating)
        f1 = 2 * self.F if act == "swiglu" else self.F
        if self.q4:
            if (w1.E, w1.K, w1.N) != (self.E, self.H, f1) or w1.group != w2.group:
                raise ValueError(f"w1 is [{w1.E}, {w1.K}, {w1.N}] in groups of {w1.group}; w2 needs "
                                 f"[{self.E}, {self.H}, {f1}] in groups of {w2.group}")
        elif tuple(w1.shape) != (self.E, self.H, f1):
            raise ValueError(f"w1 is {tuple(w1.shape)}; w2 and act = {act!r} need {(self.E, self.H, f1)}")
        if tuple(w_router.shape) != (self.H, self.E):
            raise ValueError(f"w_router is {tuple(w_router.shape)}, not {(self.H, self.E)}")
        dev = w_router.device.index
        weights = (w1.codes, w1.scales, w2.codes, w2.scales) if self.q4 else (w1, w2)
        types = (_I32, _BF, _I32, _BF) if self.q4 else (_BF, _BF)
        for t, dt, name in ((w_router, _BF, "w_router"), *zip(weights, types, ("w1", "w1", "w2", "w2")
                                                              if self.q4 else ("w1", "w2"))):
            check_tensor(t, dt, name, 0, dev)
        if bias is not None:
            check_tensor(bias, _F32, "bias", self.E, dev)
        self._w_router, self._w1, self._w2, self._bias = w_router, w1, w2, bias
        # aliases, so that the memory stays even if those tensors are given other
        self._held = [t.detach() for t in (w_router, bias, *weights) if t is not None]
        self._device, self._index = w_router.device, dev
        self._ptrs = (ctypes.c_void_p(w_router.data_ptr()),
                      ctypes.c_void_p(None if bias is None else bias.data_ptr()),
                      *(ctypes.c_void_p(t.data_ptr()) for t in weights))
        self._shape(1)
        self._fn = _lib().moed_forward_q4 if self.q4 else _lib().moed_forward
        self._buffers = {}   # (T, stream) -> _Buffers
        self._streams = {}   # stream -> its workspace, as large as any T needed so far
        self._lock = threading.Lock()  # a call's two kernels are enqueued together
        self._last = None

    def __reduce__(self):  # a copy has addresses and buffers of its own
        return MoEDecodeLayer, (self._w_router, self._w1, self._w2, self.k, self._bias, self.capacity_factor,
                                self.gating, self.act)

    # fixed for the layer's life: the calls use the tensors' addresses and keep the
    # shape of every batch size they have seen
    w_router = property(lambda self: self._w_router)
    w1 = property(lambda self: self._w1)
    w2 = property(lambda self: self._w2)
    bias = property(lambda self: self._bias)
    q4 = property(lambda self: self._q4)
    E = property(lambda self: self._E)
    F = property(lambda self: self._F)
    H = property(lambda self: self._H)
    k = property(lambda self: self._k)
    act = property(lambda self: self._act)
    capacity_factor = property(lambda self: self._capacity_factor)
    gating = property(lambda self: self._gating)

    def _shape(self, T: int) -> moe_shape:
        s = make_shape(T, self.H, self.F, self.E, self.k, self.capacity_factor, self.gating, self.act)
        moed_workspace_size(s)  # raises for a shape the operators do not take
        return s

    def __call__(self, x: torch.Tensor, stream=None) -> torch.Tensor:
        if stream is not None:  # as if it were the current stream
            with _on(stream):
                return self(x)
        dev, raw = _here()
        if x.dim() != 2 or x.shape[1] != self._H:
            raise ValueError(f"x must be [T, {self.H}], got {tuple(x.shape)}")
        if self._index != dev:
            raise ValueError(f"the layer's weights are on {self._device}, the current device is cuda:{dev}")
        T = x.shape[0]
        src = _addr(x, _BF, "x", T * self._H, dev)
        y = torch.empty((T, self._H), dtype=_BF, device=self._device)
        capturing = torch.cuda.is_current_stream_capturing()
        with self._lock:
            b = _Buffers(self, T, raw, None) if capturing else self._buffers.get((T, raw)) or self._new(T, raw)
            rc = self._fn(*b.head, src, *self._ptrs, y.data_ptr(), *b.tail)
            self._last = b
        if rc:
            _check(rc)
        return y

    def _new(self, T: int, raw: int) -> _Buffers:
        """Buffers of a first call with T tokens on a stream."""
        b = _Buffers(self, T, raw, self._streams.get(raw))
        if b.ws is not self._streams.get(raw):  # the smaller one goes
            for key in [key for key in self._buffers if key[1] == raw]:
                del self._buffers[key]
            self._streams[raw] = b.ws
        self._buffers[T, raw] = b
        return b

    @property
    def ws(self) -> torch.Tensor:
        """Workspace of the last call (for moe_get_device_status)."""
        return self._last.ws

    @property
    def routing(self) -> RoutingBuffers:
        """Routing outputs of the last call."""
        return self._last.routing
