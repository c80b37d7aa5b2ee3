"""Training operators of the MoE layer: Python binding of include/moe_train.h.

The layer's forward that keeps what its gradients need and the gradients
themselves (:class:`MoETrainLayer`), the same for single steps
(:func:`expert_ffn`, :func:`expert_ffn_backward`, :func:`route_backward`,
:func:`combine_backward`, :func:`dispatch_rows_backward`,
:func:`router_probs`), and activations kept in 8 bits
(:func:`quantize_a8`, :func:`dequantize_a8`).  Gradients are explicit calls, as
every other step of this package; all of them run in the library's CUDA kernels
on the current stream (or `stream`), allocate their outputs and workspace there
and keep nothing between calls.  An output that the caller gives must not overlap
an input (MoEError).
"""
from __future__ import annotations

import ctypes
import functools
import threading
from typing import NamedTuple

import torch

from . import (_BF, _F32, _I32, _check, MOE_ERR_UNSUPPORTED, MOE_GATE_SOFTMAX_TOPK, MOE_GATE_TOPK_SOFTMAX,
               MOE_WS_MIN_BYTES, RoutingBuffers, check_tensor, load_library, make_shape, moe_get_device_status,
               moe_shape)
from .decode import _addr, _here, _on

# Every symbol include/moe_train.h declares.
TRAIN_EXPORTS = ("moet_quantize_a8", "moet_dequantize_a8", "moet_dispatch_rows_backward",
                 "moet_combine_backward", "moet_expert_ffn_workspace_size", "moet_expert_ffn",
                 "moet_expert_ffn_backward_workspace_size", "moet_expert_ffn_backward",
                 "moet_router_probs_workspace_size", "moet_router_probs",
                 "moet_route_backward_workspace_size", "moet_route_backward",
                 "moet_forward_workspace_size", "moet_forward", "moet_backward_workspace_size",
                 "moet_backward")

_I8, _U8 = torch.int8, torch.uint8
_sig_lock = threading.Lock()
_sig_lib = None


def _lib():
    """The library with the training entry points' signatures set."""
    global _sig_lib
    if _sig_lib is not None:
        return _sig_lib
    lib = load_library()
    with _sig_lock:
        P, S, I, Z = ctypes.c_void_p, ctypes.POINTER(moe_shape), ctypes.c_int32, ctypes.c_size_t
        L = ctypes.c_int64
        call = [P, P, Z, P]  # status, ws, ws_bytes, stream
        sig = {
            "moet_quantize_a8": ([L, I] + [P] * 4, ctypes.c_int),
            "moet_dequantize_a8": ([L, I] + [P] * 4, ctypes.c_int),
            "moet_dispatch_rows_backward": ([S] + [P] * 4, ctypes.c_int),
            "moet_combine_backward": ([S] + [P] * 7, ctypes.c_int),
            "moet_expert_ffn_workspace_size": ([S], Z),
            "moet_expert_ffn": ([S, I] + [P] * 7 + call, ctypes.c_int),
            "moet_expert_ffn_backward_workspace_size": ([S], Z),
            "moet_expert_ffn_backward": ([S, I] + [P] * 10 + call, ctypes.c_int),
            "moet_router_probs_workspace_size": ([S], Z),
            "moet_router_probs": ([S] + [P] * 4 + call, ctypes.c_int),
            "moet_route_backward_workspace_size": ([S], Z),
            "moet_route_backward": ([S] + [P] * 9 + call, ctypes.c_int),
            "moet_forward_workspace_size": ([S], Z),
            "moet_forward": ([S, I] + [P] * 17 + call, ctypes.c_int),
            "moet_backward_workspace_size": ([S, I], Z),
            "moet_backward": ([S, I] + [P] * 19 + call, ctypes.c_int),
        }
        for name, (args, res) in sig.items():
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, res
        _sig_lib = lib
    return lib


# ------------------------------------------------------------------- shared --

_status: dict = {}  # device -> the status block of the calls that have no layer


def _status_block(dev: int) -> torch.Tensor:
    return torch.zeros(MOE_WS_MIN_BYTES, dtype=_U8, device=torch.device("cuda", dev))


def _shared_status(dev: int) -> torch.Tensor:
    t = _status.get(dev)
    if t is None:
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("the status block of this device is made by the first call on it, which cannot be "
                               "one that is captured: call train_status() before the capture")
        t = _status_block(dev)
        torch.cuda.synchronize(dev)  # zeroed before a call on any stream
        t = _status.setdefault(dev, t)
    return t


def train_status(stream=None) -> int:
    """Synchronises the stream, returns and clears the status word of this
    module's functions on the current device (0 if all is well).  Raises
    MoEError if a status bit is set.  A layer's calls have a word of their own
    (``moe_get_device_status(layer.status)``)."""
    return moe_get_device_status(_shared_status(torch.cuda.current_device()), stream)


class _Call:
    """A shape as the calls pass it, and the workspace each needs for it."""

    __slots__ = ("shape", "ref", "_sizes")

    def __init__(self, *args):
        self.shape = make_shape(*args)
        self.ref = ctypes.byref(self.shape)
        self._sizes = {}

    def workspace(self, name: str, device, *extra) -> torch.Tensor:
        n = self._sizes.get((name, extra))
        if n is None:
            n = int(getattr(_lib(), name + "_workspace_size")(self.ref, *extra))
            if n == 0:
                _check(MOE_ERR_UNSUPPORTED)
            self._sizes[name, extra] = n
        return torch.empty(n, dtype=_U8, device=device)


# T, H, F, E, k, capacity_factor, gating, act -> _Call
_call = functools.lru_cache(maxsize=1024)(_Call)


@functools.lru_cache(maxsize=64)
def _current_stream(dev: int, raw: int) -> torch.cuda.Stream:
    """torch's object for the current stream, whose handle is `raw` (kept, as making
    one takes longer than the rest of a record_stream: 8 us of a backward's 55)."""
    return torch.cuda.current_stream(dev)


def _out(t, shape, dtype, name: str, dev: int, device) -> torch.Tensor:
    """`t` checked against a shape, or a new tensor of it."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    _addr(t, dtype, name, t.numel(), dev)
    return t


def _shaped(t, shape, dtype, name: str, dev: int) -> int:
    """Address of `t`, which must have just this shape."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    return _addr(t, dtype, name, t.numel(), dev)


# --------------------------------------------------- activations in 8 bits --

class A8Tensor:
    """bf16 values [..., C] kept in 8 bits: codes int8 of that shape and scales
    uint8 [..., ceil(C / 32)], the exponents (biased by 127) of the power of two
    that 32 columns share (layout and rounding: include/moe_train.h)."""

    __slots__ = ("codes", "scales")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        if codes.dtype != _I8 or scales.dtype != _U8:
            raise TypeError(f"codes must be int8 and scales uint8, got {codes.dtype} and {scales.dtype}")
        if codes.dim() < 1 or tuple(scales.shape) != _scales_shape(codes.shape):
            raise ValueError(f"scales {tuple(scales.shape)} do not match codes {tuple(codes.shape)}")
        self.codes, self.scales = codes, scales

    @property
    def shape(self):
        return self.codes.shape


def _scales_shape(shape):
    return *shape[:-1], -(-shape[-1] // 32)


def _a8_new(shape, device) -> A8Tensor:
    q = A8Tensor.__new__(A8Tensor)
    q.codes = torch.empty(shape, dtype=_I8, device=device)
    q.scales = torch.empty(_scales_shape(shape), dtype=_U8, device=device)
    return q


def _matrix(shape):
    """(rows, columns) of a tensor as the 8-bit calls take it."""
    n = 1
    for v in shape[:-1]:
        n *= v
    if shape[-1] >= 2 ** 31:  # ctypes would drop the upper bits
        raise ValueError(f"a last dimension of {shape[-1]}: it must be below 2^31")
    return n, shape[-1]


def quantize_a8(x: torch.Tensor, stream=None) -> A8Tensor:
    """bf16 x [..., C] (C % 8 == 0) -> :class:`A8Tensor`."""
    if stream is not None:
        with _on(stream):
            return quantize_a8(x)
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    dev, raw = _here()
    rows, cols = _matrix(x.shape)
    src = _addr(x, _BF, "x", x.numel(), dev)
    q = _a8_new(tuple(x.shape), x.device)
    rc = _lib().moet_quantize_a8(rows, cols, src, q.codes.data_ptr(), q.scales.data_ptr(), raw)
    if rc:
        _check(rc)
    return q


def dequantize_a8(q: A8Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The bf16 values that `q` stands for."""
    if stream is not None:
        with _on(stream):
            return dequantize_a8(q, out)
    dev, raw = _here()
    rows, cols = _matrix(q.shape)
    codes = _addr(q.codes, _I8, "codes", q.codes.numel(), dev)
    scales = _shaped(q.scales, _scales_shape(q.shape), _U8, "scales", dev)
    out = _out(out, q.codes.shape, _BF, "out", dev, q.codes.device)
    rc = _lib().moet_dequantize_a8(rows, cols, codes, scales, out.data_ptr(), raw)
    if rc:
        _check(rc)
    return out


def _kept_ptrs(z, shape, name: str, dev: int):
    """(keep_bits, address, scales' address) of bf16 values or an A8Tensor."""
    if isinstance(z, A8Tensor):
        a = _shaped(z.codes, shape, _I8, f"{name}.codes", dev)
        return 8, a, _shaped(z.scales, _scales_shape(shape), _U8, f"{name}.scales", dev)
    return 16, _shaped(z, shape, _BF, name, dev), None


# ------------------------------------------------------- rows there and back --

def _slot_shape(rows: torch.Tensor, slot: torch.Tensor, name: str) -> _Call:
    if slot.dim() != 2:
        raise ValueError(f"slot must be [T, k], got {tuple(slot.shape)}")
    T, k = slot.shape
    if rows.dim() != 2 or rows.shape[0] < T * k:
        raise ValueError(f"{name} must be [T * k, H] with T * k = {T * k}, got {tuple(rows.shape)}")
    return _call(T, rows.shape[1], 8, max(k, 1), k)


def dispatch_rows_backward(dxp: torch.Tensor, slot: torch.Tensor, out: torch.Tensor | None = None,
                           stream=None) -> torch.Tensor:
    """The gradient of moe_dispatch_rows: dx[t] = sum of dxp[slot[t, j]] over
    the kept slots (slot >= 0); dxp [T * k, H] in dispatch order."""
    if stream is not None:
        with _on(stream):
            return dispatch_rows_backward(dxp, slot, out)
    c = _slot_shape(dxp, slot, "dxp")
    dev, raw = _here()
    src, sl = _addr(dxp, _BF, "dxp", dxp.numel(), dev), _addr(slot, _I32, "slot", slot.numel(), dev)
    out = _out(out, (c.shape.T, c.shape.H), _BF, "out", dev, dxp.device)
    rc = _lib().moet_dispatch_rows_backward(c.ref, src, sl, out.data_ptr(), raw)
    if rc:
        _check(rc)
    return out


def combine_backward(dy: torch.Tensor, Y: torch.Tensor, weights: torch.Tensor, slot: torch.Tensor,
                     dY: torch.Tensor | None = None, dweights: torch.Tensor | None = None, stream=None):
    """The gradients of moe_combine, (dY, dweights): dY[slot[t, j]] =
    weights[t, j] dy[t], dweights[t, j] = <dy[t], Y[slot[t, j]]>, 0 for a dropped
    slot.  Rows of dY that no slot names are not written."""
    if stream is not None:
        with _on(stream):
            return combine_backward(dy, Y, weights, slot, dY, dweights)
    c = _slot_shape(Y, slot, "Y")
    s = c.shape
    dev, raw = _here()
    p = (_shaped(dy, (s.T, s.H), _BF, "dy", dev), _addr(Y, _BF, "Y", Y.numel(), dev),
         _shaped(weights, (s.T, s.k), _F32, "weights", dev), _addr(slot, _I32, "slot", slot.numel(), dev))
    dY = _out(dY, Y.shape, _BF, "dY", dev, Y.device)
    dweights = _out(dweights, (s.T, s.k), _F32, "dweights", dev, Y.device)
    rc = _lib().moet_combine_backward(c.ref, *p, dY.data_ptr(), dweights.data_ptr(), raw)
    if rc:
        _check(rc)
    return dY, dweights


# ------------------------------------------------------------- experts' FFN --

def _ffn_shape(xp, w1, w2, act: str) -> _Call:
    if w2.dim() != 3:
        raise ValueError(f"w2 must be [E, F, H], got {tuple(w2.shape)}")
    E, F, H = w2.shape
    if xp.dim() != 2 or xp.shape[1] != H:
        raise ValueError(f"xp must be [rows, {H}], got {tuple(xp.shape)}")
    c = _call(xp.shape[0], H, F, E, 1, None, MOE_GATE_TOPK_SOFTMAX, act)
    f1 = 2 * F if c.shape.expert_act else F
    if tuple(w1.shape) != (E, H, f1):
        raise ValueError(f"w1 must be {(E, H, f1)} for act = {act!r}, got {tuple(w1.shape)}")
    return c


def _z_shape(rows: int, s: moe_shape):
    return (rows, 2, s.F) if s.expert_act else (rows, s.F)


def expert_ffn(xp: torch.Tensor, w1: torch.Tensor, w2: torch.Tensor, offsets: torch.Tensor, act: str = "gelu",
               keep_bits: int = 16, stream=None):
    """The experts' FFN on rows grouped by expert (rows [offsets[e], offsets[e + 1])
    of xp belong to expert e): (Y, z), z the pre-activations xp W1 for the
    backward pass, bf16 (keep_bits 16) or :class:`A8Tensor` (8), of shape
    [rows, F] or [rows, 2, F] for "swiglu".  Rows outside every segment are not
    written."""
    if stream is not None:
        with _on(stream):
            return expert_ffn(xp, w1, w2, offsets, act, keep_bits)
    c = _ffn_shape(xp, w1, w2, act)
    s, d = c.shape, xp.device
    dev, raw = _here()
    rows = xp.shape[0]
    p = (_addr(xp, _BF, "xp", xp.numel(), dev), _addr(w1, _BF, "w1", w1.numel(), dev),
         _addr(w2, _BF, "w2", w2.numel(), dev), _shaped(offsets, (s.E + 1,), _I32, "offsets", dev))
    Y = torch.empty((rows, s.H), dtype=_BF, device=d)
    if keep_bits == 8:
        z = _a8_new(_z_shape(rows, s), d)
        zp = z.codes.data_ptr(), z.scales.data_ptr()
    else:
        z = torch.empty(_z_shape(rows, s), dtype=_BF, device=d)
        zp = z.data_ptr(), None
    lib = _lib()
    ws = c.workspace("moet_expert_ffn", d)
    rc = lib.moet_expert_ffn(c.ref, keep_bits, *p, Y.data_ptr(), *zp, _shared_status(dev).data_ptr(),
                             ws.data_ptr(), ws.numel(), raw)
    if rc:
        _check(rc)
    return Y, z


def expert_ffn_backward(xp: torch.Tensor, z, w1: torch.Tensor, w2: torch.Tensor, offsets: torch.Tensor,
                        dY: torch.Tensor, act: str = "gelu", stream=None):
    """The gradients of :func:`expert_ffn`, (dxp, dw1, dw2), from its inputs, the
    kept z and dY.  Rows of dxp outside every segment are not written; experts
    without rows get zeros."""
    if stream is not None:
        with _on(stream):
            return expert_ffn_backward(xp, z, w1, w2, offsets, dY, act)
    c = _ffn_shape(xp, w1, w2, act)
    s, d = c.shape, xp.device
    dev, raw = _here()
    rows = xp.shape[0]
    bits, zp, zs = _kept_ptrs(z, _z_shape(rows, s), "z", dev)
    src = _addr(xp, _BF, "xp", xp.numel(), dev)
    p = (_addr(w1, _BF, "w1", w1.numel(), dev), _addr(w2, _BF, "w2", w2.numel(), dev),
         _shaped(offsets, (s.E + 1,), _I32, "offsets", dev), _shaped(dY, (rows, s.H), _BF, "dY", dev))
    dxp, dw1, dw2 = (torch.empty(t.shape, dtype=_BF, device=d) for t in (xp, w1, w2))
    lib = _lib()
    ws = c.workspace("moet_expert_ffn_backward", d)
    rc = lib.moet_expert_ffn_backward(c.ref, bits, src, zp, zs, *p, dxp.data_ptr(), dw1.data_ptr(),
                                      dw2.data_ptr(), _shared_status(dev).data_ptr(), ws.data_ptr(), ws.numel(), raw)
    if rc:
        _check(rc)
    return dxp, dw1, dw2


# ---------------------------------------------------------- router and gate --

def _route_shape(x, w_router, k: int, gating: int) -> _Call:
    if w_router.dim() != 2:
        raise ValueError(f"w_router must be [H, E], got {tuple(w_router.shape)}")
    H, E = w_router.shape
    if x.dim() != 2 or x.shape[1] != H:
        raise ValueError(f"x must be [T, {H}], got {tuple(x.shape)}")
    return _call(x.shape[0], H, 8, E, k, None, gating)


def router_probs(x: torch.Tensor, w_router: torch.Tensor, bias: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """softmax(x W_router + bias) over all experts, fp32 [T, E]: what the
    gradient of MOE_GATE_SOFTMAX_TOPK needs of the forward."""
    if stream is not None:
        with _on(stream):
            return router_probs(x, w_router, bias)
    c = _route_shape(x, w_router, 1, MOE_GATE_TOPK_SOFTMAX)
    s = c.shape
    dev, raw = _here()
    p = (_addr(x, _BF, "x", x.numel(), dev), _addr(w_router, _BF, "w_router", w_router.numel(), dev),
         None if bias is None else _shaped(bias, (s.E,), _F32, "bias", dev))
    probs = torch.empty((s.T, s.E), dtype=_F32, device=x.device)
    lib = _lib()
    ws = c.workspace("moet_router_probs", x.device)
    rc = lib.moet_router_probs(c.ref, *p, probs.data_ptr(), _shared_status(dev).data_ptr(),
                               ws.data_ptr(), ws.numel(), raw)
    if rc:
        _check(rc)
    return probs


def route_backward(x: torch.Tensor, w_router: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor,
                   dweights: torch.Tensor, gating: int = MOE_GATE_TOPK_SOFTMAX,
                   probs: torch.Tensor | None = None, stream=None):
    """The gradients of router and gate, (dx, dw_router, dbias), from those of the
    gate weights [T, k]: dx the router's part alone, dbias that of a router bias.
    probs (:func:`router_probs`) is needed for MOE_GATE_SOFTMAX_TOPK."""
    if stream is not None:
        with _on(stream):
            return route_backward(x, w_router, ids, weights, dweights, gating, probs)
    if ids.dim() != 2:
        raise ValueError(f"ids must be [T, k], got {tuple(ids.shape)}")
    c = _route_shape(x, w_router, ids.shape[1], gating)
    s, d = c.shape, x.device
    dev, raw = _here()
    tk = (s.T, s.k)
    if gating == MOE_GATE_SOFTMAX_TOPK:
        if probs is None:
            raise ValueError("MOE_GATE_SOFTMAX_TOPK needs probs")
        pp = _shaped(probs, (s.T, s.E), _F32, "probs", dev)
    else:
        pp = None
    p = (_addr(x, _BF, "x", x.numel(), dev), _addr(w_router, _BF, "w_router", w_router.numel(), dev),
         _shaped(ids, tk, _I32, "ids", dev), _shaped(weights, tk, _F32, "weights", dev), pp,
         _shaped(dweights, tk, _F32, "dweights", dev))
    dx = torch.empty(x.shape, dtype=_BF, device=d)
    dw = torch.empty(w_router.shape, dtype=_BF, device=d)
    db = torch.empty(s.E, dtype=_F32, device=d)
    lib = _lib()
    ws = c.workspace("moet_route_backward", d)
    rc = lib.moet_route_backward(c.ref, *p, dx.data_ptr(), dw.data_ptr(), db.data_ptr(),
                                 _shared_status(dev).data_ptr(), ws.data_ptr(), ws.numel(), raw)
    if rc:
        _check(rc)
    return dx, dw, db


# ---------------------------------------------------------------- the layer --

class Gradients(NamedTuple):
    """What :meth:`MoETrainLayer.backward` returns; dbias is None unless asked for."""
    dx: torch.Tensor
    dw_router: torch.Tensor
    dbias: torch.Tensor | None
    dw1: torch.Tensor
    dw2: torch.Tensor


def _version(t: torch.Tensor):
    return None if t.is_inference() else t._version


class Saved:
    """What a forward keeps for its backward: z and, with keep_bits 8, x in 8
    bits (else x itself), the routing (``routing``) and, for
    MOE_GATE_SOFTMAX_TOPK, the router's probabilities."""

    __slots__ = ("call", "x", "z", "probs", "versions", "_block", "_stream")

    def _tensors(self):
        """What the forward allocated."""
        ts = [self._block]
        for t in (self.z, self.x, self.probs):
            if isinstance(t, A8Tensor):
                ts += [t.codes, t.scales]
            elif t is not None and t is not self.x:
                ts.append(t)
        return ts

    # ids, perm, slot, gate weights, counts and offsets in one block of 32-bit
    # words, each on a 16-byte boundary
    @staticmethod
    def _layout(T: int, k: int, E: int):
        n4, e4 = (T * k + 3) // 4 * 4, (E + 4) // 4 * 4
        return 0, n4, 2 * n4, 3 * n4, 4 * n4, 4 * n4 + e4, 4 * n4 + 2 * e4

    def _addresses(self):
        """Of ids, perm, slot, weights, counts, offsets."""
        s, a = self.call.shape, self._block.data_ptr()
        return [a + 4 * o for o in self._layout(s.T, s.k, s.E)[:6]]

    @property
    def routing(self) -> RoutingBuffers:
        s, b = self.call.shape, self._block
        n, (o_ids, o_perm, o_slot, o_w, o_cnt, o_off, _) = s.T * s.k, self._layout(s.T, s.k, s.E)
        tk = (s.T, s.k)
        return RoutingBuffers(ids=b[o_ids:o_ids + n].view(tk), weights=b[o_w:o_w + n].view(_F32).view(tk),
                              counts=b[o_cnt:o_cnt + s.E], offsets=b[o_off:o_off + s.E + 1], perm=b[o_perm:o_perm + n],
                              slot=b[o_slot:o_slot + n].view(tk))

    @property
    def shape(self) -> moe_shape:
        """For the moe_* functions (a copy)."""
        return moe_shape.from_buffer_copy(self.call.shape)

    def nbytes(self) -> int:
        """Device bytes held (x itself not counted with keep_bits 16)."""
        return sum(t.numel() * t.element_size() for t in self._tensors())


class MoETrainLayer:
    """A layer's weights for training: bf16 w_router [H, E], w1 [E, H, F] ([E, H,
    2F] = [gate | up] for "swiglu"), w2 [E, F, H] and an optional fp32 bias [E]
    on the logits, all updated in place by the caller's optimizer.

    ``y, saved = layer(x)`` runs the forward and keeps what its gradients need, in
    16 or in 8 bits (`keep_bits`); ``layer.backward(saved, dy)`` returns
    :class:`Gradients`.  A `saved` may be used once or several times, as long as
    x (with keep_bits 16) and the weights are what they were.  Both calls run on
    the current stream (or `stream`), allocate what they return and their
    workspace, and may be captured into CUDA graphs; several forwards may be in
    flight before their backwards.  The layer itself is made outside a capture (it
    waits for its status block).  ``moe_get_device_status(layer.status)`` reads the
    device status of all calls so far."""

    def __init__(self, w_router, w1, w2, k: int, bias=None, capacity_factor=None,
                 gating: int = MOE_GATE_TOPK_SOFTMAX, act: str = "gelu", keep_bits: int = 16):
        if w2.dim() != 3:
            raise ValueError(f"w2 must be [E, F, H], got {tuple(w2.shape)}")
        if keep_bits not in (8, 16):
            raise ValueError(f"keep_bits = {keep_bits}: 8 or 16")
        if torch.cuda.is_available() and torch.cuda.is_current_stream_capturing():
            raise RuntimeError("a layer is made outside a capture: it waits for its status block")
        self.E, self.F, self.H = w2.shape
        self.k, self.act, self.keep_bits = int(k), act, int(keep_bits)
        self.capacity_factor, self.gating = capacity_factor, int(gating)
        self.w_router, self.w1, self.w2, self.bias = w_router, w1, w2, bias
        s = self._call(1).shape
        dev = w_router.device.index
        for (t, dt, shape, name) in self._params(s):
            check_tensor(t, dt, name, 0, dev)
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} must be {shape}, got {tuple(t.shape)}")
        if int(_lib().moet_forward_workspace_size(ctypes.byref(s))) == 0:
            _check(MOE_ERR_UNSUPPORTED)
        self.status = _status_block(dev)
        torch.cuda.synchronize(dev)  # zeroed before a call on any stream

    def _params(self, s):
        f1 = 2 * self.F if s.expert_act else self.F
        p = [(self.w_router, _BF, (self.H, self.E), "w_router"), (self.w1, _BF, (self.E, self.H, f1), "w1"),
             (self.w2, _BF, (self.E, self.F, self.H), "w2")]
        if self.bias is not None:
            p.append((self.bias, _F32, (self.E,), "bias"))
        return p

    def _call(self, T: int) -> _Call:
        return _call(T, self.H, self.F, self.E, self.k, self.capacity_factor, self.gating, self.act)

    def _weights(self, s, dev: int):
        """Addresses of w_router, w1, w2 and the bias (or None)."""
        b = None if self.bias is None else _shaped(self.bias, (self.E,), _F32, "bias", dev)
        return (_shaped(self.w_router, (self.H, self.E), _BF, "w_router", dev),
                _shaped(self.w1, (self.E, self.H, 2 * self.F if s.expert_act else self.F), _BF, "w1", dev),
                _shaped(self.w2, (self.E, self.F, self.H), _BF, "w2", dev), b)

    def __call__(self, x: torch.Tensor, stream=None):
        """(y, saved)"""
        if stream is not None:
            with _on(stream):
                return self(x)
        if x.dim() != 2 or x.shape[1] != self.H:
            raise ValueError(f"x must be [T, {self.H}], got {tuple(x.shape)}")
        dev, raw = _here()
        T, d = x.shape[0], x.device
        c = self._call(T)
        s = c.shape
        wr, w1, w2, b = self._weights(s, dev)
        src = _addr(x, _BF, "x", T * self.H, dev)
        ws = c.workspace("moet_forward", d)
        y = torch.empty((T, self.H), dtype=_BF, device=d)
        v = Saved()
        v.call, v.probs, v._stream = c, None, raw
        v._block = torch.empty(v._layout(T, self.k, self.E)[-1], dtype=_I32, device=d)
        ids, perm, slot, weights, counts, offsets = v._addresses()
        if self.keep_bits == 8:
            v.z, v.x = _a8_new(_z_shape(T * self.k, s), d), _a8_new((T, self.H), d)
            kept = v.z.codes.data_ptr(), v.z.scales.data_ptr(), v.x.codes.data_ptr(), v.x.scales.data_ptr()
        else:
            v.z, v.x = torch.empty(_z_shape(T * self.k, s), dtype=_BF, device=d), x
            kept = v.z.data_ptr(), None, None, None
        if self.gating == MOE_GATE_SOFTMAX_TOPK:
            v.probs = torch.empty((T, self.E), dtype=_F32, device=d)
        v.versions = self._versions(v)
        rc = _lib().moet_forward(c.ref, self.keep_bits, src, wr, b, w1, w2, y.data_ptr(), ids, weights, counts,
                                 offsets, perm, slot, *kept, None if v.probs is None else v.probs.data_ptr(),
                                 self.status.data_ptr(), ws.data_ptr(), ws.numel(), raw)
        if rc:
            _check(rc)
        return y, v

    def _versions(self, saved):
        ts = [self.w_router, self.w1, self.w2]
        if not isinstance(saved.x, A8Tensor):
            ts.append(saved.x)
        return [(t.data_ptr(), _version(t)) for t in ts]

    def backward(self, saved: Saved, dy: torch.Tensor, bias_grad: bool = False, stream=None) -> Gradients:
        """The gradients of the forward that `saved` comes from, for the gradient
        dy [T, H] of its y; bias_grad: dbias too (fp32 [E])."""
        if stream is not None:
            with _on(stream):
                return self.backward(saved, dy, bias_grad)
        if not isinstance(saved, Saved):
            raise TypeError("saved must be what a forward of this layer returned")
        c, s = saved.call, saved.call.shape
        if (s.H, s.F, s.E, s.k) != (self.H, self.F, self.E, self.k):
            raise ValueError("saved is of a layer of another shape")
        if self._versions(saved) != saved.versions:
            raise ValueError("x or a weight was changed or replaced after the forward that saved is of")
        dev, raw = _here()
        wr, w1, w2, _ = self._weights(s, dev)
        g = _shaped(dy, (s.T, s.H), _BF, "dy", dev)
        bits, zp, zs = _kept_ptrs(saved.z, _z_shape(s.T * s.k, s), "z", dev)
        x_bits, xp, xs = _kept_ptrs(saved.x, (s.T, s.H), "x", dev)
        if x_bits != bits:
            raise ValueError(f"z is kept in {bits} bits and x in {x_bits}")
        probs = None
        if s.gating == MOE_GATE_SOFTMAX_TOPK:
            probs = _shaped(saved.probs, (s.T, s.E), _F32, "probs", dev)
        ids, perm, slot, weights, _, offsets = saved._addresses()
        d = dy.device
        ws = c.workspace("moet_backward", d, bits)
        out = Gradients(torch.empty((s.T, s.H), dtype=_BF, device=d), torch.empty_like(self.w_router),
                        torch.empty(s.E, dtype=_F32, device=d) if bias_grad else None,
                        torch.empty_like(self.w1), torch.empty_like(self.w2))
        rc = _lib().moet_backward(c.ref, bits, g, xp, xs, wr, w1, w2, ids, weights, offsets, perm, slot, zp, zs,
                                  probs, out.dx.data_ptr(), out.dw_router.data_ptr(),
                                  None if out.dbias is None else out.dbias.data_ptr(), out.dw1.data_ptr(),
                                  out.dw2.data_ptr(), self.status.data_ptr(), ws.data_ptr(), ws.numel(), raw)
        if rc:
            _check(rc)
        # Not given out again before this call has run: what the forward allocated, if that was on another stream, and
        # x, whatever stream it was made on (it may be saved's alone by now; a no-op on its own stream).
        if bits == 16:
            saved.x.record_stream(_current_stream(dev, raw))
        if raw != saved._stream:
            for t in saved._tensors():
                t.record_stream(_current_stream(dev, raw))
        return out
