"""Python entry points of include/hcmix_experts.h, with the C ABI's names.

The experts' feed-forward network on rows sorted by expert, between
`sublayer.hc_mix_expert_dispatch` and `sublayer.hc_mix_expert_combine`: products
of each expert's rows with its weights (gated too), their gradients, and the
same products with weights of 4 bits for serving single tokens.

As in `sublayer`: argument marshalling only, outputs are allocated here (or given
with `out`), a call goes to the current stream of its tensors' device unless
`stream` says otherwise, a non-OK status raises HcMixError, and results carry no
autograd graph.  There is no CPU fallback.

Rows are 2-D CUDA tensors of bf16 or fp16 (the gate's gradient: fp32 too) with unit
inner stride; weights are 3-D of the same type, [expert, ., .], with unit inner
stride and any stride between rows and experts that leaves them apart.  `offsets`
is int32 [E + 1], as `sublayer.hc_mix_expert_sort` gives it.

A product whose kernel gives up a wait leaves its results incomplete, and no call says
so: ask hc_mix_expert_device_status where the host waits for the results anyway.
"""
from __future__ import annotations

import ctypes
import threading

import torch

from . import binding
from .binding import _check
from .sublayer import TYPES, _device, _like, _matrix, _output, _ptr, _stream, _there

# every symbol include/hcmix_experts.h declares
EXPORTS = ("hc_mix_expert_product", "hc_mix_expert_product_gated",
           "hc_mix_expert_product_weight_backward", "hc_mix_expert_gate_backward",
           "hc_mix_expert_product_q4", "hc_mix_expert_device_status")

_lib = None
_lock = threading.Lock()
_empty = torch.empty
_I32, _U8 = torch.int32, torch.uint8


def lib() -> ctypes.CDLL:
    """libhcmix.so with the argument types of this module's entry points set."""
    global _lib
    if _lib is None:
        with _lock:
            L = binding.lib()
            P, N, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
            args = {
                "hc_mix_expert_product": [P, N, I, N, N, N, P, N, N, I, P, N, P, P],
                "hc_mix_expert_product_gated": [P, N, I, N, N, N, P, N, N, I, P, N, P, P, P],
                "hc_mix_expert_product_weight_backward": [P, N, P, N, I, N, N, N, I, P, N, P, I, P],
                "hc_mix_expert_gate_backward": [P, N, P, N, I, N, N, P, P],
                "hc_mix_expert_product_q4": [P, N, I, N, N, N, P, P, N, I, P, N, P, P],
                "hc_mix_expert_device_status": [P],
            }
            for name in EXPORTS:
                f = getattr(L, name)
                f.argtypes = args[name]
                f.restype = I
            _lib = L
    return _lib


def _weight(w, dtype, device, width: int, transposed: bool):
    """(pointer, row stride, expert stride, experts, features) of W[E, features, width], or
    transposed [E, width, features]."""
    if w.dtype is not dtype or w.device != device or w.dim() != 3:
        raise ValueError("weight must be 3-D of the type and device of the rows")
    E, outer, inner = w.shape
    if (outer if transposed else inner) != width:
        raise ValueError(f"weight of shape {tuple(w.shape)} does not fit rows of width {width}"
                         + (" (transposed)" if transposed else ""))
    expert, row, one = w.stride()
    if one != 1 and inner > 1:
        raise ValueError("weight must have unit inner stride")
    if outer <= 1 and row < inner:
        row = inner
    return w.data_ptr(), row, expert, E, inner if transposed else outer


def _experts(offsets, device, E=None):
    """(pointer, experts)"""
    if (offsets.dtype is not _I32 or offsets.dim() != 1 or offsets.device != device
            or not offsets.is_contiguous() or offsets.shape[0] < 2):
        raise ValueError("offsets must be contiguous int32 of shape (E + 1,) on the device of the "
                         "rows")
    n = offsets.shape[0] - 1
    if E is not None and E != n:
        raise ValueError(f"offsets are of {n} experts, the weights of {E}")
    return offsets.data_ptr(), n


def hc_mix_expert_product(xs: torch.Tensor, weight: torch.Tensor, offsets: torch.Tensor,
                          transposed: bool = False, out=None, stream=None) -> torch.Tensor:
    """ys[R, N]: each row of xs[R, K] times its expert's weight[E, N, K] (with `transposed`
    weight[E, K, N]); rows from offsets[E] on are zero.  dxs of dys[R, N] is the same call
    on dys with the other `transposed`."""
    px, sx, code, R, K, dtype, device = _matrix(xs, "xs")
    if stream is not None or device.index != _device():
        return _there(stream, device, hc_mix_expert_product, xs, weight, offsets, transposed, out)
    pw, row, expert, E, N = _weight(weight, dtype, device, K, transposed)
    po, E = _experts(offsets, device, E)
    ys = _output(out, (R, N), dtype, device)
    st = lib().hc_mix_expert_product(px, sx, code, R, K, N, pw, row, expert, transposed, po, E,
                                     ys.data_ptr(), _stream(xs))
    if st:
        _check(st, "hc_mix_expert_product")
    return ys


def hc_mix_expert_product_gated(xs: torch.Tensor, weight: torch.Tensor, offsets: torch.Tensor,
                                transposed: bool = False, want_saved: bool = False, out=None,
                                stream=None):
    """h[R, F] = silu(g) * u with (g, u) the halves of hc_mix_expert_product's rows, for
    weight[E, 2 * F, K] (with `transposed` [E, K, 2 * F]); with want_saved (h, gu[R, 2 * F]),
    for hc_mix_expert_gate_backward."""
    px, sx, code, R, K, dtype, device = _matrix(xs, "xs")
    if stream is not None or device.index != _device():
        return _there(stream, device, hc_mix_expert_product_gated, xs, weight, offsets, transposed,
                      want_saved, out)
    pw, row, expert, E, N = _weight(weight, dtype, device, K, transposed)
    if N % 2:
        raise ValueError("a gated product's weight has an even number of features")
    po, E = _experts(offsets, device, E)
    h = _output(out, (R, N // 2), dtype, device)
    gu = _empty((R, N), dtype=dtype, device=device) if want_saved else None
    st = lib().hc_mix_expert_product_gated(px, sx, code, R, K, N // 2, pw, row, expert, transposed,
                                           po, E, h.data_ptr(), _ptr(gu), _stream(xs))
    if st:
        _check(st, "hc_mix_expert_product_gated")
    return (h, gu) if want_saved else h


def hc_mix_expert_product_weight_backward(dys: torch.Tensor, xs: torch.Tensor,
                                          offsets: torch.Tensor, transposed: bool = False,
                                          weight_dtype=None, out=None, stream=None) -> torch.Tensor:
    """dweight[E, N, K] (with `transposed` [E, K, N]) of hc_mix_expert_product for dys[R, N]
    and xs[R, K], of the rows' type or, with weight_dtype=torch.float32, fp32; zero for an
    expert without rows."""
    px, sx, code, R, K, dtype, device = _matrix(xs, "xs")
    if stream is not None or device.index != _device():
        return _there(stream, device, hc_mix_expert_product_weight_backward, dys, xs, offsets,
                      transposed, weight_dtype, out)
    if dys.dim() != 2:
        raise ValueError("dys must be 2-D")
    N = dys.shape[1]
    pd, sd = _like(dys, "dys", (R, N), dtype, device)
    po, E = _experts(offsets, device)
    to = dtype if weight_dtype is None else weight_dtype
    if to is not dtype and to is not torch.float32:
        raise ValueError("weight_dtype must be the rows' type or torch.float32")
    dweight = _output(out, (E, K, N) if transposed else (E, N, K), to, device)
    st = lib().hc_mix_expert_product_weight_backward(pd, sd, px, sx, code, R, K, N, transposed, po,
                                                     E, dweight.data_ptr(), TYPES[to], _stream(xs))
    if st:
        _check(st, "hc_mix_expert_product_weight_backward")
    return dweight


def hc_mix_expert_product_backward(dys: torch.Tensor, xs: torch.Tensor, weight: torch.Tensor,
                                   offsets: torch.Tensor, transposed: bool = False,
                                   weight_dtype=None, stream=None):
    """(dxs[R, K], dweight) of hc_mix_expert_product, dweight of weight's shape: a call of
    hc_mix_expert_product and one of hc_mix_expert_product_weight_backward."""
    _, _, _, R, K, dtype, device = _matrix(xs, "xs")
    if stream is not None or device.index != _device():
        return _there(stream, device, hc_mix_expert_product_backward, dys, xs, weight, offsets,
                      transposed, weight_dtype)
    _, _, _, E, N = _weight(weight, dtype, device, K, transposed)
    _like(dys, "dys", (R, N), dtype, device)
    dxs = hc_mix_expert_product(dys, weight, offsets, not transposed)
    return dxs, hc_mix_expert_product_weight_backward(dys, xs, offsets, transposed, weight_dtype)


def hc_mix_expert_gate_backward(dh: torch.Tensor, gu: torch.Tensor, out=None,
                                stream=None) -> torch.Tensor:
    """dgu[R, 2 * F] of h = silu(g) * u for dh[R, F] and gu[R, 2 * F] = (g, u)."""
    pd, sd, code, R, F, dtype, device = _matrix(dh, "dh")
    if stream is not None or device.index != _device():
        return _there(stream, device, hc_mix_expert_gate_backward, dh, gu, out)
    pg, sg = _like(gu, "gu", (R, 2 * F), dtype, device)
    dgu = _output(out, (R, 2 * F), dtype, device)
    st = lib().hc_mix_expert_gate_backward(pd, sd, pg, sg, code, R, F, dgu.data_ptr(), _stream(dh))
    if st:
        _check(st, "hc_mix_expert_gate_backward")
    return dgu


def hc_mix_expert_product_q4(xs: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                             offsets: torch.Tensor, gated: bool = False, out=None,
                             stream=None) -> torch.Tensor:
    """hc_mix_expert_product (with `gated` hc_mix_expert_product_gated) with weights of 4 bits,
    w = (code - 8) * scale: codes[E, N, K // 2] uint8, the lower four bits of a byte for the
    even k, and scales[E, N, K // group] of xs's type, both contiguous; group is 32, 64, 128
    or 256.  Meant for up to eight rows an expert: with more, hc_mix_expert_product with weights of
    16 bits takes less time."""
    px, sx, code, R, K, dtype, device = _matrix(xs, "xs")
    if stream is not None or device.index != _device():
        return _there(stream, device, hc_mix_expert_product_q4, xs, codes, scales, offsets, gated,
                      out)
    if (codes.dtype is not _U8 or codes.dim() != 3 or codes.device != device
            or not codes.is_contiguous() or K % 2 or codes.shape[2] * 2 != K):
        raise ValueError(f"codes must be contiguous uint8 of shape (E, N, {K} // 2) on the device "
                         "of the rows")
    E, N, _ = codes.shape
    if (scales.dtype is not dtype or scales.dim() != 3 or scales.device != device
            or not scales.is_contiguous() or scales.shape[:2] != codes.shape[:2]
            or scales.shape[2] == 0 or K % scales.shape[2]):
        raise ValueError(f"scales must be contiguous of xs's type and of shape ({E}, {N}, K // "
                         "group) on the device of the rows")
    if gated and N % 2:
        raise ValueError("a gated product's weight has an even number of features")
    po, E = _experts(offsets, device, E)
    ys = _output(out, (R, N // 2 if gated else N), dtype, device)
    st = lib().hc_mix_expert_product_q4(px, sx, code, R, K, N, codes.data_ptr(), scales.data_ptr(),
                                        K // scales.shape[2], gated, po, E, ys.data_ptr(),
                                        _stream(xs))
    if st:
        _check(st, "hc_mix_expert_product_q4")
    return ys


def hc_mix_expert_device_status(stream=None) -> int:
    """Waits for the stream; nonzero, once, if a kernel of this module gave up a wait on the
    current device since the last call."""
    return int(lib().hc_mix_expert_device_status(binding._stream(stream)))
