"""Python entry points of include/hcmix_sublayer.h, with the C ABI's names.

The operators around a hyper-connection sublayer: the streams collapsed with
`pre` (and normalised) in front of it, the tokens sorted by expert and back
inside it, the streams expanded with `post` and `comb` behind it, and the
gradients.  As in `binding`: argument marshalling only, outputs are allocated
here (or given with `out`), a call goes to the current stream of its tensors'
device unless `stream` says otherwise, and a non-OK status raises HcMixError.
There is no CPU fallback.

Matrices are 2-D CUDA tensors of one type (bf16, fp16 or fp32) with unit inner
stride; coefficients, statistics and expert weights are contiguous fp32.
"""
from __future__ import annotations

import ctypes
import threading

import torch

from . import binding
from .binding import HC, _check

TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}

# every symbol include/hcmix_sublayer.h declares
EXPORTS = ("hc_mix_layer_norm", "hc_mix_layer_norm_workspace_bytes", "hc_mix_layer_norm_backward",
           "hc_mix_collapse", "hc_mix_collapse_norm", "hc_mix_collapse_backward", "hc_mix_expand",
           "hc_mix_expand_backward", "hc_mix_expert_sort", "hc_mix_expert_dispatch",
           "hc_mix_expert_combine", "hc_mix_expert_combine_backward")

_lib = None
_lock = threading.Lock()


def lib() -> ctypes.CDLL:
    """libhcmix.so with the argument types of this module's entry points set."""
    global _lib
    if _lib is None:
        with _lock:
            L = binding.lib()
            P, N, I, F, S = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float,
                             ctypes.c_size_t)
            args = {
                "hc_mix_layer_norm": [P, N, I, N, N, P, P, I, F, P, P, P, P],
                "hc_mix_layer_norm_workspace_bytes": [I, N, N],
                "hc_mix_layer_norm_backward": [P, N, P, N, I, N, N, P, P, P, I, P, P, P, P, S, P],
                "hc_mix_collapse": [P, N, I, N, N, I, P, P, P],
                "hc_mix_collapse_norm": [P, N, I, N, N, I, P, P, P, I, F, P, P, P, P, P],
                "hc_mix_collapse_backward": [P, N, P, N, P, N, I, N, N, I, P, P, P, P],
                "hc_mix_expand": [P, N, P, N, I, N, N, I, P, P, P, P],
                "hc_mix_expand_backward": [P, N, P, N, P, N, I, N, N, I, P, P, P, P, P, P, P],
                "hc_mix_expert_sort": [P, I, N, N, N, P, P, P, P],
                "hc_mix_expert_dispatch": [P, N, I, N, N, N, P, P, N, P, P],
                "hc_mix_expert_combine": [P, N, I, N, N, N, N, P, P, P, P],
                "hc_mix_expert_combine_backward": [P, N, P, N, I, N, N, N, N, P, P, N, P, P, P, P],
            }
            for name in EXPORTS:
                f = getattr(L, name)
                f.argtypes = args[name]
                f.restype = S if name.endswith("_bytes") else I
            _lib = L
    return _lib


def _stream(stream, device: int):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return binding._stream(stream)


def _matrix(t: torch.Tensor, name: str, like: torch.Tensor | None = None, shape=None):
    """(pointer, row stride) of a matrix; its type, device and shape checked."""
    if not (t.is_cuda and t.dim() == 2 and t.dtype in TYPES):
        raise ValueError(f"{name} must be a 2-D CUDA tensor of bf16, fp16 or fp32")
    rows, width = t.shape
    stride, inner = t.stride()
    if inner != 1 and width > 1:
        raise ValueError(f"{name} must have unit inner stride")
    if like is not None and (t.dtype != like.dtype or t.device != like.device):
        raise ValueError(f"{name} must have the type and device of the other matrices")
    if shape is not None and (rows, width) != shape:
        raise ValueError(f"{name} must be of shape {shape}, not {(rows, width)}")
    return t.data_ptr(), stride if rows > 1 else max(stride, width)


def _floats(t: torch.Tensor, name: str, like: torch.Tensor, shape) -> int:
    if not (t.dtype == torch.float32 and t.device == like.device and t.shape == shape
            and t.is_contiguous()):
        raise ValueError(f"{name} must be contiguous fp32 of shape {tuple(shape)} on the device "
                         "of the matrices")
    return t.data_ptr()


def _ints(t: torch.Tensor, name: str, like: torch.Tensor, dim: int) -> int:
    if not (t.dtype == torch.int32 and t.device == like.device and t.dim() == dim
            and t.is_contiguous()):
        raise ValueError(f"{name} must be contiguous int32 with {dim} dimension(s) on the device "
                         "of the matrices")
    return t.data_ptr()


def _params(weight, bias, like: torch.Tensor, width: int):
    """(weight, bias, type code) of a norm's parameters, either of which may be None."""
    dtype, at = None, []
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is None:
            at.append(None)
            continue
        if not (t.dtype in (torch.float32, like.dtype) and t.device == like.device
                and t.shape == (width,) and t.is_contiguous() and dtype in (None, t.dtype)):
            raise ValueError(f"{name} must be contiguous of shape ({width},), fp32 or of the "
                             "matrices' type, on their device, weight and bias alike")
        dtype = t.dtype
        at.append(t.data_ptr())
    return at[0], at[1], TYPES[dtype or torch.float32]


def _output(out, like: torch.Tensor, *shape) -> torch.Tensor:
    """A contiguous matrix of `like`'s type and device: `out`, or a new one."""
    if out is None:
        return like.new_empty(shape)
    if not (out.shape == shape and out.dtype == like.dtype and out.device == like.device
            and out.is_contiguous()):
        raise ValueError(f"out must be contiguous of shape {shape} and the inputs' type, on their "
                         "device")
    return out


def _f32(like: torch.Tensor, *shape) -> torch.Tensor:
    return torch.empty(shape, dtype=torch.float32, device=like.device)


def _width(x: torch.Tensor) -> int:
    """The width of one stream of x[M, HC * D]."""
    if x.dim() != 2 or x.shape[1] % HC or x.shape[1] == 0:
        raise ValueError(f"x must be of shape (M, {HC} * D)")
    return x.shape[1] // HC


# ---------------------------------------------------------------- layer norm


def hc_mix_layer_norm(x: torch.Tensor, weight=None, bias=None, eps: float = 1e-5,
                      want_stats: bool = False, out=None, stream=None):
    """y[M, N], each row of x normalised, scaled by weight[N] and shifted by
    bias[N] (fp32 or x's type; None: ones, zeros); with want_stats (y, mean[M],
    rstd[M]), which hc_mix_layer_norm_backward takes."""
    px, sx = _matrix(x, "x")
    M, N = x.shape
    pw, pb, ptype = _params(weight, bias, x, N)
    y = _output(out, x, M, N)
    stats = _f32(x, 2, M).unbind() if want_stats else None
    st = lib().hc_mix_layer_norm(px, sx, TYPES[x.dtype], M, N, pw, pb, ptype, eps, y.data_ptr(),
                                 stats[0].data_ptr() if want_stats else None,
                                 stats[1].data_ptr() if want_stats else None,
                                 _stream(stream, x.get_device()))
    _check(st, "hc_mix_layer_norm")
    return (y, *stats) if want_stats else y


def layer_norm_workspace_bytes(M: int, N: int, dtype: torch.dtype) -> int:
    return int(lib().hc_mix_layer_norm_workspace_bytes(TYPES[dtype], M, N))


def hc_mix_layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor,
                               rstd: torch.Tensor, weight=None, want_params: bool = True,
                               out=None, workspace=None, stream=None):
    """(dx[M, N], dweight[N], dbias[N]) of hc_mix_layer_norm, the latter two in
    fp32 (with want_params=False only dx).  `workspace`: a uint8 tensor of
    layer_norm_workspace_bytes() bytes, allocated here if not given."""
    px, sx = _matrix(x, "x")
    M, N = x.shape
    pd, sd = _matrix(dy, "dy", x, (M, N))
    pm, pr = _floats(mean, "mean", x, (M,)), _floats(rstd, "rstd", x, (M,))
    pw, _, ptype = _params(weight, None, x, N)
    dx = _output(out, x, M, N)
    grads, nbytes = (None, None), 0
    if want_params:
        grads = _f32(x, 2, N).unbind()
        nbytes = layer_norm_workspace_bytes(M, N, x.dtype)
        if workspace is None:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
        nbytes = workspace.numel()
    st = lib().hc_mix_layer_norm_backward(
        pd, sd, px, sx, TYPES[x.dtype], M, N, pm, pr, pw, ptype, dx.data_ptr(),
        grads[0].data_ptr() if want_params else None, grads[1].data_ptr() if want_params else None,
        workspace.data_ptr() if want_params else None, nbytes, _stream(stream, x.get_device()))
    _check(st, "hc_mix_layer_norm_backward")
    return (dx, *grads) if want_params else dx


# ---------------------------------------------------------------- streams


def hc_mix_collapse(x: torch.Tensor, pre: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    """h[M, D] = sum_i pre[:, i] x_i of the streams x[M, 4 * D]."""
    px, sx = _matrix(x, "x")
    M, D = x.shape[0], _width(x)
    pp = _floats(pre, "pre", x, (M, HC))
    h = _output(out, x, M, D)
    st = lib().hc_mix_collapse(px, sx, TYPES[x.dtype], M, D, HC, pp, h.data_ptr(),
                               _stream(stream, x.get_device()))
    _check(st, "hc_mix_collapse")
    return h


def hc_mix_collapse_norm(x: torch.Tensor, pre: torch.Tensor, weight=None, bias=None,
                         eps: float = 1e-5, want_saved: bool = False, out=None, stream=None):
    """y[M, D], the layer norm of hc_mix_collapse's h in one pass over x; with
    want_saved (y, h, mean, rstd), for hc_mix_layer_norm_backward on h."""
    px, sx = _matrix(x, "x")
    M, D = x.shape[0], _width(x)
    pp = _floats(pre, "pre", x, (M, HC))
    pw, pb, ptype = _params(weight, bias, x, D)
    y = _output(out, x, M, D)
    saved = (x.new_empty((M, D)), *_f32(x, 2, M).unbind()) if want_saved else (None,) * 3
    st = lib().hc_mix_collapse_norm(px, sx, TYPES[x.dtype], M, D, HC, pp, pw, pb, ptype, eps,
                                    y.data_ptr(), *(s if s is None else s.data_ptr() for s in saved),
                                    _stream(stream, x.get_device()))
    _check(st, "hc_mix_collapse_norm")
    return (y, *saved) if want_saved else y


def hc_mix_collapse_backward(dh: torch.Tensor, x: torch.Tensor, pre: torch.Tensor, dx_add=None,
                             out=None, stream=None):
    """(dx[M, 4 * D], dpre[M, 4]) of hc_mix_collapse, dx with dx_add[M, 4 * D]
    added (the gradient of x through hc_mix_expand); out may be dx_add."""
    px, sx = _matrix(x, "x")
    M, D = x.shape[0], _width(x)
    pd, sd = _matrix(dh, "dh", x, (M, D))
    pa, sa = (None, 0) if dx_add is None else _matrix(dx_add, "dx_add", x, (M, HC * D))
    pp = _floats(pre, "pre", x, (M, HC))
    dx = _output(out, x, M, HC * D)
    dpre = _f32(x, M, HC)
    st = lib().hc_mix_collapse_backward(pd, sd, px, sx, pa, sa, TYPES[x.dtype], M, D, HC, pp,
                                        dx.data_ptr(), dpre.data_ptr(),
                                        _stream(stream, x.get_device()))
    _check(st, "hc_mix_collapse_backward")
    return dx, dpre


def hc_mix_expand(x: torch.Tensor, y: torch.Tensor, post: torch.Tensor, comb: torch.Tensor,
                  out=None, stream=None) -> torch.Tensor:
    """The next streams [M, 4 * D]: stream i is post[:, i] y + sum_j
    comb[:, i, j] x_j.  out may be x."""
    px, sx = _matrix(x, "x")
    M, D = x.shape[0], _width(x)
    py, sy = _matrix(y, "y", x, (M, D))
    pp, pc = _floats(post, "post", x, (M, HC)), _floats(comb, "comb", x, (M, HC, HC))
    out = _output(out, x, M, HC * D)
    st = lib().hc_mix_expand(px, sx, py, sy, TYPES[x.dtype], M, D, HC, pp, pc, out.data_ptr(),
                             _stream(stream, x.get_device()))
    _check(st, "hc_mix_expand")
    return out


def hc_mix_expand_backward(dout: torch.Tensor, x: torch.Tensor, y: torch.Tensor,
                           post: torch.Tensor, comb: torch.Tensor, out=None, stream=None):
    """(dx[M, 4 * D], dy[M, D], dpost[M, 4], dcomb[M, 4, 4]) of hc_mix_expand;
    out (for dx) may be dout."""
    px, sx = _matrix(x, "x")
    M, D = x.shape[0], _width(x)
    pd, sd = _matrix(dout, "dout", x, (M, HC * D))
    py, sy = _matrix(y, "y", x, (M, D))
    pp, pc = _floats(post, "post", x, (M, HC)), _floats(comb, "comb", x, (M, HC, HC))
    dx, dy = _output(out, x, M, HC * D), x.new_empty((M, D))
    dpost, dcomb = _f32(x, M, HC), _f32(x, M, HC, HC)
    st = lib().hc_mix_expand_backward(pd, sd, px, sx, py, sy, TYPES[x.dtype], M, D, HC, pp, pc,
                                      dx.data_ptr(), dy.data_ptr(), dpost.data_ptr(),
                                      dcomb.data_ptr(), _stream(stream, x.get_device()))
    _check(st, "hc_mix_expand_backward")
    return dx, dy, dpost, dcomb


# ---------------------------------------------------------------- experts


def hc_mix_expert_sort(ids: torch.Tensor, n_experts: int, stream=None):
    """(offsets[E + 1], slots[T, k], source[T * k]), int32, of ids[T, k] (int32
    or int64): expert e's rows are offsets[e] .. offsets[e + 1] - 1, slots gives
    each pair's row and source each row's pair, in the order of ids within an
    expert.  An id outside 0 .. E - 1 has slot -1; rows without a pair source -1."""
    if not (ids.is_cuda and ids.dim() == 2 and ids.dtype in (torch.int32, torch.int64)
            and ids.is_contiguous()):
        raise ValueError("ids must be a contiguous 2-D CUDA tensor of int32 or int64")
    T, k = ids.shape
    offsets = torch.empty(max(n_experts, 0) + 1, dtype=torch.int32, device=ids.device)
    slots = torch.empty((T, k), dtype=torch.int32, device=ids.device)
    source = torch.empty(T * k, dtype=torch.int32, device=ids.device)
    st = lib().hc_mix_expert_sort(ids.data_ptr(), ids.element_size(), T, k, n_experts,
                                  offsets.data_ptr(), slots.data_ptr(), source.data_ptr(),
                                  _stream(stream, ids.get_device()))
    _check(st, "hc_mix_expert_sort")
    return offsets, slots, source


def _slots(slots, like, T):
    p = _ints(slots, "slots", like, 2)
    if slots.shape[0] != T:
        raise ValueError(f"slots must have {T} rows")
    return p, slots.shape[1]


def _offsets(offsets, like):
    return (None, 0) if offsets is None else (_ints(offsets, "offsets", like, 1),
                                              offsets.shape[0] - 1)


def hc_mix_expert_dispatch(x: torch.Tensor, slots: torch.Tensor, offsets=None, out=None,
                           stream=None) -> torch.Tensor:
    """xs[T * k, D] with xs[slots[t, j]] = x[t] and zeros from row offsets[E] on
    (without offsets those rows are left as they are)."""
    px, sx = _matrix(x, "x")
    T, D = x.shape
    ps, k = _slots(slots, x, T)
    po, E = _offsets(offsets, x)
    xs = _output(out, x, T * k, D)
    st = lib().hc_mix_expert_dispatch(px, sx, TYPES[x.dtype], T, k, D, ps, po, E, xs.data_ptr(),
                                      _stream(stream, x.get_device()))
    _check(st, "hc_mix_expert_dispatch")
    return xs


def hc_mix_expert_combine(ys: torch.Tensor, slots: torch.Tensor, weights=None, out=None,
                          stream=None) -> torch.Tensor:
    """y[T, D] with y[t] = sum_j weights[t, j] ys[slots[t, j]]; without weights,
    of ones: the gradient of hc_mix_expert_dispatch."""
    py, sy = _matrix(ys, "ys")
    rows, D = ys.shape
    ps, k = _slots(slots, ys, slots.shape[0])
    T = slots.shape[0]
    pw = None if weights is None else _floats(weights, "weights", ys, (T, k))
    y = _output(out, ys, T, D)
    st = lib().hc_mix_expert_combine(py, sy, TYPES[ys.dtype], rows, T, k, D, ps, pw, y.data_ptr(),
                                     _stream(stream, ys.get_device()))
    _check(st, "hc_mix_expert_combine")
    return y


def hc_mix_expert_combine_backward(dy: torch.Tensor, ys: torch.Tensor, slots: torch.Tensor,
                                   offsets, weights: torch.Tensor, out=None, stream=None):
    """(dys, dweights[T, k]) of hc_mix_expert_combine: dys[slots[t, j]] =
    weights[t, j] dy[t], zeros from row offsets[E] on (offsets None: left as
    they are), dweights[t, j] = dy[t] . ys[slots[t, j]]."""
    py, sy = _matrix(ys, "ys")
    rows, D = ys.shape
    T = dy.shape[0]
    pd, sd = _matrix(dy, "dy", ys, (T, D))
    ps, k = _slots(slots, ys, T)
    po, E = _offsets(offsets, ys)
    pw = _floats(weights, "weights", ys, (T, k))
    dys = _output(out, ys, rows, D)
    dweights = _f32(ys, T, k)
    st = lib().hc_mix_expert_combine_backward(pd, sd, py, sy, TYPES[ys.dtype], rows, T, k, D, ps,
                                              po, E, pw, dys.data_ptr(), dweights.data_ptr(),
                                              _stream(stream, ys.get_device()))
    _check(st, "hc_mix_expert_combine_backward")
    return dys, dweights
