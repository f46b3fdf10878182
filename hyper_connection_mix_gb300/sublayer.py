"""Python entry points of include/hcmix_sublayer.h, with the C ABI's names.

The operators around a hyper-connection sublayer: the streams collapsed with
`pre` (and normalised) in front of it, the tokens sorted by expert and back
inside it, the streams expanded with `post` and `comb` behind it, and the
gradients.  As in `binding`: argument marshalling only, outputs are allocated
here (or given with `out`), a call goes to the current stream of its tensors'
device unless `stream` says otherwise, and a non-OK status raises HcMixError.
There is no CPU fallback.

With `stream` (a torch stream or a raw handle) outputs are allocated there, as
in a `with torch.cuda.stream(...)` block.  The caller orders the streams' work, as
for any kernel; tensors may be let go at once on either side, since the inputs are
recorded on `stream` and the outputs on the stream that was current.  That
takes about 25 us of host time a call (a stream that is current, about 6).

Matrices are 2-D CUDA tensors of one type (bf16, fp16 or fp32) with unit inner
stride; coefficients, statistics and expert weights are contiguous fp32.

Results carry no autograd graph, whether or not the inputs require gradients:
each gradient is a call of its own, `hc_mix_..._backward`.  That of the mix
statistics themselves (of hc_mix_fused) is not in the library, so dpre, dpost and
dcomb are as far as a gradient goes towards x through them.
"""
from __future__ import annotations

import ctypes
import threading

import torch

from . import binding
from .binding import HC, _check

MOST_EXPERTS = 4096
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


# A small call's time is this module's, so the checks read each attribute once and
# every output is an allocation of its own (views of a shared one cost more).

_empty = torch.empty
_F32, _I32 = torch.float32, torch.int32
_device = torch._C._cuda_getDevice  # the current device's index


def _there(stream, device, call, *args):
    """call(*args) with the tensors' device current (the library launches on the current one) and,
    if given, on `stream`: what the call allocates and frees is memory of the stream that uses it.
    """
    if device.index != _device():
        with torch.cuda.device(device):
            return _there(stream, device, call, *args)
    if stream is None:
        return call(*args)
    if isinstance(stream, torch.cuda.Stream) and stream.device != device:
        raise ValueError("stream must be of the device of the matrices")
    handle = binding._stream(stream)
    if handle == torch._C._cuda_getCurrentRawStream(device.index):
        return call(*args)
    if not isinstance(stream, torch.cuda.Stream):
        stream = (torch.cuda.ExternalStream(handle, device=device) if handle
                  else torch.cuda.default_stream(device))
    before = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        result = call(*args)
    # either stream may still use a tensor when its last reference goes
    for t in args:
        if isinstance(t, torch.Tensor):
            t.record_stream(stream)
    for t in result if isinstance(result, tuple) else (result,):
        t.record_stream(before)
    return result


def _stream(t: torch.Tensor) -> int:
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _matrix(t: torch.Tensor, name: str):
    """(pointer, row stride, type code, rows, width, dtype, device) of a call's first matrix."""
    dtype = t.dtype
    code = TYPES.get(dtype)
    shape = t.shape
    if code is None or len(shape) != 2 or not t.is_cuda:
        raise ValueError(f"{name} must be a 2-D CUDA tensor of bf16, fp16 or fp32")
    rows, width = shape
    stride, inner = t.stride()
    if inner != 1 and width > 1:
        raise ValueError(f"{name} must have unit inner stride")
    if rows <= 1 and stride < width:
        stride = width
    return t.data_ptr(), stride, code, rows, width, dtype, t.device


def _like(t: torch.Tensor, name: str, shape, dtype, device):
    """(pointer, row stride) of a further matrix."""
    if t.dtype is not dtype or t.device != device:
        raise ValueError(f"{name} must have the type and device of the other matrices")
    if t.shape != shape:
        raise ValueError(f"{name} must be of shape {shape}, not {tuple(t.shape)}")
    rows, width = shape
    stride, inner = t.stride()
    if inner != 1 and width > 1:
        raise ValueError(f"{name} must have unit inner stride")
    return t.data_ptr(), width if rows <= 1 and stride < width else stride


def _floats(t: torch.Tensor, name: str, shape, device) -> int:
    if t.dtype is not _F32 or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous fp32 of shape {shape} on the device of the "
                         "matrices")
    return t.data_ptr()


def _ints(t: torch.Tensor, name: str, dim: int, device) -> int:
    if t.dtype is not _I32 or t.dim() != dim or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous int32 with {dim} dimension(s) on the device "
                         "of the matrices")
    return t.data_ptr()


def _params(weight, bias, dtype, width: int, device):
    """(weight, bias, type code) of a norm's parameters, either of which may be None."""
    kind, at = None, [None, None]
    for i, t in enumerate((weight, bias)):
        if t is not None:
            d = t.dtype
            if ((d is not _F32 and d is not dtype) or (kind is not None and d is not kind)
                    or t.shape != (width,) or t.device != device or not t.is_contiguous()):
                raise ValueError(f"{'bias' if i else 'weight'} must be contiguous of shape "
                                 f"({width},), fp32 or of the matrices' type, on their device, "
                                 "weight and bias alike")
            kind = d
            at[i] = t.data_ptr()
    return at[0], at[1], TYPES[kind or _F32]


def _output(out, shape, dtype, device) -> torch.Tensor:
    """A contiguous matrix: `out`, or a new one."""
    if out is None:
        return _empty(shape, dtype=dtype, device=device)
    if out.shape != shape or out.dtype is not dtype or out.device != device or not out.is_contiguous():
        raise ValueError(f"out must be contiguous of shape {shape} and the inputs' type, on their "
                         "device")
    return out


def _f32(shape, device) -> torch.Tensor:
    return _empty(shape, dtype=_F32, device=device)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _width(K: int) -> int:
    """The width of one stream of x[M, K]."""
    if K % HC or K == 0:
        raise ValueError(f"x must be of shape (M, {HC} * D)")
    return K // HC


# ---------------------------------------------------------------- layer norm


def hc_mix_layer_norm(x: torch.Tensor, weight=None, bias=None, eps: float = 1e-5,
                      want_stats: bool = False, out=None, stream=None):
    """y[M, N], each row of x normalised, scaled by weight[N] and shifted by
    bias[N] (fp32 or x's type; None: ones, zeros); with want_stats (y, mean[M],
    rstd[M]), which hc_mix_layer_norm_backward takes."""
    px, sx, code, M, N, dtype, device = _matrix(x, "x")
    if stream is not None or device.index != _device():
        return _there(stream, device, hc_mix_layer_norm, x, weight, bias, eps, want_stats, out)
    pw, pb, ptype = _params(weight, bias, dtype, N, device)
    y = _output(out, (M, N), dtype, device)
    mean, rstd = (_f32((M,), device), _f32((M,), device)) if want_stats else (None, None)
    st = lib().hc_mix_layer_norm(px, sx, code, M, N, pw, pb, ptype, eps, y.data_ptr(), _ptr(mean),
                                 _ptr(rstd), _stream(x))
    if st:
        _check(st, "hc_mix_layer_norm")
    return (y, mean, rstd) if want_stats else y


def layer_norm_workspace_bytes(M: int, N: int, dtype: torch.dtype) -> int:
    return int(lib().hc_mix_layer_norm_workspace_bytes(TYPES[dtype], M, N))


def hc_mix_layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor,
                               rstd: torch.Tensor, weight=None, want_params: bool = True,
                               out=None, workspace=None, stream=None):
    """(dx[M, N], dweight[N], dbias[N]) of hc_mix_layer_norm, the latter two in
    fp32 (with want_params=False only dx).  `workspace`: a uint8 tensor of
    layer_norm_workspace_bytes() bytes, allocated here if not given."""
    px, sx, code, M, N, dtype, device = _matrix(x, "x")
    if stream is not None or device.index != _device():
        return _there(stream, device, hc_mix_layer_norm_backward, dy, x, mean, rstd, weight,
                      want_params, out, workspace)
    pd, sd = _like(dy, "dy", (M, N), dtype, device)
    pm, pr = _floats(mean, "mean", (M,), device), _floats(rstd, "rstd", (M,), device)
    pw, _, ptype = _params(weight, None, dtype, N, device)
    dx = _output(out, (M, N), dtype, device)
    L = lib()
    dweight = dbias = None
    nbytes = 0
    if want_params:
        dweight, dbias = _f32((N,), device), _f32((N,), device)
        if workspace is None:
            nbytes = L.hc_mix_layer_norm_workspace_bytes(code, M, N)
            workspace = _empty(nbytes, dtype=torch.uint8, device=device)
        else:
            if (workspace.dtype is not torch.uint8 or workspace.device != device
                    or not workspace.is_contiguous()):
                raise ValueError("workspace must be contiguous uint8 on the device of the matrices")
            nbytes = workspace.numel()
    st = L.hc_mix_layer_norm_backward(pd, sd, px, sx, code, M, N, pm, pr, pw, ptype, dx.data_ptr(),
                                      _ptr(dweight), _ptr(dbias),
                                      _ptr(workspace) if want_params else None, nbytes,
                                      _stream(x))
    if st:
        _check(st, "hc_mix_layer_norm_backward")
    return (dx, dweight, dbias) if want_params else dx


# ---------------------------------------------------------------- streams


def hc_mix_collapse(x: torch.Tensor, pre: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    """h[M, D] = sum_i pre[:, i] x_i of the streams x[M, 4 * D]."""
    px, sx, code, M, K, dtype, device = _matrix(x, "x")
    if stream is not None or device.index != _device():
        return _there(stream, device, hc_mix_collapse, x, pre, out)
    D = _width(K)
    pp = _floats(pre, "pre", (M, HC), device)
    h = _output(out, (M, D), dtype, device)
    st = lib().hc_mix_collapse(px, sx, code, M, D, HC, pp, h.data_ptr(), _stream(x))
    if st:
        _check(st, "hc_mix_collapse")
    return h


def hc_mix_collapse_norm(x: torch.Tensor, pre: torch.Tensor, weight=None, bias=None,
                         eps: float = 1e-5, want_saved: bool = False, out=None, stream=None):
    """y[M, D], the layer norm of hc_mix_collapse's h in one pass over x; with
    want_saved (y, h, mean, rstd), for hc_mix_layer_norm_backward on h."""
    px, sx, code, M, K, dtype, device = _matrix(x, "x")
    if stream is not None or device.index != _device():
        return _there(stream, device, hc_mix_collapse_norm, x, pre, weight, bias, eps,
                      want_saved, out)
    D = _width(K)
    pp = _floats(pre, "pre", (M, HC), device)
    pw, pb, ptype = _params(weight, bias, dtype, D, device)
    y = _output(out, (M, D), dtype, device)
    h = mean = rstd = None
    if want_saved:
        h = _empty((M, D), dtype=dtype, device=device)
        mean, rstd = _f32((M,), device), _f32((M,), device)
    st = lib().hc_mix_collapse_norm(px, sx, code, M, D, HC, pp, pw, pb, ptype, eps, y.data_ptr(),
                                    _ptr(h), _ptr(mean), _ptr(rstd), _stream(x))
    if st:
        _check(st, "hc_mix_collapse_norm")
    return (y, h, mean, rstd) if want_saved else y


def hc_mix_collapse_backward(dh: torch.Tensor, x: torch.Tensor, pre: torch.Tensor, dx_add=None,
                             out=None, stream=None):
    """(dx[M, 4 * D], dpre[M, 4]) of hc_mix_collapse, dx with dx_add[M, 4 * D]
    added (the gradient of x through hc_mix_expand); out may be dx_add."""
    px, sx, code, M, K, dtype, device = _matrix(x, "x")
    if stream is not None or device.index != _device():
        return _there(stream, device, hc_mix_collapse_backward, dh, x, pre, dx_add, out)
    D = _width(K)
    pd, sd = _like(dh, "dh", (M, D), dtype, device)
    pa, sa = (None, 0) if dx_add is None else _like(dx_add, "dx_add", (M, K), dtype, device)
    pp = _floats(pre, "pre", (M, HC), device)
    dx = _output(out, (M, K), dtype, device)
    dpre = _f32((M, HC), device)
    st = lib().hc_mix_collapse_backward(pd, sd, px, sx, pa, sa, code, M, D, HC, pp, dx.data_ptr(),
                                        dpre.data_ptr(), _stream(x))
    if st:
        _check(st, "hc_mix_collapse_backward")
    return dx, dpre


def hc_mix_expand(x: torch.Tensor, y: torch.Tensor, post: torch.Tensor, comb: torch.Tensor,
                  out=None, stream=None) -> torch.Tensor:
    """The next streams [M, 4 * D]: stream i is post[:, i] y + sum_j
    comb[:, i, j] x_j.  out may be x.  A model whose weights mean the sum over
    comb's first index passes comb.transpose(1, 2).contiguous()."""
    px, sx, code, M, K, dtype, device = _matrix(x, "x")
    if stream is not None or device.index != _device():
        return _there(stream, device, hc_mix_expand, x, y, post, comb, out)
    D = _width(K)
    py, sy = _like(y, "y", (M, D), dtype, device)
    pp, pc = _floats(post, "post", (M, HC), device), _floats(comb, "comb", (M, HC, HC), device)
    out = _output(out, (M, K), dtype, device)
    st = lib().hc_mix_expand(px, sx, py, sy, code, M, D, HC, pp, pc, out.data_ptr(),
                             _stream(x))
    if st:
        _check(st, "hc_mix_expand")
    return out


def hc_mix_expand_backward(dout: torch.Tensor, x: torch.Tensor, y: torch.Tensor,
                           post: torch.Tensor, comb: torch.Tensor, out=None, stream=None):
    """(dx[M, 4 * D], dy[M, D], dpost[M, 4], dcomb[M, 4, 4]) of hc_mix_expand;
    out (for dx) may be dout."""
    px, sx, code, M, K, dtype, device = _matrix(x, "x")
    if stream is not None or device.index != _device():
        return _there(stream, device, hc_mix_expand_backward, dout, x, y, post, comb, out)
    D = _width(K)
    pd, sd = _like(dout, "dout", (M, K), dtype, device)
    py, sy = _like(y, "y", (M, D), dtype, device)
    pp, pc = _floats(post, "post", (M, HC), device), _floats(comb, "comb", (M, HC, HC), device)
    dx = _output(out, (M, K), dtype, device)
    dy = _empty((M, D), dtype=dtype, device=device)
    dpost, dcomb = _f32((M, HC), device), _f32((M, HC, HC), device)
    st = lib().hc_mix_expand_backward(pd, sd, px, sx, py, sy, code, M, D, HC, pp, pc, dx.data_ptr(),
                                      dy.data_ptr(), dpost.data_ptr(), dcomb.data_ptr(),
                                      _stream(x))
    if st:
        _check(st, "hc_mix_expand_backward")
    return dx, dy, dpost, dcomb


# ---------------------------------------------------------------- experts


def hc_mix_expert_sort(ids: torch.Tensor, n_experts: int, stream=None):
    """(offsets[E + 1], slots[T, k], source[T * k]), int32, of ids[T, k] (int32
    or int64): expert e's rows are offsets[e] .. offsets[e + 1] - 1, slots gives
    each pair's row and source each row's pair, in the order of ids within an
    expert.  An id outside 0 .. E - 1 has slot -1; rows without a pair source -1."""
    dtype, shape = ids.dtype, ids.shape
    wide = dtype is torch.int64
    if not (wide or dtype is _I32) or len(shape) != 2 or not ids.is_cuda or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous 2-D CUDA tensor of int32 or int64")
    T, k = shape
    device = ids.device
    if stream is not None or device.index != _device():
        return _there(stream, device, hc_mix_expert_sort, ids, n_experts)
    # the library refuses a number of experts outside 1 .. MOST_EXPERTS
    offsets = _empty(min(max(n_experts, 0), MOST_EXPERTS) + 1, dtype=_I32, device=device)
    slots = _empty(shape, dtype=_I32, device=device)
    source = _empty(T * k, dtype=_I32, device=device)
    st = lib().hc_mix_expert_sort(ids.data_ptr(), 8 if wide else 4, T, k, n_experts,
                                  offsets.data_ptr(), slots.data_ptr(), source.data_ptr(),
                                  _stream(ids))
    if st:
        _check(st, "hc_mix_expert_sort")
    return offsets, slots, source


def _slots(slots, T: int, device):
    p = _ints(slots, "slots", 2, device)
    rows, k = slots.shape
    if rows != T:
        raise ValueError(f"slots must have {T} rows")
    return p, k


def _offsets(offsets, device):
    return (None, 0) if offsets is None else (_ints(offsets, "offsets", 1, device),
                                              offsets.shape[0] - 1)


def hc_mix_expert_dispatch(x: torch.Tensor, slots: torch.Tensor, offsets=None, out=None,
                           stream=None) -> torch.Tensor:
    """xs[T * k, D] with xs[slots[t, j]] = x[t] and zeros from row offsets[E] on
    (without offsets those rows are left as they are)."""
    px, sx, code, T, D, dtype, device = _matrix(x, "x")
    if stream is not None or device.index != _device():
        return _there(stream, device, hc_mix_expert_dispatch, x, slots, offsets, out)
    ps, k = _slots(slots, T, device)
    po, E = _offsets(offsets, device)
    xs = _output(out, (T * k, D), dtype, device)
    st = lib().hc_mix_expert_dispatch(px, sx, code, T, k, D, ps, po, E, xs.data_ptr(),
                                      _stream(x))
    if st:
        _check(st, "hc_mix_expert_dispatch")
    return xs


def hc_mix_expert_combine(ys: torch.Tensor, slots: torch.Tensor, weights=None, out=None,
                          stream=None) -> torch.Tensor:
    """y[T, D] with y[t] = sum_j weights[t, j] ys[slots[t, j]]; without weights,
    of ones: the gradient of hc_mix_expert_dispatch."""
    py, sy, code, rows, D, dtype, device = _matrix(ys, "ys")
    if stream is not None or device.index != _device():
        return _there(stream, device, hc_mix_expert_combine, ys, slots, weights, out)
    T = slots.shape[0]
    ps, k = _slots(slots, T, device)
    pw = None if weights is None else _floats(weights, "weights", (T, k), device)
    y = _output(out, (T, D), dtype, device)
    st = lib().hc_mix_expert_combine(py, sy, code, rows, T, k, D, ps, pw, y.data_ptr(),
                                     _stream(ys))
    if st:
        _check(st, "hc_mix_expert_combine")
    return y


def hc_mix_expert_combine_backward(dy: torch.Tensor, ys: torch.Tensor, slots: torch.Tensor,
                                   offsets, weights: torch.Tensor, out=None, stream=None):
    """(dys, dweights[T, k]) of hc_mix_expert_combine: dys[slots[t, j]] =
    weights[t, j] dy[t], zeros from row offsets[E] on (offsets None: left as
    they are), dweights[t, j] = dy[t] . ys[slots[t, j]]."""
    py, sy, code, rows, D, dtype, device = _matrix(ys, "ys")
    if stream is not None or device.index != _device():
        return _there(stream, device, hc_mix_expert_combine_backward, dy, ys, slots, offsets,
                      weights, out)
    T = dy.shape[0]
    pd, sd = _like(dy, "dy", (T, D), dtype, device)
    ps, k = _slots(slots, T, device)
    po, E = _offsets(offsets, device)
    pw = _floats(weights, "weights", (T, k), device)
    dys = _output(out, (rows, D), dtype, device)
    dweights = _f32((T, k), device)
    st = lib().hc_mix_expert_combine_backward(pd, sd, py, sy, code, rows, T, k, D, ps, po, E, pw,
                                              dys.data_ptr(), dweights.data_ptr(),
                                              _stream(ys))
    if st:
        _check(st, "hc_mix_expert_combine_backward")
    return dys, dweights
