"""Torch-facing wrappers of the C ABI: argument marshalling only.

Every op checks dtype, device and contiguity, allocates its outputs with torch
when none are given, and passes raw pointers plus the current CUDA stream to
libslope.so.  No arithmetic of the layer happens here.

bf16 tensors are torch.bfloat16; the 16-bit position-code words ("meta") are
torch.int16 tensors holding the uint16 patterns.
"""
import ctypes
import warnings

import torch

from . import _lib


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need(t, dtype, name, shape=None):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def _empty(shape, dtype, like):
    return torch.empty(shape, dtype=dtype, device=like.device)


def prune24(W, vals=None, meta=None):
    """Row-wise 2:4 magnitude pruning: W [rows, K] -> (vals [rows, K/2], meta [rows, K/16])."""
    _need(W, torch.bfloat16, "W")
    rows, K = W.shape
    vals = _empty((rows, K // 2), torch.bfloat16, W) if vals is None else _need(vals, torch.bfloat16, "vals", (rows, K // 2))
    meta = _empty((rows, K // 16), torch.int16, W) if meta is None else _need(meta, torch.int16, "meta", (rows, K // 16))
    _lib.call("slope_prune24", _ptr(W), rows, K, _ptr(vals), _ptr(meta), _stream())
    return vals, meta


def prune_nm(W, N, M, vals=None, pos=None):
    """Row-wise N:M magnitude pruning: W [rows, K] -> (vals [rows, K*N/M] bf16,
    pos [rows, K*N/M] uint8 positions within each group)."""
    _need(W, torch.bfloat16, "W")
    rows, K = W.shape
    shape = (rows, K // M * N) if M > 0 and K % M == 0 else (rows, 0)
    vals = _empty(shape, torch.bfloat16, W) if vals is None else _need(vals, torch.bfloat16, "vals", shape)
    pos = _empty(shape, torch.uint8, W) if pos is None else _need(pos, torch.uint8, "pos", shape)
    _lib.call("slope_prune_nm", _ptr(W), rows, K, int(N), int(M), _ptr(vals), _ptr(pos), _stream())
    return vals, pos


def double_prune(vals, meta, out_features, in_features, vals_t=None, meta_t=None):
    """W^R (compressed [out, in]) -> (W^{R,C})^T compressed: (vals_t [in, out/2], meta_t [in, out/16])."""
    _need(vals, torch.bfloat16, "vals", (out_features, in_features // 2))
    _need(meta, torch.int16, "meta", (out_features, in_features // 16))
    if vals_t is None:
        vals_t = _empty((in_features, out_features // 2), torch.bfloat16, vals)
    if meta_t is None:
        meta_t = _empty((in_features, out_features // 16), torch.int16, vals)
    _need(vals_t, torch.bfloat16, "vals_t", (in_features, out_features // 2))
    _need(meta_t, torch.int16, "meta_t", (in_features, out_features // 16))
    _lib.call("slope_double_prune", _ptr(vals), _ptr(meta), out_features, in_features, _ptr(vals_t), _ptr(meta_t),
              _stream())
    return vals_t, meta_t


def prune24_double(W, vals=None, meta=None, vals_t=None, meta_t=None):
    """Both prunings in one launch: W [out, in] bf16 -> (vals, meta, vals_t, meta_t),
    equal to prune24 followed by double_prune."""
    _need(W, torch.bfloat16, "W")
    out, in_ = W.shape
    vals = _empty((out, in_ // 2), torch.bfloat16, W) if vals is None else _need(vals, torch.bfloat16, "vals", (out, in_ // 2))
    meta = _empty((out, in_ // 16), torch.int16, W) if meta is None else _need(meta, torch.int16, "meta", (out, in_ // 16))
    vals_t = (_empty((in_, out // 2), torch.bfloat16, W) if vals_t is None
              else _need(vals_t, torch.bfloat16, "vals_t", (in_, out // 2)))
    meta_t = (_empty((in_, out // 16), torch.int16, W) if meta_t is None
              else _need(meta_t, torch.int16, "meta_t", (in_, out // 16)))
    _lib.call("slope_prune24_double", _ptr(W), out, in_, _ptr(vals), _ptr(meta), _ptr(vals_t), _ptr(meta_t),
              _stream())
    return vals, meta, vals_t, meta_t


def adamw_double_prune(vals, meta, dW_vals, m, v, out_features, in_features, lr, beta1, beta2, eps,
                       weight_decay, step, vals_t=None, meta_t=None):
    """One AdamW step on the kept values (vals, m, v updated in place) fused
    with the second pruning of the updated W^R: returns (vals_t, meta_t)."""
    _need(vals, torch.bfloat16, "vals", (out_features, in_features // 2))
    _need(meta, torch.int16, "meta", (out_features, in_features // 16))
    _need(dW_vals, torch.bfloat16, "dW_vals", (out_features, in_features // 2))
    _need(m, torch.float32, "m", (out_features, in_features // 2))
    _need(v, torch.float32, "v", (out_features, in_features // 2))
    if vals_t is None:
        vals_t = _empty((in_features, out_features // 2), torch.bfloat16, vals)
    if meta_t is None:
        meta_t = _empty((in_features, out_features // 16), torch.int16, vals)
    _need(vals_t, torch.bfloat16, "vals_t", (in_features, out_features // 2))
    _need(meta_t, torch.int16, "meta_t", (in_features, out_features // 16))
    _lib.call("slope_adamw_double_prune", _ptr(vals), _ptr(meta), _ptr(dW_vals), _ptr(m), _ptr(v), out_features,
              in_features, float(lr), float(beta1), float(beta2), float(eps), float(weight_decay), int(step),
              _ptr(vals_t), _ptr(meta_t), _stream())
    return vals_t, meta_t


def adapter_fwd(X, L, XL=None):
    """XL = X . L  (X [T, in], L [in, r])."""
    _need(X, torch.bfloat16, "X")
    T, in_ = X.shape
    _need(L, torch.bfloat16, "L")
    r = L.shape[1]
    XL = _empty((T, r), torch.bfloat16, X) if XL is None else _need(XL, torch.bfloat16, "XL", (T, r))
    _lib.call("slope_adapter_fwd", _ptr(X), _ptr(L), T, in_, r, _ptr(XL), _stream())
    return XL


def fwd(X, vals, meta, XL, R, out_features, Y=None):
    """Y = X . (W^R)^T + XL . R  (XL, R may be None: no adapter)."""
    _need(X, torch.bfloat16, "X")
    T, in_ = X.shape
    _need(vals, torch.bfloat16, "vals", (out_features, in_ // 2))
    _need(meta, torch.int16, "meta", (out_features, in_ // 16))
    r = 0
    if R is not None:
        r = R.shape[0]
        _need(R, torch.bfloat16, "R", (r, out_features))
        _need(XL, torch.bfloat16, "XL", (T, r))
    Y = _empty((T, out_features), torch.bfloat16, X) if Y is None else _need(Y, torch.bfloat16, "Y", (T, out_features))
    _lib.call("slope_fwd", _ptr(X), _ptr(vals), _ptr(meta), _ptr(XL), _ptr(R), T, in_, out_features, r, _ptr(Y),
              _stream())
    return Y


def fwd_fused(X, vals, meta, L, R, out_features, XL=None, Y=None):
    """(XL, Y): XL = X . L and Y = X . (W^R)^T + XL . R in one launch where
    the shapes allow (L, R None: no adapter, XL is None)."""
    _need(X, torch.bfloat16, "X")
    T, in_ = X.shape
    _need(vals, torch.bfloat16, "vals", (out_features, in_ // 2))
    _need(meta, torch.int16, "meta", (out_features, in_ // 16))
    r = 0
    if R is not None:
        r = R.shape[0]
        _need(R, torch.bfloat16, "R", (r, out_features))
        _need(L, torch.bfloat16, "L", (in_, r))
        XL = _empty((T, r), torch.bfloat16, X) if XL is None else _need(XL, torch.bfloat16, "XL", (T, r))
    Y = _empty((T, out_features), torch.bfloat16, X) if Y is None else _need(Y, torch.bfloat16, "Y", (T, out_features))
    _lib.call("slope_fwd_fused", _ptr(X), _ptr(vals), _ptr(meta), _ptr(L), _ptr(R), T, in_, out_features, r,
              _ptr(XL) if r else None, _ptr(Y), _stream())
    return (XL if r else None), Y


def bwd_dx_fused(dY, vals_t, meta_t, R, L, in_features, G=None, dX=None):
    """(G, dX): G = dY . R^T and dX = dY . W^{R,C} + G . L^T in one launch
    where the shapes allow (R, L None: no adapter, G is None)."""
    _need(dY, torch.bfloat16, "dY")
    T, out = dY.shape
    _need(vals_t, torch.bfloat16, "vals_t", (in_features, out // 2))
    _need(meta_t, torch.int16, "meta_t", (in_features, out // 16))
    r = 0
    if L is not None:
        r = L.shape[1]
        _need(L, torch.bfloat16, "L", (in_features, r))
        _need(R, torch.bfloat16, "R", (r, out))
        G = _empty((T, r), torch.bfloat16, dY) if G is None else _need(G, torch.bfloat16, "G", (T, r))
    dX = _empty((T, in_features), torch.bfloat16, dY) if dX is None else _need(dX, torch.bfloat16, "dX", (T, in_features))
    _lib.call("slope_bwd_dx_fused", _ptr(dY), _ptr(vals_t), _ptr(meta_t), _ptr(R), _ptr(L), T, in_features, out, r,
              _ptr(G) if r else None, _ptr(dX), _stream())
    return (G if r else None), dX


def adapter_bwd(X, dY, XL, R, dL=None, dR=None, G=None):
    """(dL [in, r] fp32, dR [r, out] fp32, G [T, r] bf16) for Y += (X L) R."""
    _need(X, torch.bfloat16, "X")
    _need(dY, torch.bfloat16, "dY")
    T, in_ = X.shape
    out = dY.shape[1]
    r = R.shape[0]
    _need(XL, torch.bfloat16, "XL", (T, r))
    _need(R, torch.bfloat16, "R", (r, out))
    dL = _empty((in_, r), torch.float32, X) if dL is None else _need(dL, torch.float32, "dL", (in_, r))
    dR = _empty((r, out), torch.float32, X) if dR is None else _need(dR, torch.float32, "dR", (r, out))
    G = _empty((T, r), torch.bfloat16, X) if G is None else _need(G, torch.bfloat16, "G", (T, r))
    _lib.call("slope_adapter_bwd", _ptr(X), _ptr(dY), _ptr(XL), _ptr(R), T, in_, out, r, _ptr(dL), _ptr(dR),
              _ptr(G), _stream())
    return dL, dR, G


def bwd_dx(dY, vals_t, meta_t, G, L, in_features, dX=None):
    """dX = dY . W^{R,C} + G . L^T."""
    _need(dY, torch.bfloat16, "dY")
    T, out = dY.shape
    _need(vals_t, torch.bfloat16, "vals_t", (in_features, out // 2))
    _need(meta_t, torch.int16, "meta_t", (in_features, out // 16))
    r = 0
    if L is not None:
        r = L.shape[1]
        _need(L, torch.bfloat16, "L", (in_features, r))
        _need(G, torch.bfloat16, "G", (T, r))
    dX = _empty((T, in_features), torch.bfloat16, dY) if dX is None else _need(dX, torch.bfloat16, "dX", (T, in_features))
    _lib.call("slope_bwd_dx", _ptr(dY), _ptr(vals_t), _ptr(meta_t), _ptr(G), _ptr(L), T, in_features, out, r,
              _ptr(dX), _stream())
    return dX


def bwd_dw_masked(dY, X, meta, dW_vals=None):
    """dW restricted to the static mask, compressed like vals: [out, in/2]."""
    _need(dY, torch.bfloat16, "dY")
    _need(X, torch.bfloat16, "X")
    T, out = dY.shape
    in_ = X.shape[1]
    _need(meta, torch.int16, "meta", (out, in_ // 16))
    if dW_vals is None:
        dW_vals = _empty((out, in_ // 2), torch.bfloat16, X)
    _need(dW_vals, torch.bfloat16, "dW_vals", (out, in_ // 2))
    _lib.call("slope_bwd_dw_masked", _ptr(dY), _ptr(X), _ptr(meta), T, in_, out, _ptr(dW_vals), _stream())
    return dW_vals


def bwd_dw_fused(dY, X, meta, XL, G, dW_vals=None, dL=None, dR=None):
    """(dW_vals, dL, dR): the masked weight gradient and the adapter gradients
    dR = XL^T . dY, dL = X^T . G in one launch (XL, G None: no adapter)."""
    _need(dY, torch.bfloat16, "dY")
    _need(X, torch.bfloat16, "X")
    T, out = dY.shape
    in_ = X.shape[1]
    _need(meta, torch.int16, "meta", (out, in_ // 16))
    dW_vals = _empty((out, in_ // 2), torch.bfloat16, X) if dW_vals is None else _need(dW_vals, torch.bfloat16, "dW_vals",
                                                                                         (out, in_ // 2))
    r = 0
    if XL is not None:
        r = XL.shape[1]
        _need(XL, torch.bfloat16, "XL", (T, r))
        _need(G, torch.bfloat16, "G", (T, r))
        dL = _empty((in_, r), torch.float32, X) if dL is None else _need(dL, torch.float32, "dL", (in_, r))
        dR = _empty((r, out), torch.float32, X) if dR is None else _need(dR, torch.float32, "dR", (r, out))
    _lib.call("slope_bwd_dw_fused", _ptr(dY), _ptr(X), _ptr(meta), _ptr(XL), _ptr(G), T, in_, out, r, _ptr(dW_vals),
              _ptr(dL) if r else None, _ptr(dR) if r else None, _stream())
    return dW_vals, (dL if r else None), (dR if r else None)


def bwd_dw_masked_noalloc(dY, X, meta, dW_vals):
    """bwd_dw_masked into a caller-provided dW_vals; the library allocates
    nothing (token-split scratch from a fixed device array; see slope.h)."""
    _need(dY, torch.bfloat16, "dY")
    _need(X, torch.bfloat16, "X")
    T, out = dY.shape
    in_ = X.shape[1]
    _need(meta, torch.int16, "meta", (out, in_ // 16))
    _need(dW_vals, torch.bfloat16, "dW_vals", (out, in_ // 2))
    _lib.call("slope_bwd_dw_masked_noalloc", _ptr(dY), _ptr(X), _ptr(meta), T, in_, out, _ptr(dW_vals), _stream())
    return dW_vals


# The calls below may be a few microseconds of GPU work each, so they go through
# the module _calls (csrc/calls.cpp) when everything fits: 4.5 us of host time
# for fwd_q8 where the way from here takes 10.1.  What does not fit (another
# device than the current one, a subclass, a vector that does not start on 16
# bytes, an error) goes the way from here,
# with its messages; so does everything where the module was not built.
_calls = None


class _NoCalls:
    """Stands for the module _calls where there is none for this Python and torch: leaves every call."""
    rmsnorm = rmsnorm_bwd = quant_rows = fwd_q8 = staticmethod(lambda *a: None)


def _bind():
    """The module _calls, on the entry points of the loaded library."""
    global _calls
    from . import build
    try:
        if not build.calls_current():
            raise ImportError("not built for this Python and torch")
        from . import _calls as calls
    except ImportError as e:
        warnings.warn(f"_calls.so is not used ({e}); the int8 path's small calls take twice the host time: run "
                      "structured_sparse_pretraining_b200/build.py", RuntimeWarning, stacklevel=3)
        _lib.load()
        _calls = _NoCalls
        return _calls
    lib = _lib.load()
    names = ("rmsnorm", "rmsnorm_bwd", "rmsnorm_bwd_ws", "quant_rows", "fwd_q8")
    calls.bind(*(ctypes.cast(getattr(lib, "slope_" + n), ctypes.c_void_p).value for n in names))
    _calls = calls
    return calls


def _done(out):
    """The result of a call through _calls, or its status raised."""
    if type(out) is int:
        raise _lib.error(out)
    return out


def _fit(t, dtype, name, shape, dev):
    """t as a contiguous CUDA tensor of `dtype` and `shape` on device `dev`, or an error."""
    if t is not None and t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr()
    _need(t, dtype, name, shape)
    raise ValueError(f"{name} is on {t.device}: every tensor of a call must be on one device")


def _rows(t, dtype, name):
    """(rows, columns) of a contiguous two-dimensional CUDA tensor."""
    if t is not None and t.dtype is dtype and t.is_cuda and t.dim() == 2 and t.is_contiguous():
        return t.shape
    _need(t, dtype, name)
    raise ValueError(f"{name} has shape {tuple(t.shape)}, expected two dimensions")


def _place(t):
    """(device index of a CUDA tensor, whether it is the current device)."""
    dev = t.get_device()
    return dev, dev == torch.cuda.current_device()


def _out(t, dtype, name, shape, like, place):
    """(output tensor, pointer): the given one, checked, or a new one."""
    if t is None:
        t = like.new_empty(shape, dtype=dtype)
        return t, t.data_ptr()
    return t, _fit(t, dtype, name, shape, place[0])


# fp32 vectors (scales, rstd, dw) may be slices, s[3:], that do not start on the
# 16 bytes that the entry points ask of every tensor: such a one goes through a
# copy of its own, one more small launch.
def _vector(t, name, shape, dev):
    """(vector, pointer) of an fp32 input, copied where it does not start on 16 bytes."""
    p = _fit(t, torch.float32, name, shape, dev)
    if p % 16:
        t = t.clone()
        p = t.data_ptr()
    return t, p


def _vector_out(t, name, shape, like, place, back):
    """(vector, pointer) of an fp32 output; where the given one does not start on 16 bytes the pointer is that of a new
    one, and `back` takes the name and the two for _write_back."""
    t, p = _out(t, torch.float32, name, shape, like, place)
    if p % 16:
        new = torch.empty_like(t)
        back.append((name, t, new))
        p = new.data_ptr()
    return t, p


def _span(t):
    return t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()


def _check_back(back, call, **tensors):
    """Refuse what the entry point cannot see behind the copies: a vector of `back` that overlaps another buffer."""
    for name, t, _ in back:
        a, b = _span(t)
        for other, o in tensors.items():
            if o is None or other == name:
                continue
            c, d = _span(o)
            if a < d and c < b:
                raise ValueError(f"{call}: {name} overlaps {other}")


def _write_back(back):
    for _, t, new in back:
        t.copy_(new)


def _call_on(place, name, *args):
    """Call an entry point on the device of `place` (current or not) and that device's current stream."""
    dev, current = place
    stream = torch._C._cuda_getCurrentRawStream(dev)
    if current:
        return _lib.call(name, *args, stream)
    with torch.cuda.device(dev):
        return _lib.call(name, *args, stream)


def _norm_bwd_floats(T, D):
    floats = ctypes.c_int64(0)
    _lib.call("slope_rmsnorm_bwd_ws", T, D, ctypes.byref(floats))
    return floats.value


def rmsnorm(X, w, eps, res=None, with_rstd=False, H=None, Y=None, rstd=None):
    """(Y, H, rstd): h = bf16(X + res), Y = h rstd w with rstd = (mean h^2 + eps)^(-1/2)
    per token.  X, res [T, D] bf16, w [D] bf16.  H (h, the residual stream) is
    None without res; rstd [T] fp32 is written with with_rstd (rmsnorm_bwd
    needs it), else None."""
    return _rmsnorm(X, w, eps, res, True, False, with_rstd, H, Y, None, None, rstd)[2:]


def rmsnorm_q8(X, w, eps, res=None, with_y=False, with_rstd=False, H=None, Y=None, Q=None, qscale=None, rstd=None):
    """(Q, qscale, Y, H, rstd): rmsnorm with its output in int8, Q [T, D] with
    one scale per token (Q qscale stands for h rstd w), and with with_y in bf16
    too (the adapter's product reads that)."""
    return _rmsnorm(X, w, eps, res, with_y or Y is not None, True, with_rstd, H, Y, Q, qscale, rstd)


def _rmsnorm(X, w, eps, res, with_y, with_q8, with_rstd, H, Y, Q, qscale, rstd):
    out = (_calls or _bind()).rmsnorm(X, w, eps, res, with_y, with_q8, with_rstd, H, Y, Q, qscale, rstd)
    if out is not None:
        return _done(out)
    shape = T, D = tuple(_rows(X, torch.bfloat16, "X"))
    dev, _ = place = _place(X)
    pw = _fit(w, torch.bfloat16, "w", (D,), dev)
    pe = ph = py = pq = ps = pr = None
    back = []
    if res is not None:
        pe = _fit(res, torch.bfloat16, "res", shape, dev)
        H, ph = _out(H, torch.bfloat16, "H", shape, X, place)
    elif H is not None:
        raise ValueError("H without res (H would be X)")
    if with_y:
        Y, py = _out(Y, torch.bfloat16, "Y", shape, X, place)
    if with_q8:
        Q, pq = _out(Q, torch.int8, "Q", shape, X, place)
        qscale, ps = _vector_out(qscale, "qscale", (T,), X, place, back)
    if with_rstd or rstd is not None:
        rstd, pr = _vector_out(rstd, "rstd", (T,), X, place, back)
    _check_back(back, "rmsnorm", X=X, res=res, w=w, H=H if res is not None else None, Y=Y if with_y else None,
                Q=Q if with_q8 else None, qscale=qscale if with_q8 else None, rstd=rstd)
    _call_on(place, "slope_rmsnorm", X.data_ptr(), pe, pw, T, D, eps, ph, py, pq, ps, pr)
    _write_back(back)
    return Q, qscale, Y, H, rstd


def rmsnorm_bwd(dY, H, w, rstd, dres=None, dH=None, dw=None):
    """(dH, dw): gradients of rmsnorm's Y with respect to h (X and res both
    take dH; dres, the gradient reaching h along the residual stream, is added)
    [T, D] bf16 and to w [D] fp32.  H is rmsnorm's (or X without a residual)."""
    out = (_calls or _bind()).rmsnorm_bwd(dY, H, w, rstd, dres, dH, dw)
    if out is not None:
        return _done(out)
    shape = T, D = tuple(_rows(dY, torch.bfloat16, "dY"))
    dev, _ = place = _place(dY)
    ph = _fit(H, torch.bfloat16, "H", shape, dev)
    pw = _fit(w, torch.bfloat16, "w", (D,), dev)
    aligned, pr = _vector(rstd, "rstd", (T,), dev)  # (held until the call)
    pe = None if dres is None else _fit(dres, torch.bfloat16, "dres", shape, dev)
    dH, pdh = _out(dH, torch.bfloat16, "dH", shape, dY, place)
    back = []
    dw, pdw = _vector_out(dw, "dw", (D,), dY, place, back)
    _check_back(back, "rmsnorm_bwd", dY=dY, H=H, w=w, rstd=rstd, dres=dres, dH=dH, dw=dw)
    floats = _norm_bwd_floats(T, D)
    ws, pws = _out(None, torch.float32, "ws", (floats,), dY, place) if floats else (None, None)
    _call_on(place, "slope_rmsnorm_bwd", dY.data_ptr(), ph, pw, pr, pe, T, D, pdh, pdw, pws, floats)
    _write_back(back)
    return dH, dw


def quant_rows(A, Q=None, scale=None):
    """(Q, scale): rows of A [rows, K] bf16 in int8 with one fp32 scale per row
    (the kept weights of prune24: one per output channel)."""
    out = (_calls or _bind()).quant_rows(A, Q, scale)
    if out is not None:
        return _done(out)
    shape = rows, K = tuple(_rows(A, torch.bfloat16, "A"))
    place = _place(A)
    Q, pq = _out(Q, torch.int8, "Q", shape, A, place)
    back = []
    scale, ps = _vector_out(scale, "scale", (rows,), A, place, back)
    _check_back(back, "quant_rows", A=A, Q=Q, scale=scale)
    _call_on(place, "slope_quant_rows", A.data_ptr(), rows, K, pq, ps)
    _write_back(back)
    return Q, scale


def fwd_q8(Xq, xscale, vals_q, wscale, meta, XL, R, out_features, Y=None):
    """Y [T, out] bf16 = xscale wscale (Xq . Wq^T) + XL . R: fwd in int8, with
    Xq [T, in] and xscale [T] from rmsnorm_q8 or quant_rows, and vals_q
    [out, in/2], wscale [out] the kept weights through quant_rows (XL, R None:
    no adapter)."""
    out = (_calls or _bind()).fwd_q8(Xq, xscale, vals_q, wscale, meta, XL, R, out_features, Y)
    if out is not None:
        return _done(out)
    T, in_ = _rows(Xq, torch.int8, "Xq")
    dev, _ = place = _place(Xq)
    xscale, ps = _vector(xscale, "xscale", (T,), dev)
    pv = _fit(vals_q, torch.int8, "vals_q", (out_features, in_ // 2), dev)
    wscale, pws = _vector(wscale, "wscale", (out_features,), dev)
    pm = _fit(meta, torch.int16, "meta", (out_features, in_ // 16), dev)
    r, px, pr = 0, None, None
    if R is not None:
        r = _rows(R, torch.bfloat16, "R")[0]
        pr = _fit(R, torch.bfloat16, "R", (r, out_features), dev)
        px = _fit(XL, torch.bfloat16, "XL", (T, r), dev)
    elif XL is not None:
        raise ValueError("XL without R")
    Y, py = _out(Y, torch.bfloat16, "Y", (T, out_features), Xq, place)
    _call_on(place, "slope_fwd_q8", Xq.data_ptr(), ps, pv, pws, pm, px, pr, T, in_, out_features, r, py)
    return Y


def q8_plan(M, T, K, r=0, sms=148):
    """(rows, token width, splits) of fwd_q8's launch for M output channels, T
    tokens, K input features and rank r (rows 0: CUDA cores; host-only query)."""
    rows, bn, splits = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    _lib.call("slope_q8_plan", M, T, K, r, sms, ctypes.byref(rows), ctypes.byref(bn), ctypes.byref(splits))
    return rows.value, bn.value, splits.value


def sparse_plan(M, T, K, sms=148):
    """(BN, splits) the sparse products use for an M x K operand and T tokens
    on a device with `sms` SMs (host-only query, no GPU needed)."""
    bn, splits = ctypes.c_int(0), ctypes.c_int(0)
    _lib.call("slope_sparse_plan", M, T, K, sms, ctypes.byref(bn), ctypes.byref(splits))
    return bn.value, splits.value


def sparse_tile_rows(M, T, K, sms=148):
    """Output-tile height (256 or 512 rows) the sparse products use for an
    M x K operand and T tokens (host-only query, no GPU needed)."""
    rows = ctypes.c_int(0)
    _lib.call("slope_sparse_tile_rows", M, T, K, sms, ctypes.byref(rows))
    return rows.value


def fused_launches(M, T, K, r, sms=148):
    """Launches (1 or 2) of fwd_fused (M = out, K = in) or bwd_dx_fused
    (M = in, K = out) for these sizes (host-only query, no GPU needed)."""
    n = ctypes.c_int(0)
    _lib.call("slope_fused_launches", M, T, K, r, sms, ctypes.byref(n))
    return n.value


def status_sync():
    """Wait for the current stream and raise if a kernel flagged an error."""
    _lib.call("slope_status_sync", _stream())


def selftest_wait_timeout():
    """Launch the failure-path self-test: a bounded wait that runs out; the next
    status_sync raises SlopeError with SLOPE_ERR_TIMEOUT (5)."""
    _lib.call("slope_selftest_wait_timeout", _stream())


def device_check():
    _lib.call("slope_device_check")


def launch_count(reset=False):
    return int(_lib.load().slope_launch_count(1 if reset else 0))
