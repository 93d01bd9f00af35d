"""Sequence operators on PyTorch device tensors: what stands around a causal
depthwise convolution in a recurrent language-model layer.

    y, h_last = glr_fwd(x, r, i, lam, h0=h)            # a prompt
    y, h = glr_step(x, r, i, lam, h)                   # one token, h updated in place
    y, h_last, states = glr_fwd(..., save=True)        # training:
    dx, dr, di, dlam, dh0 = glr_bwd(dy, x, r, i, lam, states)
    q, scale, total = rmsnorm_q8(x, weight, residual=res)
    y = matmul_q8(q, scale, w_q, w_scale)

Argument checks, output allocation and marshalling only: every operation runs
in the HIP kernels of libgconv.so (``include/gconv.h`` states what each
computes).  There is no fallback; if the library has not been built, the
first call raises ``gconv.GconvUnavailable``.

Activations need unit stride along their last axis; their other strides are
free, so slices of a wider projection are taken as they are.  A call runs on
the current stream of its tensors' device, or on ``stream`` (a hipStream_t as
an int, 0 the default stream), and then its outputs and workspace are allocated for that stream.

A call's arguments are checked once per set of sizes, strides, types and
devices; the descriptor made then is kept under these (of an address, only
its alignment), so that a call for one token costs little more than its launch.
"""
from __future__ import annotations

import ctypes

import torch

from . import gconv as G

try:
    from torch._C import _cuda_getCurrentRawStream as _raw_stream   # a tenth of current_stream()'s time
except ImportError:
    def _raw_stream(index):
        return torch.cuda.current_stream(index).cuda_stream

try:
    from torch._C import _cuda_getDevice as _current_device   # a GPU tensor is there: nothing is left to initialise
except ImportError:
    _current_device = torch.cuda.current_device

_CODES = {torch.float32: G.GCONV_F32, torch.float16: G.GCONV_F16, torch.bfloat16: G.GCONV_BF16}
_MOST_PLANS = 4096
_plans: dict = {}


def _meta(t):
    """What a plan may depend on of an argument."""
    return None if t is None else (t.shape, t.dtype, t.stride(), t.get_device())


def _keep(key, plan):
    if len(_plans) >= _MOST_PLANS:
        _plans.clear()
    _plans[key] = plan
    return plan


def _here(t):
    """Whether t is on the current device, where calls go without further ado."""
    k = t.get_device()
    return k >= 0 and k == _current_device()


def _elsewhere(f, t, stream, *args, **kw):
    """f on t's device, and on `stream` where one is given."""
    if not t.is_cuda:
        raise ValueError("%s takes tensors on the GPU" % f.__name__)
    with torch.cuda.device(t.device):
        if stream is None:
            return f(*args, **kw)
        # 0 is the default stream's handle; ExternalStream takes it for a request for a new stream
        on = torch.cuda.ExternalStream(stream, device=t.device) if stream else torch.cuda.default_stream(t.device)
        with torch.cuda.stream(on):
            return f(*args, **kw)


def _check(name, t, shape, dtype, like, packed=False):
    """t is a tensor of this shape, type and like's device with unit stride along its last axis (or packed)."""
    if t.shape != shape:
        raise ValueError("%s must have shape %s, not %s" % (name, tuple(shape), tuple(t.shape)))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, not %s" % (name, dtype, t.dtype))
    if t.device != like.device:
        raise ValueError("%s is on %s, not on %s" % (name, t.device, like.device))
    if packed:
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)
    elif shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError("%s must have unit stride along its last axis" % name)


def _check_written(name, t, shape, dtype, like):
    """_check, and no two elements of t share memory."""
    _check(name, t, shape, dtype, like)
    reach = 1
    for st, n in sorted((st, n) for n, st in zip(t.shape, t.stride()) if n > 1):
        if st < reach:
            raise ValueError("%s's elements overlap" % name)
        reach += (n - 1) * st


def _check_type(t):
    if t.dtype not in _CODES:
        raise TypeError("unsupported dtype %s" % t.dtype)


def _packed_like(t):
    """A new packed tensor of t's shape and type."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _raise(rc, what):
    raise G.GconvError(rc, what)


def _room(ws, need, like):
    """(address, bytes, owner) of the caller's workspace or of a new one."""
    if ws is None:
        if not need:
            return None, 0, None
        ws = torch.empty_strided((need,), (1,), dtype=torch.uint8, device=like.device)
    elif ws.device != like.device or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s" % like.device)
    return ws.data_ptr(), ws.numel() * ws.element_size(), ws


# ------------------------------------------------- gated linear recurrence


def _rows(t, packed):
    """(batch, time) strides of [B, L, D]; an axis of one step needs none.  packed: of a tensor still to be made."""
    B, L, D = t.shape
    b, l = (L * D, D) if packed else t.stride()[:2]
    return (ctypes.c_int64 * 2)(b if B > 1 else 0, l if L > 1 else 0)


def _glr_desc(x, c):
    if x.shape[-1] < 1:
        raise ValueError("the last axis must hold at least one channel")
    _check_type(x)
    B, L, D = x.shape
    return G.gconv_glr_desc(dtype=_CODES[x.dtype], c=c, B=B, L=L, D=D)


def _glr_inputs(x, r, i, lam, lengths):
    if x.dim() != 3:
        raise ValueError("x must be [B, L, D]")
    for name, t in (("x", x), ("r", r), ("i", i)):
        _check(name, t, x.shape, x.dtype, x)
    _check("lam", lam, x.shape[-1:], torch.float32, x, packed=True)
    if lengths is not None:
        _check("lengths", lengths, x.shape[:1], torch.int32, x, packed=True)


def _states_shape(x):
    return (x.shape[0], -(-x.shape[1] // G.GCONV_GLR_SPAN), x.shape[2])


def _plan_fwd(key, x, r, i, lam, h0, lengths, c, out, h_last, states):
    _glr_inputs(x, r, i, lam, lengths)
    B, L, D = x.shape
    for name, t in (("h0", h0), ("h_last", h_last)):
        if t is not None:
            _check(name, t, (B, D), torch.float32, x, packed=True)
    if out is not None:
        _check_written("out", out, x.shape, x.dtype, x)
    if states is not None:
        _check("states", states, _states_shape(x), torch.float32, x, packed=True)
    d = _glr_desc(x, c)
    d.x_stride, d.r_stride, d.i_stride = (_rows(t, False) for t in (x, r, i))
    d.y_stride = _rows(x if out is None else out, out is None)
    n = ctypes.c_size_t()
    rc = G.lib().gconv_glr_fwd_workspace(ctypes.byref(d), ctypes.byref(n))
    if rc:
        _raise(rc, "gconv_glr_fwd")
    return _keep(key, (ctypes.byref(d), n.value))


def glr_fwd(x, r, i, lam, h0=None, lengths=None, c=8.0, save=False, out=None, h_last=None, states=None,
            workspace=None, stream=None):
    """Gated linear recurrence over x, r, i [B, L, D]: (y, h_last), or (y, h_last, states) with ``save``.

    Per channel, h = a h + sqrt(1 - a^2) sigmoid(i) x with log a = -c
    softplus(lam) sigmoid(r); y is h at every step, in x's type.  lam: fp32
    [D]; h0 and h_last: fp32 [B, D], h0 None for zeros, and h_last may be h0
    itself.  lengths: int32 [B] on the device; past its length a row's y is 0
    and its state stays.  states: fp32 [B, ceil(L / 64), D], what glr_bwd
    starts from.  out, h_last, states and workspace are allocated unless
    given.
    """
    if stream is not None or not _here(x):
        return _elsewhere(glr_fwd, x, stream, x, r, i, lam, h0, lengths, c, save, out, h_last, states, workspace)
    key = (0, c, _meta(x), _meta(r), _meta(i), _meta(lam), _meta(h0), _meta(lengths), _meta(out), _meta(h_last),
           _meta(states))
    d, need = _plans.get(key) or _plan_fwd(key, x, r, i, lam, h0, lengths, c, out, h_last, states)
    B, L, D = x.shape
    if out is None:
        out = _packed_like(x)
    if h_last is None:
        h_last = torch.empty_strided((B, D), (D, 1), dtype=torch.float32, device=x.device)
    if save and states is None:
        n = -(-L // G.GCONV_GLR_SPAN)
        states = torch.empty_strided((B, n, D), (n * D, D, 1), dtype=torch.float32, device=x.device)
    ws, nbytes, owner = _room(workspace, need, x)
    rc = G.lib().gconv_glr_fwd(d, x.data_ptr(), r.data_ptr(), i.data_ptr(), lam.data_ptr(), _ptr(h0), _ptr(lengths),
                               out.data_ptr(), h_last.data_ptr(), _ptr(states), ws, nbytes,
                               _raw_stream(x.get_device()))
    if rc:
        _raise(rc, "gconv_glr_fwd")
    return (out, h_last, states) if save else (out, h_last)


def _plan_step(key, x, r, i, lam, h, c, out, h_out):
    if x.dim() != 2:
        raise ValueError("x must be [B, D]")
    _check("h", h, x.shape, torch.float32, x, packed=True)
    if h_out is not None:
        _check("h_out", h_out, x.shape, torch.float32, x, packed=True)
    if out is not None:
        _check_written("out", out, x.shape, x.dtype, x)
        out = out[:, None]
    x, r, i = (t[:, None] if t.dim() == 2 else t for t in (x, r, i))
    _glr_inputs(x, r, i, lam, None)
    d = _glr_desc(x, c)
    d.x_stride, d.r_stride, d.i_stride = (_rows(t, False) for t in (x, r, i))
    d.y_stride = _rows(x if out is None else out, out is None)
    rc = G.lib().gconv_glr_fwd_workspace(ctypes.byref(d), ctypes.byref(ctypes.c_size_t()))
    if rc:
        _raise(rc, "gconv_glr_fwd")
    return _keep(key, ctypes.byref(d))


def glr_step(x, r, i, lam, h, c=8.0, out=None, h_out=None, stream=None):
    """One token: x, r, i [B, D] and the state h (fp32 [B, D]); (y, h_out), h_out being h itself unless given."""
    if stream is not None or not _here(x):
        return _elsewhere(glr_step, x, stream, x, r, i, lam, h, c, out, h_out)
    key = (1, c, _meta(x), _meta(r), _meta(i), _meta(lam), _meta(h), _meta(out), _meta(h_out))
    d = _plans.get(key) or _plan_step(key, x, r, i, lam, h, c, out, h_out)
    if out is None:
        out = _packed_like(x)
    if h_out is None:
        h_out = h
    rc = G.lib().gconv_glr_fwd(d, x.data_ptr(), r.data_ptr(), i.data_ptr(), lam.data_ptr(), h.data_ptr(), None,
                               out.data_ptr(), h_out.data_ptr(), None, None, 0, _raw_stream(x.get_device()))
    if rc:
        _raise(rc, "gconv_glr_fwd")
    return out, h_out


def _plan_bwd(key, dy, x, r, i, lam, states, lengths, dh_last, c, grads):
    _glr_inputs(x, r, i, lam, lengths)
    B, L, D = x.shape
    _check("dy", dy, x.shape, x.dtype, x)
    _check("states", states, _states_shape(x), torch.float32, x, packed=True)
    if dh_last is not None:
        _check("dh_last", dh_last, (B, D), torch.float32, x, packed=True)
    d = _glr_desc(x, c)
    d.x_stride, d.r_stride, d.i_stride, d.y_stride = (_rows(t, False) for t in (x, r, i, dy))
    for name, t in zip(("dx", "dr", "di"), grads):
        if t is not None:
            _check_written(name, t, x.shape, x.dtype, x)
        setattr(d, name + "_stride", _rows(x if t is None else t, t is None))
    n = ctypes.c_size_t()
    rc = G.lib().gconv_glr_bwd_workspace(ctypes.byref(d), ctypes.byref(n), None)
    if rc:
        _raise(rc, "gconv_glr_bwd")
    return _keep(key, (ctypes.byref(d), n.value))


def glr_bwd(dy, x, r, i, lam, states, lengths=None, dh_last=None, c=8.0, dx=None, dr=None, di=None, workspace=None,
            stream=None):
    """Gradients of glr_fwd: (dx, dr, di, dlam, dh0).

    dy [B, L, D] is the gradient of y, dh_last (fp32 [B, D], None for zeros)
    that of h_last; x, r, i, lam, lengths and c as in the forward call, and
    states what it saved.  dx, dr and di are allocated packed unless given;
    dlam is fp32 [D], summed over batch and time, and dh0 fp32 [B, D].
    """
    if stream is not None or not _here(x):
        return _elsewhere(glr_bwd, x, stream, dy, x, r, i, lam, states, lengths, dh_last, c, dx, dr, di, workspace)
    key = (2, c, _meta(dy), _meta(x), _meta(r), _meta(i), _meta(lam), _meta(states), _meta(lengths), _meta(dh_last),
           _meta(dx), _meta(dr), _meta(di))
    d, need = _plans.get(key) or _plan_bwd(key, dy, x, r, i, lam, states, lengths, dh_last, c, (dx, dr, di))
    B, L, D = x.shape
    dx, dr, di = (_packed_like(x) if t is None else t for t in (dx, dr, di))
    dlam = torch.empty_strided((D,), (1,), dtype=torch.float32, device=x.device)
    dh0 = torch.empty_strided((B, D), (D, 1), dtype=torch.float32, device=x.device)
    ws, nbytes, owner = _room(workspace, need, x)
    rc = G.lib().gconv_glr_bwd(d, x.data_ptr(), r.data_ptr(), i.data_ptr(), lam.data_ptr(), _ptr(lengths),
                               states.data_ptr(), dy.data_ptr(), _ptr(dh_last), dx.data_ptr(), dr.data_ptr(),
                               di.data_ptr(), dlam.data_ptr(), dh0.data_ptr(), ws, nbytes, _raw_stream(x.get_device()))
    if rc:
        _raise(rc, "gconv_glr_bwd")
    return dx, dr, di, dlam, dh0


# ---------------------------------------------- 8-bit rows and their product


def _row(t, M, D):
    """The stride between rows of [M, D]; D of a tensor still to be made."""
    return D if t is None else t.stride(0) if M > 1 else 0


def _plan_q8(key, x, weight, residual, eps, q, scale, total):
    if x.dim() != 2 or x.shape[1] < 1:
        raise ValueError("x must be [M, D], D at least 1")
    _check_type(x)
    M, D = x.shape
    _check("x", x, x.shape, x.dtype, x)
    if weight is not None:
        _check("weight", weight, (D,), torch.float32, x, packed=True)
    if residual is not None:
        _check("residual", residual, x.shape, x.dtype, x)
        if total is not None:
            _check_written("total", total, x.shape, x.dtype, x)
    elif total is not None:
        raise ValueError("total needs a residual")
    if q is not None:
        _check_written("q", q, x.shape, torch.int8, x)
    if scale is not None:
        _check("scale", scale, (M,), torch.float32, x, packed=True)
    d = G.gconv_q8_desc(dtype=_CODES[x.dtype], eps=eps, M=M, D=D, x_stride=_row(x, M, D),
                        residual_stride=_row(residual, M, D), sum_stride=_row(total, M, D), q_stride=_row(q, M, D))
    return _keep(key, ctypes.byref(d))


def _codes(x, q, scale):
    if q is None:
        M, D = x.shape
        q = torch.empty_strided((M, D), (D, 1), dtype=torch.int8, device=x.device)
    if scale is None:
        scale = torch.empty_strided((x.shape[0],), (1,), dtype=torch.float32, device=x.device)
    return q, scale


def rmsnorm_q8(x, weight, residual=None, eps=1e-6, q=None, scale=None, total=None, stream=None):
    """Residual addition, root-mean-square norm and 8-bit rows: (q, scale, total).

    total = x + residual rounded to their type (x itself without a residual;
    given, it may be residual or x), and q * scale[:, None] stands for total /
    sqrt(mean(total^2) + eps) * weight.  x, residual: [M, D]; weight: fp32
    [D]; q: int8 [M, D]; scale: fp32 [M].
    """
    if stream is not None or not _here(x):
        return _elsewhere(rmsnorm_q8, x, stream, x, weight, residual, eps, q, scale, total)
    key = (3, eps, _meta(x), _meta(weight), _meta(residual), _meta(q), _meta(scale), _meta(total))
    d = _plans.get(key) or _plan_q8(key, x, weight, residual, eps, q, scale, total)
    q, scale = _codes(x, q, scale)
    if residual is not None and total is None:
        total = _packed_like(x)
    rc = G.lib().gconv_rmsnorm_q8(d, x.data_ptr(), _ptr(residual), weight.data_ptr(), q.data_ptr(), scale.data_ptr(),
                                  _ptr(total), _raw_stream(x.get_device()))
    if rc:
        _raise(rc, "gconv_rmsnorm_q8")
    return q, scale, x if total is None else total


def quant_q8(x, q=None, scale=None, stream=None):
    """8-bit rows of x [M, D] as they are (weights laid out once, activations without a norm): (q, scale)."""
    if stream is not None or not _here(x):
        return _elsewhere(quant_q8, x, stream, x, q, scale)
    key = (4, _meta(x), _meta(q), _meta(scale))
    d = _plans.get(key) or _plan_q8(key, x, None, None, 0.0, q, scale, None)
    q, scale = _codes(x, q, scale)
    rc = G.lib().gconv_quant_q8(d, x.data_ptr(), q.data_ptr(), scale.data_ptr(), _raw_stream(x.get_device()))
    if rc:
        _raise(rc, "gconv_quant_q8")
    return q, scale


def _plan_mm(key, a, a_scale, w, w_scale, bias, out_dtype, out):
    if a.dim() != 2 or w.dim() != 2 or w.shape[0] < 1 or w.shape[1] < 1:
        raise ValueError("a must be [M, K] and w [N, K], N and K at least 1")
    M, K = a.shape
    N = w.shape[0]
    _check("a", a, (M, K), torch.int8, a)
    _check("w", w, (N, K), torch.int8, a)
    _check("a_scale", a_scale, (M,), torch.float32, a, packed=True)
    _check("w_scale", w_scale, (N,), torch.float32, a, packed=True)
    if bias is not None:
        _check("bias", bias, (N,), torch.float32, a, packed=True)
    if out_dtype not in _CODES:
        raise TypeError("unsupported dtype %s" % out_dtype)
    if out is not None:
        _check_written("out", out, (M, N), out_dtype, a)
    d = G.gconv_mm_q8_desc(dtype=_CODES[out_dtype], M=M, N=N, K=K, a_stride=_row(a, M, K), w_stride=_row(w, N, K),
                           y_stride=_row(out, M, N))
    n = ctypes.c_size_t()
    rc = G.lib().gconv_matmul_q8_workspace(ctypes.byref(d), ctypes.byref(n))
    if rc:
        _raise(rc, "gconv_matmul_q8")
    pieces = (K | d.a_stride | d.w_stride | a.data_ptr() | w.data_ptr()) % 16 == 0   # rows need no laying out
    return _keep(key, (ctypes.byref(d), 0 if pieces else n.value))


def matmul_q8(a, a_scale, w, w_scale, bias=None, out_dtype=torch.bfloat16, out=None, workspace=None, stream=None):
    """y[m, n] = (sum_k a[m, k] w[n, k]) a_scale[m] w_scale[n] + bias[n], the sum exact in 32-bit integers.

    a: int8 [M, K]; w: int8 [N, K]; a_scale, w_scale and bias: fp32 [M], [N],
    [N]; y: [M, N] of out_dtype (out's own where it is given).
    """
    if stream is not None or not _here(a):
        return _elsewhere(matmul_q8, a, stream, a, a_scale, w, w_scale, bias, out_dtype, out, workspace)
    if out is not None:
        out_dtype = out.dtype
    key = (5, out_dtype, _meta(a), _meta(a_scale), _meta(w), _meta(w_scale), _meta(bias), _meta(out),
           (a.data_ptr() | w.data_ptr()) % 16)
    d, need = _plans.get(key) or _plan_mm(key, a, a_scale, w, w_scale, bias, out_dtype, out)
    if out is None:
        N = w.shape[0]
        out = torch.empty_strided((a.shape[0], N), (N, 1), dtype=out_dtype, device=a.device)
    ws, nbytes, owner = _room(workspace, need, a)
    rc = G.lib().gconv_matmul_q8(d, a.data_ptr(), a_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(), _ptr(bias),
                                 out.data_ptr(), ws, nbytes, _raw_stream(a.get_device()))
    if rc:
        _raise(rc, "gconv_matmul_q8")
    return out
