"""Python binding of include/hkg_linear.h: the 16-bit linear layer with bias,
activation, dropout and residual in its epilogue, its gradients, and dropout by
itself, on GPU tensors.

    y = linear(x, W, bias, activation="gelu", residual=r, p=0.1, rng=(seed, offset), z=z)
    dx, dw, dbias = linear_backward(dy, x, W, z=z, activation="gelu", p=0.1, rng=(seed, offset))
    out = dropout(x, 0.1, (seed, offset), residual=r)

`rng` decides which elements dropout drops: (seed, offset), two whole numbers below
2^64, or an int64 GPU tensor that holds them and is read when the kernels run (a
captured graph takes other masks when it is changed between replays).  No mask is
stored: the backward pass takes the same rng.  Calls that shall drop independently
take different offsets.

Streams, outputs, workspaces and errors are those of the other operators (ops.py).
"""
from __future__ import annotations

import ctypes

import dense_gemm_fp8_amd as _hkg

from . import ops as _ops

HKG_T_F16 = 2
HKG_ACTIVATIONS = {None: 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}

# exported symbols, in the order include/hkg_linear.h declares them
LINEAR_EXPORTS = (
    "hkg_dropout",
    "hkg_linear_workspace_bytes",
    "hkg_linear",
    "hkg_linear_backward_workspace_bytes",
    "hkg_linear_backward",
)


class hkg_dropout_opts(ctypes.Structure):
    _fields_ = [("p", ctypes.c_float), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64), ("rng", ctypes.c_void_p)]


class hkg_epilogue(ctypes.Structure):
    _fields_ = [("bias", ctypes.c_void_p), ("bias_type", ctypes.c_int32), ("activation", ctypes.c_int32),
                ("residual", ctypes.c_void_p), ("ldr", ctypes.c_int64),
                ("z", ctypes.c_void_p), ("ldz", ctypes.c_int64), ("dropout", hkg_dropout_opts)]


_typed = None


def _lib():
    """The library the operators use, with the argument types of hkg_linear.h set."""
    global _typed
    lib = _ops._lib()
    if lib is not _typed:
        i64, i32, p = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p
        drop, epi = ctypes.POINTER(hkg_dropout_opts), ctypes.POINTER(hkg_epilogue)
        sig = {
            "hkg_dropout": [i64, i64, p, i32, i64, drop, p, i64, p, i32, i64, p],
            "hkg_linear_workspace_bytes": [i64, i64, i64],
            "hkg_linear": [i64, i64, i64, i32, p, i64, p, i64, epi, p, i32, i64, p, i64, p],
            "hkg_linear_backward_workspace_bytes": [i64, i64, i64],
            "hkg_linear_backward": [i64, i64, i64, i32, p, i32, i64, p, i64, p, i64, p, i64, i32, drop, p, i64, p, i64, p,
                                    p, i64, p],
        }
        for name, args in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = i64 if name.endswith("_bytes") else ctypes.c_int
        _typed = lib
    return lib


def _on(t):
    _lib()
    return _ops._on(t)


def _types():
    import torch
    return {torch.bfloat16: _ops.HKG_T_BF16, torch.float32: _ops.HKG_T_F32, torch.float16: HKG_T_F16}


def _type(t, name, allowed=None) -> int:
    """HKG_T_* of t, which has to be bf16, fp16 or fp32, or of one of the types `allowed`."""
    code = _types().get(t.dtype)
    if code is None or (allowed is not None and t.dtype not in allowed):
        raise TypeError("%s must be %s" % (name, " or ".join(str(d) for d in (allowed or _types()))))
    return code


def _operand(t, name):
    """(HKG_T_*, pointer, pitch) of a matrix of bf16 or fp16 values."""
    import torch
    code = _type(t, name, (torch.bfloat16, torch.float16))
    return (code, *_hkg._matrix(t, name))


def _beside(t, shape, like, name):
    """(pointer, pitch) of a matrix of `shape` that is of like's type, or None."""
    if t is None:
        return None, 0
    if tuple(t.shape) != tuple(shape) or t.dtype is not like:
        raise ValueError("%s must be a %s tensor of shape %s" % (name, like, tuple(shape)))
    return _hkg._matrix(t, name)


def _activation(name) -> int:
    if name not in HKG_ACTIVATIONS:
        raise ValueError("activation must be one of %s" % ", ".join(repr(k) for k in HKG_ACTIVATIONS))
    return HKG_ACTIVATIONS[name]


def _dropout(opts, p, rng):
    """Fill `opts`; -> the GPU tensor of rng, or None."""
    p = float(p)
    if not 0.0 <= p <= 1.0:
        raise ValueError("p must be in 0 .. 1")
    opts.p = p
    if p == 0.0:
        return None
    if rng is None:
        raise ValueError("dropout needs rng: (seed, offset), or an int64 GPU tensor of the two")
    if isinstance(rng, (tuple, list)):
        seed, offset = (int(v) for v in rng)
        if not (0 <= seed < 1 << 64 and 0 <= offset < 1 << 64):
            raise ValueError("seed and offset must be in 0 .. 2^64 - 1")
        opts.seed, opts.offset = seed, offset
        return None
    import torch
    if rng.dtype is not torch.int64 or tuple(rng.shape) != (2,):
        raise ValueError("rng must be (seed, offset), or an int64 GPU tensor of the two")
    opts.rng = _hkg._dev_ptr(rng, "rng")
    return rng


def dropout(x, p, rng, residual=None, out=None, stream=None):
    """residual + D(x) for x [rows, cols] (bf16, fp16 or fp32, rows contiguous): an
    element is dropped with probability p (rounded to a multiple of 2^-16), the others
    are divided by 1 - p.  Its own backward pass on dy, with the same rng.  out: of x's
    type or fp32, default a new tensor of residual's type, or x's; residual has out's
    type; out may be x or residual itself."""
    code = _type(x, "x")
    px, ldx = _hkg._matrix(x, "x")
    shape = tuple(x.shape)
    opts = hkg_dropout_opts()
    drawn = _dropout(opts, p, rng)
    like = out if out is not None else residual if residual is not None else x
    out_code = _type(like, "out")
    pr, ldr = _beside(residual, shape, like.dtype, "residual")
    st = _ops._handle(stream, x, residual, out, drawn)
    out, po, ldo = _ops._output(out, shape, like.dtype, "out", x, stream)
    _ops._check(_on(x).hkg_dropout(shape[0], shape[1], px, code, ldx, opts, pr, ldr, po, out_code, ldo, st), "hkg_dropout")
    return out


def linear(x, W, bias=None, activation=None, residual=None, p=0.0, rng=None, y=None, z=None, workspace=None, stream=None):
    """y [M,N] = residual + D(act(x [M,K] · W [N,K]ᵀ + bias)), x and W bf16 or fp16.
    bias [N]: of their type or fp32.  activation: None, "relu", "gelu", "gelu_tanh" or
    "silu".  residual: of y's type; y may be the residual itself.  p, rng: dropout.
    y: of x's type or fp32, default a new tensor of residual's type, or x's.
    z: a tensor [M,N] of x's type that receives x Wᵀ + bias, for linear_backward."""
    code, px, ldx = _operand(x, "x")
    M, K = x.shape
    N = W.shape[0]
    pw, ldw = _beside(W, (N, K), x.dtype, "W")
    e = hkg_epilogue()
    if bias is not None:
        e.bias_type = _type(bias, "bias")
        if tuple(bias.shape) != (N,):
            raise ValueError("bias must be [%d]" % N)
        e.bias = _hkg._dev_ptr(bias, "bias")
    e.activation = _activation(activation)
    drawn = _dropout(e.dropout, p, rng)
    like = y if y is not None else residual if residual is not None else x
    y_code = _type(like, "y")
    e.residual, e.ldr = _beside(residual, (M, N), like.dtype, "residual")
    e.z, e.ldz = _beside(z, (M, N), x.dtype, "z")
    st = _ops._handle(stream, x, W, bias, residual, y, z, drawn, workspace)
    y, py, ldy = _ops._output(y, (M, N), like.dtype, "y", x, stream)
    need = _ops._check(_lib().hkg_linear_workspace_bytes(M, N, K), "hkg_linear_workspace_bytes")
    workspace, pws, nws = _ops._workspace(workspace, need, x, stream)
    _ops._check(_on(x).hkg_linear(M, N, K, code, px, ldx, pw, ldw, e, py, y_code, ldy, pws, nws, st), "hkg_linear")
    return y


def linear_backward(dy, x, W, z=None, activation=None, p=0.0, rng=None, dx=None, dw=None, dbias=None, need_dx=True,
                    need_dw=True, need_dbias=True, workspace=None, stream=None):
    """Gradients of linear(): (dx [M,K], dw [N,K], dbias [N] fp32) from dy [M,N] (x's
    type or fp32) and the z that linear() kept (unused without an activation), with the
    p and rng of the forward call; the residual's gradient is dy itself.  need_*: which
    to compute; the others come back as None (W may be None without dx, x without dw, not
    both)."""
    import torch
    if x is None and W is None:
        raise ValueError("x or W is needed")
    like = x if x is not None else W
    code = _type(like, "x" if x is not None else "W", (torch.bfloat16, torch.float16))
    M, N = dy.shape
    K = like.shape[1]
    dy_code = _type(dy, "dy", (like.dtype, torch.float32))
    pdy, lddy = _hkg._matrix(dy, "dy")
    if (need_dx and W is None) or (need_dw and x is None):
        raise ValueError("dx needs W, dw needs x")
    px, ldx = _beside(x, (M, K), like.dtype, "x")
    pw, ldw = _beside(W, (N, K), like.dtype, "W")
    act = _activation(activation)
    if act and z is None:
        raise ValueError("an activation's gradient needs z")
    pz, ldz = _beside(z, (M, N), like.dtype, "z")
    opts = hkg_dropout_opts()
    drawn = _dropout(opts, p, rng)
    st = _ops._handle(stream, dy, x, W, z, dx, dw, dbias, drawn, workspace)
    pdx = pdw = pdb = None
    lddx = lddw = 0
    if need_dx:
        dx, pdx, lddx = _ops._output(dx, (M, K), like.dtype, "dx", dy, stream)
    if need_dw:
        dw, pdw, lddw = _ops._output(dw, (N, K), like.dtype, "dw", dy, stream)
    if need_dbias:
        if dbias is None:
            dbias = _ops._empty((N,), torch.float32, dy, stream)
            pdb = dbias.data_ptr()
        elif tuple(dbias.shape) != (N,) or dbias.dtype is not torch.float32:
            raise ValueError("dbias must be a float32 tensor of shape (%d,)" % N)
        else:
            pdb = _hkg._dev_ptr(dbias, "dbias")
    need = _ops._check(_lib().hkg_linear_backward_workspace_bytes(M, N, K), "hkg_linear_backward_workspace_bytes")
    workspace, pws, nws = _ops._workspace(workspace, need, dy, stream)
    _ops._check(_on(dy).hkg_linear_backward(M, N, K, code, pdy, dy_code, lddy, px, ldx, pw, ldw, pz, ldz, act, opts, pdx, lddx,
                                            pdw, lddw, pdb, pws, nws, st), "hkg_linear_backward")
    return dx if need_dx else None, dw if need_dw else None, dbias if need_dbias else None
