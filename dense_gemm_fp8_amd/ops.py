"""Python binding of include/hkg_ops.h: the MXFP4 linear layer and the
orthogonalised weight update, on GPU tensors.

An MXFP4 matrix is a pair (codes, packed): uint8 [rows, Kp / 2] with two e2m1
codes a byte (Kp = K rounded up to 32) and its E8M0 scales in packed order.

    w, sw, wt, swt = mxfp4_quantize_both(W, B, B)        # once per weight update
    x, sx, xt, sxt = mxfp4_quantize_both(X, A, B)        # a training step's input
    y = gemm_mxfp4(x, w, sx, sw)                         # its forward product
    dx, dw = linear_mxfp4_backward(dy, wt, swt, xt, sxt)
    W -= lr * orthogonalize(momentum)
    y = linear_mxfp4(X, w, sw)                           # serving, from one row up

with A, B = HKG_MX_OPERAND_A, HKG_MX_OPERAND_B.  Every function takes `stream`
(default: torch's current one on the tensors' GPU, whichever GPU is current) and
enqueues its work there; outputs and workspaces it allocates belong to that
stream.  All tensors of a call, and the stream, are on one GPU.  A failed check
raises HkgError with the library's status (ValueError / TypeError for tensors of
the wrong kind); nothing has run then.
"""
from __future__ import annotations

import ctypes

import dense_gemm_fp8_amd as _hkg

HKG_T_BF16 = 0
HKG_T_F32 = 1

# exported symbols, in the order include/hkg_ops.h declares them
OPS_EXPORTS = (
    "hkg_mxfp4_code_bytes",
    "hkg_mxfp4_quantize",
    "hkg_mxfp4_quantize_both",
    "hkg_mxfp4_dequantize",
    "hkg_gemm_mxfp4",
    "hkg_linear_mxfp4_workspace_bytes",
    "hkg_linear_mxfp4",
    "hkg_linear_mxfp4_backward_workspace_bytes",
    "hkg_linear_mxfp4_backward",
    "hkg_orthogonalize_workspace_bytes",
    "hkg_orthogonalize",
)

_ready = None
_raw_stream = None       # device index -> handle of torch's current stream there
_several = True          # whether there is more than one GPU that a tensor can be on


def _lib() -> ctypes.CDLL:
    """libhkg with the argument types of hkg_ops.h set."""
    global _ready, _raw_stream, _several
    if _ready is None:
        lib = _hkg.load()
        i64, i32, p, f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float
        sig = {
            "hkg_mxfp4_code_bytes": [i64, i64],
            "hkg_mxfp4_quantize": [i32, i64, i64, p, i32, i64, p, p, p],
            "hkg_mxfp4_quantize_both": [i32, i32, i64, i64, p, i32, i64, p, p, p, p, p],
            "hkg_mxfp4_dequantize": [i32, i64, i64, p, p, p, i32, i64, p],
            "hkg_gemm_mxfp4": [i64, i64, i64, p, p, p, p, p, p, i64, p],
            "hkg_linear_mxfp4_workspace_bytes": [i64, i64, i64],
            "hkg_linear_mxfp4": [i64, i64, i64, p, i32, i64, p, p, p, i64, p, i64, p],
            "hkg_linear_mxfp4_backward_workspace_bytes": [i64, i64, i64],
            "hkg_linear_mxfp4_backward": [i64, i64, i64, p, i32, i64, p, p, p, p, p, i64, p, i64, p,
                                          i64, p],
            "hkg_orthogonalize_workspace_bytes": [i64, i64],
            "hkg_orthogonalize": [i64, i64, p, i32, i64, i32, f32, f32, f32, f32, p, i64, p, i64, p],
        }
        for name, args in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = i64 if name.endswith("_bytes") else ctypes.c_int
        import torch
        # the handle alone costs a tenth of a torch Stream object, which is a good
        # part of a small call's time on the host
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda device: torch.cuda.current_stream(device).cuda_stream)
        _several = torch.cuda.device_count() > 1
        _ready = lib
    return _ready


def _check(rc, name):
    if rc < 0:
        raise _hkg.HkgError(rc, name)
    return rc


def _pad32(k: int) -> int:
    return (k + 31) & ~31


def _scale_bytes(rows: int, k: int) -> int:
    """hkg_mx_packed_scale_bytes(rows, k padded) for sizes the call itself will check."""
    return ((rows + 127) >> 7) * ((k + 127) >> 7) * 512


def _elem_type(t, name) -> int:
    import torch
    dt = t.dtype
    if dt is torch.bfloat16:
        return HKG_T_BF16
    if dt is torch.float32:
        return HKG_T_F32
    raise TypeError("%s must be bfloat16 or float32" % name)


def _codes(t, rows, K, name):
    """Pointer of the codes of a [rows, K] MXFP4 matrix."""
    import torch
    if t.dtype is not torch.uint8 or t.dim() != 2:
        raise TypeError("%s must be a 2-D uint8 tensor of e2m1 codes" % name)
    if t.shape != (rows, _pad32(K) >> 1):
        raise ValueError("%s must be [%d, %d]" % (name, rows, _pad32(K) >> 1))
    return _dense(t, name)


def _packed(t, rows, K, name):
    import torch
    need = _scale_bytes(rows, K)
    if t.dtype is not torch.uint8 or t.numel() < need:
        raise ValueError("%s must be a uint8 tensor of at least %d bytes" % (name, need))
    return _dense(t, name)


def _dense(t, name):
    return t.data_ptr() if t.is_cuda and t.is_contiguous() else _hkg._dev_ptr(t, name)


class _Elsewhere:
    """The library with GPU `dev` current for each call."""

    def __init__(self, dev):
        self.dev = dev

    def __getattr__(self, name):
        def call(*args):
            import torch
            with torch.cuda.device(self.dev):
                return getattr(_lib(), name)(*args)
        return call


def _on(t):
    """The library for launches on t's GPU, which has to be current: the handle of a
    device's default stream is 0, and stands for the current device's."""
    lib = _lib()
    if not _several:      # the comparisons are a tenth of a small call's time on the host
        return lib
    import torch
    dev = t.get_device()
    return lib if dev == torch.cuda.current_device() else _Elsewhere(dev)


def _handle(stream, t, *others) -> int:
    """Handle of the stream a call runs on: `stream`, or torch's current one on t's
    device; `others`: the call's other tensors, or None."""
    _lib()
    dev = t.get_device()
    if _several:
        for o in others:
            if o is not None and o.get_device() != dev:
                raise ValueError("all tensors of a call must be on one GPU")
        if stream is not None and stream.device.index != dev:
            raise ValueError("stream must belong to the tensors' GPU")
    return int(stream.cuda_stream) if stream is not None else _raw_stream(dev)


def _empty(shape, dtype, like, stream):
    """A new tensor on like's device that belongs to the stream the call runs on (a
    block freed while that stream still uses it is then reused in its order)."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _bytes(n, like, stream):
    import torch
    return _empty((max(int(n), 16),), torch.uint8, like, stream)


def _output(t, shape, dtype, name, like, stream):
    """t, or a new tensor; -> (tensor, pointer, row pitch)."""
    if t is None:
        t = _empty(shape, dtype, like, stream)
        return t, t.data_ptr(), shape[1]
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError("%s must be a %s tensor of shape %s" % (name, dtype, shape))
    ptr, ld = _hkg._matrix(t, name)
    return t, ptr, ld


def _workspace(t, need, like, stream):
    """(tensor, pointer, size) of the caller's workspace, or of a new one."""
    if need <= 0:
        return None, None, 0
    if t is None:
        t = _bytes(need, like, stream)
    return t, _hkg._dev_ptr(t, "workspace"), t.numel() * t.element_size()


def mxfp4_quantize(x, operand, stream=None):
    """MXFP4 form of x [rows, K] (bf16 or fp32, rows contiguous) along K ->
    (codes [rows, Kp / 2], packed scales for `operand`)."""
    import torch
    xt = _elem_type(x, "x")
    px, ld = _hkg._matrix(x, "x")
    rows, K = x.shape
    st = _handle(stream, x)
    codes = _empty((rows, _pad32(K) >> 1), torch.uint8, x, stream)
    packed = _bytes(_scale_bytes(rows, K), x, stream)
    _check(_on(x).hkg_mxfp4_quantize(operand, rows, K, px, xt, ld, codes.data_ptr(), packed.data_ptr(),
                                     st), "hkg_mxfp4_quantize")
    return codes, packed


def mxfp4_quantize_both(x, operand, operand_t, stream=None):
    """mxfp4_quantize(x) and, from the same pass over x, the MXFP4 form of x^T
    -> (codes, packed, codes_t [K, Rp / 2], packed_t)."""
    import torch
    xt = _elem_type(x, "x")
    px, ld = _hkg._matrix(x, "x")
    rows, K = x.shape
    st = _handle(stream, x)
    codes = _empty((rows, _pad32(K) >> 1), torch.uint8, x, stream)
    codes_t = _empty((K, _pad32(rows) >> 1), torch.uint8, x, stream)
    packed = _bytes(_scale_bytes(rows, K), x, stream)
    packed_t = _bytes(_scale_bytes(K, rows), x, stream)
    _check(_on(x).hkg_mxfp4_quantize_both(operand, operand_t, rows, K, px, xt, ld, codes.data_ptr(),
                                          packed.data_ptr(), codes_t.data_ptr(), packed_t.data_ptr(),
                                          st), "hkg_mxfp4_quantize_both")
    return codes, packed, codes_t, packed_t


def mxfp4_dequantize(codes, packed, operand, out=None, dtype=None, stream=None):
    """The values of an MXFP4 matrix, [rows, Kp] in bf16 (default) or fp32."""
    import torch
    if codes.dim() != 2:
        raise TypeError("codes must be a 2-D uint8 tensor of e2m1 codes")
    rows, K = codes.shape[0], 2 * codes.shape[1]
    if K % 32:
        raise ValueError("codes must hold whole blocks of 32 (16 bytes a row)")
    pc, pp = _codes(codes, rows, K, "codes"), _packed(packed, rows, K, "packed")
    st = _handle(stream, codes, packed, out)
    dtype = dtype if dtype is not None else out.dtype if out is not None else torch.bfloat16
    out, po, ld = _output(out, (rows, K), dtype, "out", codes, stream)
    _check(_on(codes).hkg_mxfp4_dequantize(operand, rows, K, pc, pp, po, _elem_type(out, "out"), ld,
                                            st), "hkg_mxfp4_dequantize")
    return out


def gemm_mxfp4(A, B, SA_packed, SB_packed, C=None, C_f32=None, stream=None):
    """C[M,N] (bf16) = A[M,K] · B[N,K]ᵀ of two MXFP4 matrices; returns C."""
    import torch
    if A.dim() != 2 or B.dim() != 2 or A.shape[1] != B.shape[1]:
        raise ValueError("A is [M,K/2] and B is [N,K/2]")
    M, N, K = A.shape[0], B.shape[0], 2 * A.shape[1]
    if K % 32:
        raise ValueError("A and B must hold whole blocks of 32 (16 bytes a row)")
    pa, pb = _codes(A, M, K, "A"), _codes(B, N, K, "B")
    sa, sb = _packed(SA_packed, M, K, "SA_packed"), _packed(SB_packed, N, K, "SB_packed")
    st = _handle(stream, A, B, SA_packed, SB_packed, C, C_f32)
    C, pc, ldc = _output(C, (M, N), torch.bfloat16, "C", A, stream)
    pf = None
    if C_f32 is not None:
        C_f32, pf, ldf = _output(C_f32, (M, N), torch.float32, "C_f32", A, stream)
        if ldf != ldc:
            raise ValueError("C and C_f32 must have the same row pitch")
    _check(_on(A).hkg_gemm_mxfp4(M, N, K, pa, pb, sa, sb, pc, pf, ldc, st), "hkg_gemm_mxfp4")
    return C


def linear_mxfp4(x, W, SW_packed, y=None, workspace=None, stream=None):
    """y[M,N] (bf16) = Q(x)[M,K] · W[N,K]ᵀ with x quantised to MXFP4 on the way
    (x bf16 or fp32; W, SW_packed an MXFP4 matrix packed for operand B).
    workspace: a uint8 tensor of hkg_linear_mxfp4_workspace_bytes(M, N, K)."""
    import torch
    xt = _elem_type(x, "x")
    px, ldx = _hkg._matrix(x, "x")
    M, K = x.shape
    N = W.shape[0]
    pw, ps = _codes(W, N, K, "W"), _packed(SW_packed, N, K, "SW_packed")
    st = _handle(stream, x, W, SW_packed, y, workspace)
    y, py, ldy = _output(y, (M, N), torch.bfloat16, "y", x, stream)
    need = _check(_lib().hkg_linear_mxfp4_workspace_bytes(M, N, K), "hkg_linear_mxfp4_workspace_bytes")
    workspace, pws, nws = _workspace(workspace, need, x, stream)
    _check(_on(x).hkg_linear_mxfp4(M, N, K, px, xt, ldx, pw, ps, py, ldy, pws, nws, st),
           "hkg_linear_mxfp4")
    return y


def linear_mxfp4_backward(dy, Wt, SWt_packed, Xt, SXt_packed, dx=None, dw=None, workspace=None,
                          stream=None):
    """Gradients of y = Q(x) Wᵀ, rounding passed straight through: (dx [M,K], dw
    [N,K]) in bf16 from dy [M,N] (bf16 or fp32) and the MXFP4 forms of Wᵀ [K,N]
    and xᵀ [K,M] packed for operand B (mxfp4_quantize_both)."""
    import torch
    t = _elem_type(dy, "dy")
    pdy, lddy = _hkg._matrix(dy, "dy")
    M, N = dy.shape
    K = Wt.shape[0]
    pw, psw = _codes(Wt, K, N, "Wt"), _packed(SWt_packed, K, N, "SWt_packed")
    px, psx = _codes(Xt, K, M, "Xt"), _packed(SXt_packed, K, M, "SXt_packed")
    st = _handle(stream, dy, Wt, SWt_packed, Xt, SXt_packed, dx, dw, workspace)
    dx, pdx, lddx = _output(dx, (M, K), torch.bfloat16, "dx", dy, stream)
    dw, pdw, lddw = _output(dw, (N, K), torch.bfloat16, "dw", dy, stream)
    need = _check(_lib().hkg_linear_mxfp4_backward_workspace_bytes(M, N, K),
                  "hkg_linear_mxfp4_backward_workspace_bytes")
    workspace, pws, nws = _workspace(workspace, need, dy, stream)
    _check(_on(dy).hkg_linear_mxfp4_backward(M, N, K, pdy, t, lddy, pw, psw, px, psx, pdx, lddx, pdw,
                                             lddw, pws, nws, st), "hkg_linear_mxfp4_backward")
    return dx, dw


MUON_COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def orthogonalize(G, steps=5, coefficients=MUON_COEFFICIENTS, eps=1e-7, out=None, workspace=None,
                  stream=None):
    """The orthogonalised direction of an update G [rows, cols] (bf16 or fp32): X =
    G / (|G| + eps), then `steps` times X <- a X + (b A + c A A) X with A = X Xᵀ
    (on Gᵀ where G is tall); bf16, in `out` (which may be G).  workspace: a uint8
    tensor of hkg_orthogonalize_workspace_bytes(rows, cols)."""
    import torch
    t = _elem_type(G, "G")
    pg, ldg = _hkg._matrix(G, "G")
    rows, cols = G.shape
    a, b, c = coefficients
    st = _handle(stream, G, out, workspace)
    out, po, ldo = _output(out, (rows, cols), torch.bfloat16, "out", G, stream)
    need = _check(_lib().hkg_orthogonalize_workspace_bytes(rows, cols), "hkg_orthogonalize_workspace_bytes")
    workspace, pws, nws = _workspace(workspace, need, G, stream)
    _check(_on(G).hkg_orthogonalize(rows, cols, pg, t, ldg, steps, a, b, c, eps, po, ldo, pws, nws, st),
           "hkg_orthogonalize")
    return out
