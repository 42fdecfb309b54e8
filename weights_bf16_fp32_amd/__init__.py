"""Python binding of the gfx950 spectral library (libspec.so, C ABI in include/spec.h).

Argument marshalling only: every step of the path runs in the library's HIP
kernels.  PyTorch provides device memory and the current stream.  The library
is loaded on first use and a missing library raises immediately; there is no
fallback of any kind.

    import weights_bf16_fp32_amd as spec
    spec.cov_accumulate(X, C, alpha=1/n, beta=0.0)          # C <- beta C + alpha X^T X (lower)
    band = spec.gram_window(H, N=30)                          # [S, T, N] <h_t, h_{t-j}>
    w, info = spec.eigvalsh_batched_band(band, n=30, scale=1/30)
    w = spec.eigvalsh_large(C)                                # destroys C
    rec = spec.descriptors(w, n_samples=n, p_dim=d, k=1)      # structured numpy array
    sm = spec.desc_smooth(raw_records, streams=S, W=W, alpha=0.3)  # smoothed descriptor series
    rb = spec.spectrum_robust(w, n_samples=n, p_dim=d)        # median/MAD/winsor/log/KL statistics
    X = spec.embed(E, ids, scale=d ** 0.5)                    # scale * E[ids]
    loss, lse = spec.linear_xent(H, W, target)                # cross entropy of the rows of H W^T
    dH, dW = spec.linear_xent_grad(H, W, target, lse, dloss)  # its gradients
    spec.embed_grad(dX, ids, V, scale=d ** 0.5, beta=1.0, dE=dW)  # into a tied table's gradient
    O = spec.orthogonalize(G)                                 # Newton-Schulz: G with its singular values near one
    h, x, r_post, r_pre = spec.block_norm(h, y, w_post=a, gate=g, w_pre=b)  # h + g norm(y) a, and its norm times b
    q = spec.mx_quantize(x, spec.MX_INT8)                     # x in 8 bits for the backward pass
    dW = spec.mx_weight_grad(dz, q)                           # dz^T x
    y = spec.mx_linear(x, spec.mx_quantize(W, spec.MX_FP4))   # x W^T from W in 4 bits
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Any, NamedTuple

import numpy as np

__all__ = [
    "SpecError", "lib", "cov_accumulate", "gram_window", "eigvalsh_batched_dense",
    "eigvalsh_batched_band", "eigvalsh_large", "eigvalsh_large_workspace", "descriptors",
    "descriptors_workspace", "DESC_DTYPE", "desc_smooth", "spectrum_robust", "ROBUST_DTYPE", "eigvalsh_topk",
    "eigvecs_topk", "project_weight", "project_weight_workspace",
    "embed", "embed_grad", "embed_grad_workspace", "linear_xent", "linear_xent_workspace", "linear_xent_grad",
    "linear_xent_grad_workspace", "orthogonalize", "orthogonalize_workspace", "NS_COEFFS",
    "Mx", "MX_INT8", "MX_FP4", "mx_empty", "mx_quantize", "mx_dequantize", "mx_linear", "mx_linear_workspace",
    "MX_OP_LINEAR", "MX_OP_PRODUCT", "MX_OP_WEIGHT_GRAD", "mx_plan",
    "mx_product", "mx_product_workspace", "mx_weight_grad", "mx_weight_grad_workspace", "block_norm", "block_norm_grad",
    "block_norm_grad_workspace",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspec.so")

BF16, F32, F64, I32, I64 = 0, 1, 2, 3, 4
MX_INT8, MX_FP4 = 0, 1
MX_OP_LINEAR, MX_OP_PRODUCT, MX_OP_WEIGHT_GRAD = 0, 1, 2
GRAM_BAND, GRAM_DENSE = 0, 1
SRC_DENSE, SRC_BAND = 0, 1
MODE_EIG, MODE_SINGULAR = 0, 1
SIGMA2_GIVEN, SIGMA2_MEDIAN, SIGMA2_MEAN, SIGMA2_WINSOR = 0, 1, 2, 3
FLAG_NONFINITE, FLAG_GK_UNDEF, FLAG_S_ZERO, FLAG_HELD = 1, 2, 4, 8

_DESC_FIELDS_F = ["S", "H", "erank", "m1", "gk", "g1", "sigma2", "lambda_plus", "mp_w1",
                  "top_energy", "top_sigma_share", "tail_head", "tail_min", "sigma1"]
_DESC_FIELDS_I = ["n_above", "n_small", "r_pos", "flags"]
DESC_DTYPE = np.dtype([(f, "<f8") for f in _DESC_FIELDS_F] + [(f, "<i8") for f in _DESC_FIELDS_I])
assert DESC_DTYPE.itemsize == 144
_ROBUST_FIELDS_F = ["median", "sigma2_winsor", "mad", "log_mean", "log_std", "sigma2", "kl_mp"]
ROBUST_DTYPE = np.dtype([(f, "<f8") for f in _ROBUST_FIELDS_F] + [("n_mad", "<i8"), ("flags", "<i8")])
assert ROBUST_DTYPE.itemsize == 72


KT = {"syrk": 0, "gram": 1, "small_eig": 2, "desc": 3, "symm": 4, "syr2k": 5, "panel": 6, "bulge": 7,
      "tridiag": 8}


def timing_enable(kernels) -> None:
    """Start timing every launch of the named kernels (keys of KT) with HIP
    events on their own stream; an empty list stops."""
    m = 0
    for k in kernels:
        m |= 1 << KT[k]
    _check(lib().spec_timing_enable(m))


def timing_read(kernel: str):
    """(total device ms, timed launches) of one kernel since timing_enable."""
    ms, n = ctypes.c_double(0.0), ctypes.c_int64(0)
    _check(lib().spec_timing_read(KT[kernel], ctypes.byref(ms), ctypes.byref(n)))
    return ms.value, n.value


class SpecError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"spec status {status}: {msg}")
        self.status = status


class BatchSrc(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("a", ctypes.c_void_p), ("lda", ctypes.c_int64),
                ("stride_a", ctypes.c_int64), ("streams", ctypes.c_int64), ("T", ctypes.c_int64),
                ("stride", ctypes.c_int), ("scale", ctypes.c_float)]


class DescParams(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int), ("sigma2_mode", ctypes.c_int), ("sigma2", ctypes.c_double),
                ("n_samples", ctypes.c_int64), ("p_dim", ctypes.c_int64), ("k", ctypes.c_int64),
                ("top_frac", ctypes.c_double), ("small_rel", ctypes.c_double),
                ("tail_frac", ctypes.c_double)]


class RobustParams(ctypes.Structure):
    _fields_ = [("sigma2_mode", ctypes.c_int32), ("bins", ctypes.c_int32), ("sigma2", ctypes.c_double),
                ("n_samples", ctypes.c_int64), ("p_dim", ctypes.c_int64), ("winsor_frac", ctypes.c_double),
                ("mad_k", ctypes.c_double)]


class MxMatrix(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("s", ctypes.c_void_p), ("ldq", ctypes.c_int64), ("lds", ctypes.c_int64),
                ("fmt", ctypes.c_int32)]


class Block(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("d", ctypes.c_int64), ("t", ctypes.c_int32), ("post", ctypes.c_int32),
                ("alpha", ctypes.c_double), ("beta", ctypes.c_double), ("eps", ctypes.c_double),
                ("w_post", ctypes.c_void_p), ("w_pre", ctypes.c_void_p), ("gate", ctypes.c_void_p),
                ("ldg", ctypes.c_int64), ("gate_rows", ctypes.c_int64)]


EXPORTS = ["spec_strerror", "spec_version", "spec_cov_accumulate", "spec_gram_window",
           "spec_eigvalsh_batched", "spec_eigvalsh_large_workspace", "spec_eigvalsh_large",
           "spec_descriptors_workspace", "spec_descriptors", "spec_desc_smooth", "spec_spectrum_robust",
           "spec_eigvalsh_topk", "spec_eigvecs_topk", "spec_project_weight_workspace",
           "spec_project_weight", "spec_timing_enable", "spec_timing_read", "spec_descriptors_static", "spec_tail_pair_screen", "spec_eigvalsh_batched_desc",
           "spec_eigvalsh_sliding", "spec_eigh_large_workspace", "spec_eigh_large", "spec_eigh_batched",
           "spec_embed", "spec_embed_grad_workspace", "spec_embed_grad", "spec_linear_xent_workspace",
           "spec_linear_xent", "spec_linear_xent_grad_workspace", "spec_linear_xent_grad",
           "spec_orthogonalize_workspace", "spec_orthogonalize",
           "spec_mx_row_bytes", "spec_mx_quantize", "spec_mx_dequantize", "spec_mx_plan", "spec_mx_linear_workspace",
           "spec_mx_linear",
           "spec_mx_product_workspace", "spec_mx_product", "spec_mx_weight_grad_workspace", "spec_mx_weight_grad",
           "spec_block_norm", "spec_block_norm_grad_workspace", "spec_block_norm_grad"]

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libspec.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                              "(weights_bf16_fp32_amd/build.py); there is no fallback path")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, i32, dbl = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_double
        L.spec_strerror.argtypes = [i32]
        L.spec_strerror.restype = ctypes.c_char_p
        L.spec_version.argtypes = []
        L.spec_version.restype = ctypes.c_char_p
        L.spec_cov_accumulate.argtypes = [vp, vp, i32, i64, i64, i64, vp, i32, i64, dbl, dbl]
        L.spec_gram_window.argtypes = [vp, vp, i32, i64, i64, i64, i64, i64, i32, i32, dbl, i32, vp]
        L.spec_eigvalsh_batched.argtypes = [vp, ctypes.POINTER(BatchSrc), i64, i32, vp, vp]
        L.spec_eigvalsh_large_workspace.argtypes = [i64, i32, ctypes.POINTER(ctypes.c_size_t)]
        L.spec_eigvalsh_large.argtypes = [vp, vp, i32, i64, i64, vp, vp, ctypes.c_size_t, vp]
        L.spec_eigh_large_workspace.argtypes = [i64, i32, i64, ctypes.POINTER(ctypes.c_size_t)]
        L.spec_eigh_large.argtypes = [vp, vp, i32, i64, i64, vp, vp, i64, i64, vp, ctypes.c_size_t, vp]
        L.spec_descriptors_workspace.argtypes = [i64, ctypes.POINTER(ctypes.c_size_t)]
        L.spec_descriptors.argtypes = [vp, vp, i32, i64, i64, i64, ctypes.POINTER(DescParams), vp, vp,
                                       ctypes.c_size_t]
        L.spec_desc_smooth.argtypes = [vp, vp, i64, i64, dbl, vp]
        L.spec_eigvalsh_topk.argtypes = [vp, vp, i32, i64, i64, vp, i32, vp, vp, ctypes.c_size_t]
        L.spec_eigvecs_topk.argtypes = [vp, vp, i32, i64, i64, vp, i32, vp, vp, i64, vp, ctypes.c_size_t, vp]
        L.spec_project_weight_workspace.argtypes = [i64, ctypes.POINTER(ctypes.c_size_t)]
        L.spec_project_weight.argtypes = [vp, vp, i32, i64, i64, vp, i64, i32, vp, i64, vp, i64, vp,
                                          ctypes.c_size_t]
        L.spec_spectrum_robust.argtypes = [vp, vp, i32, i64, i64, i64, ctypes.POINTER(RobustParams), vp]
        L.spec_eigvalsh_batched_desc.argtypes = [vp, ctypes.POINTER(BatchSrc), i64, i32, vp, vp,
                                                  ctypes.POINTER(DescParams), vp, vp, ctypes.c_size_t]
        L.spec_tail_pair_screen.argtypes = [vp, vp, vp, i32, i64, i64, i64, i64, i64, i64, dbl, vp, i64, vp, i64,
                                             vp]
        L.spec_descriptors_static.argtypes = [vp, vp, i32, i64, i64, i64, ctypes.POINTER(DescParams), vp]
        L.spec_eigvalsh_sliding.argtypes = [vp, ctypes.POINTER(BatchSrc), i64, i32, i32, vp, vp]
        L.spec_eigh_batched.argtypes = [vp, ctypes.POINTER(BatchSrc), i64, i32, vp, vp, vp]
        sz, szp = ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t)
        L.spec_embed.argtypes = [vp, vp, i32, i64, i64, i64, vp, i32, i64, dbl, vp, i64]
        L.spec_embed_grad_workspace.argtypes = [i64, i64, i64, szp]
        L.spec_embed_grad.argtypes = [vp, vp, i32, i64, i64, i64, i64, vp, i32, dbl, dbl, vp, i32, i64, vp, sz]
        L.spec_linear_xent_workspace.argtypes = [i64, i64, i64, i32, szp]
        L.spec_linear_xent.argtypes = [vp, vp, vp, i32, i64, i64, i64, i64, i64, vp, i32, dbl, vp, vp, vp, sz]
        L.spec_linear_xent_grad_workspace.argtypes = [i64, i64, i64, i32, szp]
        L.spec_linear_xent_grad.argtypes = [vp, vp, vp, i32, i64, i64, i64, i64, i64, vp, i32, dbl, vp, vp, dbl, vp,
                                            i64, vp, i64, vp, sz]
        L.spec_orthogonalize_workspace.argtypes = [i64, i64, i64, i32, szp]
        L.spec_orthogonalize.argtypes = [vp, vp, i32, i64, i64, i64, i64, i64, ctypes.POINTER(dbl), i32, dbl, dbl,
                                         vp, i64, i64, vp, sz]
        mxp, blp, i64p = ctypes.POINTER(MxMatrix), ctypes.POINTER(Block), ctypes.POINTER(i64)
        L.spec_mx_row_bytes.argtypes = [i32, i64, i64p, i64p]
        L.spec_mx_quantize.argtypes = [vp, vp, i32, i64, i64, i64, mxp]
        L.spec_mx_dequantize.argtypes = [vp, mxp, i64, i64, vp, i32, i64]
        L.spec_mx_plan.argtypes = [i32, i64, i64, i64, i32, ctypes.POINTER(i32), ctypes.POINTER(i32)]
        L.spec_mx_linear_workspace.argtypes = [i64, i64, i64, i32, szp]
        L.spec_mx_linear.argtypes = [vp, vp, i32, i64, i64, i64, i64, mxp, vp, i64, vp, sz]
        L.spec_mx_product_workspace.argtypes = [i64, i64, i64, szp]
        L.spec_mx_product.argtypes = [vp, mxp, mxp, i64, i64, i64, vp, i32, i64, vp, sz]
        L.spec_mx_weight_grad_workspace.argtypes = [i64, i64, i64, i32, szp]
        L.spec_mx_weight_grad.argtypes = [vp, vp, i32, i64, i64, i64, i64, mxp, dbl, vp, i64, vp, sz]
        L.spec_block_norm.argtypes = [vp, blp, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, mxp, mxp, mxp]
        L.spec_block_norm_grad_workspace.argtypes = [blp, szp]
        L.spec_block_norm_grad.argtypes = [vp, blp, vp, i64, mxp, vp, i64, mxp, vp, vp, vp, i64, vp, i64, vp, i64, vp,
                                           i64, vp, vp, vp, vp, sz]
        L.spec_timing_enable.argtypes = [ctypes.c_uint]
        L.spec_timing_read.argtypes = [i32, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64)]
        for f in EXPORTS[2:]:
            getattr(L, f).restype = i32
        _lib = L
    return _lib


def _check(status: int):
    if status != 0:
        raise SpecError(status, lib().spec_strerror(status).decode())


def _torch():
    import torch
    return torch


def _stream():
    """The current stream of the current device, as a handle (torch's stream object
    costs 3 us to make, as much as a launch)."""
    torch = _torch()
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _dt(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.float64:
        return F64
    raise SpecError(-2, f"unsupported dtype {t.dtype}")


def _dev(t):
    if not t.is_cuda:
        raise SpecError(-1, "tensor must be on the GPU")
    return t.data_ptr()


def cov_accumulate(X, C, alpha: float = 1.0, beta: float = 0.0):
    """C <- beta C + alpha X^T X on the lower triangle of C (X: [n, d], C: [d, d])."""
    n, d = X.shape
    if X.stride(1) != 1 or C.stride(1) != 1:
        raise SpecError(-1, "inner dimension must be contiguous")
    _check(lib().spec_cov_accumulate(_stream(), _dev(X), _dt(X), n, d, X.stride(0), _dev(C), _dt(C),
                                     C.stride(0), float(alpha), float(beta)))
    return C


def gram_window(H, N: int, stride: int = 1, scale: float = 1.0, layout: int = GRAM_BAND, out=None):
    """Band <h_t, h_{t-j}> [S, T, N] (layout BAND) or dense scale*H_w H_w^T [S*W, N, N]."""
    torch = _torch()
    if H.dim() == 2:
        H = H.unsqueeze(0)
    S, T, d = H.shape
    if H.stride(2) != 1:
        raise SpecError(-1, "feature dimension must be contiguous")
    if out is None:
        if layout == GRAM_BAND:
            out = torch.empty((S, T, N), dtype=torch.float32, device=H.device)
        else:
            W = (T - N) // stride + 1
            out = torch.empty((S * W, N, N), dtype=torch.float32, device=H.device)
    _check(lib().spec_gram_window(_stream(), _dev(H), _dt(H), S, T, d, H.stride(1), H.stride(0), N, stride,
                                  float(scale), layout, _dev(out)))
    return out


def _batched(src: BatchSrc, batch: int, n: int, w, info, device):
    torch = _torch()
    if w is None:
        w = torch.empty((batch, n), dtype=torch.float32, device=device)
    if info is None:
        info = torch.empty((batch,), dtype=torch.int32, device=device)
    _check(lib().spec_eigvalsh_batched(_stream(), ctypes.byref(src), batch, n, _dev(w), _dev(info)))
    return w, info


def eigvalsh_batched_dense(A, w=None, info=None):
    """Eigenvalues (descending) of A [batch, n, n] f32 (lower triangle read).
    info[b] = bisection rounds, or -1 for a matrix with a non-finite entry."""
    if A.dim() == 2:
        A = A.unsqueeze(0)
    batch, n, _ = A.shape
    src = BatchSrc(SRC_DENSE, _dev(A), A.stride(1), A.stride(0), 0, 0, 1, 1.0)
    return _batched(src, batch, n, w, info, A.device)


def eigvalsh_batched_band(band, n: int, scale: float, stride: int = 1, w=None, info=None):
    """Eigenvalues of every window's Gram scale * G_w from the band [S, T, n] of gram_window."""
    S, T, N = band.shape
    if N != n or not band.is_contiguous():
        raise SpecError(-1, "band must be a contiguous [streams, T, n] tensor")
    batch = S * ((T - n) // stride + 1)
    src = BatchSrc(SRC_BAND, _dev(band), 0, 0, S, T, stride, float(scale))
    return _batched(src, batch, n, w, info, band.device)


def _eigh_batched(src, batch, n, w, V, info, device):
    torch = _torch()
    if w is None:
        w = torch.empty((batch, n), dtype=torch.float32, device=device)
    if V is None:
        V = torch.empty((batch, n, n), dtype=torch.float32, device=device)
    if info is None:
        info = torch.empty((batch,), dtype=torch.int32, device=device)
    _check(lib().spec_eigh_batched(_stream(), ctypes.byref(src), batch, n, _dev(w), _dev(V), _dev(info)))
    return w, V, info


def eigh_batched_dense(A, w=None, V=None, info=None):
    """Eigenvalues (descending) and eigenvectors of A [batch, n, n] f32 (lower
    triangle read, n <= 32): V[b][:, j] belongs to w[b][j].  info[b] = Jacobi
    sweeps, -2 (sweep limit) or -1 (non-finite entry)."""
    if A.dim() == 2:
        A = A.unsqueeze(0)
    batch, n, _ = A.shape
    src = BatchSrc(SRC_DENSE, _dev(A), A.stride(1), A.stride(0), 0, 0, 1, 1.0)
    return _eigh_batched(src, batch, n, w, V, info, A.device)


def eigh_batched_band(band, n: int, scale: float, stride: int = 1, w=None, V=None, info=None):
    """Eigenpairs of every window's Gram scale * G_w from the band [S, T, n] of gram_window."""
    S, T, N = band.shape
    if N != n or not band.is_contiguous():
        raise SpecError(-1, "band must be a contiguous [streams, T, n] tensor")
    batch = S * ((T - n) // stride + 1)
    src = BatchSrc(SRC_BAND, _dev(band), 0, 0, S, T, stride, float(scale))
    return _eigh_batched(src, batch, n, w, V, info, band.device)


def eigvalsh_sliding(band, n: int, scale: float, stride: int = 1, restart: int = 64, w=None, info=None):
    """The spectra of eigvalsh_batched_band by rank-one down/up-dates along each
    stream (fp64, a fresh start every `restart` windows).  info[b] = largest
    secular iteration count of the window's updates, or -1 (non-finite step)."""
    torch = _torch()
    S, T, N = band.shape
    if N != n or not band.is_contiguous():
        raise SpecError(-1, "band must be a contiguous [streams, T, n] tensor")
    batch = S * ((T - n) // stride + 1)
    src = BatchSrc(SRC_BAND, _dev(band), 0, 0, S, T, stride, float(scale))
    if w is None:
        w = torch.empty((batch, n), dtype=torch.float32, device=band.device)
    if info is None:
        info = torch.empty((batch,), dtype=torch.int32, device=band.device)
    _check(lib().spec_eigvalsh_sliding(_stream(), ctypes.byref(src), batch, n, int(restart), _dev(w), _dev(info)))
    return w, info


def eigh_large_workspace(n: int, dtype, k: int) -> int:
    torch = _torch()
    t = F32 if dtype == torch.float32 else F64
    b = ctypes.c_size_t(0)
    _check(lib().spec_eigh_large_workspace(n, t, k, ctypes.byref(b)))
    return b.value


def eigh_large(A, k: int, w=None, Z=None, ws=None, info=None):
    """All eigenvalues (descending) of the symmetric A [n, n] (lower triangle
    read, A destroyed) and the eigenvectors of the k largest, Z [n, k] (column j
    for w[j])."""
    torch = _torch()
    n = A.shape[0]
    if A.stride(1) != 1:
        raise SpecError(-1, "A must be row-major")
    if w is None:
        w = torch.empty((n,), dtype=A.dtype, device=A.device)
    if Z is None:
        Z = torch.empty((n, k), dtype=A.dtype, device=A.device)
    if ws is None:
        ws = torch.empty((eigh_large_workspace(n, A.dtype, k),), dtype=torch.uint8, device=A.device)
    ip = _dev(info) if info is not None else None
    _check(lib().spec_eigh_large(_stream(), _dev(A), _dt(A), n, A.stride(0), _dev(w), _dev(Z), Z.stride(0), k,
                                 _dev(ws), ws.numel(), ip))
    return w, Z


def eigvalsh_large_workspace(n: int, dtype) -> int:
    torch = _torch()
    t = F32 if dtype == torch.float32 else F64
    b = ctypes.c_size_t(0)
    _check(lib().spec_eigvalsh_large_workspace(n, t, ctypes.byref(b)))
    return b.value


def eigvalsh_large(A, w=None, ws=None, info=None):
    """Eigenvalues (descending) of the symmetric A [n, n] (lower triangle read, A destroyed)."""
    torch = _torch()
    n = A.shape[0]
    if A.stride(1) != 1:
        raise SpecError(-1, "A must be row-major")
    if w is None:
        w = torch.empty((n,), dtype=A.dtype, device=A.device)
    if ws is None:
        ws = torch.empty((eigvalsh_large_workspace(n, A.dtype),), dtype=torch.uint8, device=A.device)
    ip = _dev(info) if info is not None else None
    _check(lib().spec_eigvalsh_large(_stream(), _dev(A), _dt(A), n, A.stride(0), _dev(w), _dev(ws),
                                     ws.numel(), ip))
    return w


def descriptors_workspace(r: int) -> int:
    b = ctypes.c_size_t(0)
    _check(lib().spec_descriptors_workspace(r, ctypes.byref(b)))
    return b.value


def descriptors(w, *, n_samples: int, p_dim: int, k: int = 1, mode: int = MODE_EIG,
                sigma2: float = 1.0, sigma2_mode: int = SIGMA2_GIVEN, top_frac: float = 0.2,
                small_rel: float = 1e-2, tail_frac: float = 0.7, out=None, ws=None, to_host: bool = True):
    """Descriptors of each row of w [batch, r] (sorted descending).  Returns a numpy
    structured array of DESC_DTYPE (or the raw device buffer if to_host is False)."""
    torch = _torch()
    if w.dim() == 1:
        w = w.unsqueeze(0)
    batch, r = w.shape
    if out is None:
        out = torch.empty((batch, DESC_DTYPE.itemsize), dtype=torch.uint8, device=w.device)
    if ws is None:
        ws = torch.empty((descriptors_workspace(r),), dtype=torch.uint8, device=w.device)
    p = DescParams(mode, sigma2_mode, float(sigma2), int(n_samples), int(p_dim), int(k), float(top_frac),
                   float(small_rel), float(tail_frac))
    _check(lib().spec_descriptors(_stream(), _dev(w), _dt(w), batch, r, w.stride(0), ctypes.byref(p),
                                  _dev(out), _dev(ws), ws.numel()))
    if not to_host:
        return out
    return out.cpu().numpy().view(DESC_DTYPE).reshape(batch)


def descriptors_static(w, *, n_samples: int, p_dim: int, k: int = 1, mode: int = MODE_EIG,
                       sigma2: float = 1.0, sigma2_mode: int = SIGMA2_GIVEN, top_frac: float = 0.2,
                       small_rel: float = 1e-2, tail_frac: float = 0.7, out=None, to_host: bool = True):
    """descriptors() without a workspace: the library's own per-GPU table is used
    (spec_descriptors_static; r <= 32768; overlapping calls on one GPU race)."""
    torch = _torch()
    if w.dim() == 1:
        w = w.unsqueeze(0)
    batch, r = w.shape
    if out is None:
        out = torch.empty((batch, DESC_DTYPE.itemsize), dtype=torch.uint8, device=w.device)
    p = DescParams(mode, sigma2_mode, float(sigma2), int(n_samples), int(p_dim), int(k), float(top_frac),
                   float(small_rel), float(tail_frac))
    _check(lib().spec_descriptors_static(_stream(), _dev(w), _dt(w), batch, r, w.stride(0), ctypes.byref(p),
                                         _dev(out)))
    if not to_host:
        return out
    return out.cpu().numpy().view(DESC_DTYPE).reshape(batch)


def desc_smooth(rec, *, streams: int, W: int, alpha: float, out=None, to_host: bool = True):
    """Exponential smoothing along W of the descriptor records rec (a device uint8
    buffer of streams * W records, as descriptors(..., to_host=False) returns).
    Returns a numpy structured array [streams, W] of DESC_DTYPE (or the device
    buffer if to_host is False)."""
    torch = _torch()
    if out is None:
        out = torch.empty((streams * W, DESC_DTYPE.itemsize), dtype=torch.uint8, device=rec.device)
    _check(lib().spec_desc_smooth(_stream(), _dev(rec), streams, W, float(alpha), _dev(out)))
    if not to_host:
        return out
    return out.cpu().numpy().view(DESC_DTYPE).reshape(streams, W)


def spectrum_robust(w, *, n_samples: int, p_dim: int, sigma2: float = 1.0, sigma2_mode: int = SIGMA2_GIVEN,
                    winsor_frac: float = 0.05, mad_k: float = 3.0, bins: int = 16, out=None,
                    to_host: bool = True):
    """Median, winsorised sigma^2, MAD and MAD outlier count, log-eigenvalue mean
    and spread, and the KL form of the MP deviation of each row of w [batch, r]
    (sorted descending).  Returns a numpy structured array of ROBUST_DTYPE (or
    the device buffer if to_host is False)."""
    torch = _torch()
    if w.dim() == 1:
        w = w.unsqueeze(0)
    batch, r = w.shape
    if out is None:
        out = torch.empty((batch, ROBUST_DTYPE.itemsize), dtype=torch.uint8, device=w.device)
    p = RobustParams(int(sigma2_mode), int(bins), float(sigma2), int(n_samples), int(p_dim), float(winsor_frac),
                     float(mad_k))
    _check(lib().spec_spectrum_robust(_stream(), _dev(w), _dt(w), batch, r, w.stride(0), ctypes.byref(p),
                                      _dev(out)))
    if not to_host:
        return out
    return out.cpu().numpy().view(ROBUST_DTYPE).reshape(batch)


def eigvalsh_topk(A, Omega, q: int = 2, w=None, ws=None):
    """The 32 Ritz values (descending) of the symmetric A [n, n] (lower triangle
    read, A kept) on the range of A Omega after q subspace iterations; Omega is
    the caller's random test matrix [n, 32] (float32, contiguous)."""
    torch = _torch()
    n = A.shape[0]
    if A.stride(1) != 1 or not Omega.is_contiguous() or tuple(Omega.shape) != (n, 32):
        raise SpecError(-1, "A must be row-major and Omega a contiguous [n, 32] tensor")
    if w is None:
        w = torch.empty((32,), dtype=torch.float32, device=A.device)
    if ws is None:
        ws = torch.empty((eigvalsh_large_workspace(n, torch.float32),), dtype=torch.uint8, device=A.device)
    _check(lib().spec_eigvalsh_topk(_stream(), _dev(A), _dt(A), n, A.stride(0), _dev(Omega), int(q), _dev(w),
                                    _dev(ws), ws.numel()))
    return w


def eigvecs_topk(A, Omega, q: int = 2, w=None, P=None, ws=None, info=None):
    """Ritz values (descending, [32]) and Ritz vectors P [n, 32] (column i for
    value i, orthonormal columns, arbitrary signs) of the same projection as
    eigvalsh_topk; the columns with a value above the MP edge span the signal
    subspace.  ``info`` (int32 [1] device tensor, optional) receives 0
    (converged), 1 (non-finite input) or 2 (sweep limit reached)."""
    torch = _torch()
    n = A.shape[0]
    if A.stride(1) != 1 or not Omega.is_contiguous() or tuple(Omega.shape) != (n, 32):
        raise SpecError(-1, "A must be row-major and Omega a contiguous [n, 32] tensor")
    if w is None:
        w = torch.empty((32,), dtype=torch.float32, device=A.device)
    if P is None:
        P = torch.empty((n, 32), dtype=torch.float32, device=A.device)
    if P.dim() != 2 or P.shape[0] != n or P.shape[1] < 32 or P.stride(1) != 1 or P.dtype != torch.float32:
        raise SpecError(-1, "P must be a row-major float32 [n, >= 32] tensor")
    if ws is None:
        ws = torch.empty((eigvalsh_large_workspace(n, torch.float32),), dtype=torch.uint8, device=A.device)
    _check(lib().spec_eigvecs_topk(_stream(), _dev(A), _dt(A), n, A.stride(0), _dev(Omega), int(q), _dev(w),
                                   _dev(P), P.stride(0), _dev(ws), ws.numel(), _dev(info) if info is not None else None))
    return w, P


def project_weight_workspace(d: int) -> int:
    b = ctypes.c_size_t(0)
    _check(lib().spec_project_weight_workspace(d, ctypes.byref(b)))
    return b.value


def project_weight(W, P, k=None, Wp=None, X=None, want_factor: bool = True, ws=None):
    """W' = P^T W P ([k, k]) and, if want_factor, X = W P ([d, k]) for a square
    weight W [d, d] (bf16 or float32, row-major) and the basis P [d, >= k]
    (float32, row-major; the first k columns are used)."""
    torch = _torch()
    d = W.shape[0]
    if W.dim() != 2 or W.shape[1] != d or W.stride(1) != 1:
        raise SpecError(-1, "W must be a row-major square tensor")
    if P.dim() != 2 or P.shape[0] != d or P.stride(1) != 1 or P.dtype != torch.float32:
        raise SpecError(-1, "P must be a row-major float32 [d, k] tensor")
    k = P.shape[1] if k is None else int(k)
    if k > P.shape[1]:
        raise SpecError(-1, "k exceeds the columns of P")
    if Wp is None:
        Wp = torch.empty((k, k), dtype=torch.float32, device=W.device)
    if want_factor and X is None:
        X = torch.empty((d, k), dtype=torch.float32, device=W.device)
    if not want_factor:
        X = None
    if ws is None:
        ws = torch.empty((project_weight_workspace(d),), dtype=torch.uint8, device=W.device)
    _check(lib().spec_project_weight(_stream(), _dev(W), _dt(W), d, W.stride(0), _dev(P), P.stride(0), k, _dev(Wp),
                                     Wp.stride(0), None if X is None else _dev(X), 0 if X is None else X.stride(0),
                                     _dev(ws), ws.numel()))
    return Wp, X


def tail_pair_screen(U, V, *, i0: int | None = None, t: int | None = None, head_dim: int = 128,
                     eps: float = 0.015, absdot=None, keep=None, count=None):
    """S3 swap-candidate screen: |u_i^T v_j| for the tail columns [i0, i0 + t) of
    U and V (singular vectors as columns; default tail: i >= 0.9 N), and the
    same-head pairs below eps.  Returns (absdot [t, t] f64, keep [t, t] uint8,
    count [1] int64), device tensors."""
    import math
    torch = _torch()
    N = U.shape[1]
    if i0 is None:
        i0 = int(math.ceil(0.9 * N))
    if t is None:
        t = N - i0
    if U.dtype != V.dtype or U.stride(1) != 1 or V.stride(1) != 1 or U.shape[0] != V.shape[0]:
        raise SpecError(-1, "U and V must be row-major with the same dtype and row count")
    dev = U.device
    if absdot is None:
        absdot = torch.empty((t, t), dtype=torch.float64, device=dev)
    if keep is None:
        keep = torch.empty((t, t), dtype=torch.uint8, device=dev)
    if count is None:
        count = torch.empty((1,), dtype=torch.int64, device=dev)
    _check(lib().spec_tail_pair_screen(_stream(), _dev(U), _dev(V), _dt(U), U.shape[0], U.stride(0), V.stride(0),
                                       int(i0), int(t), int(head_dim), float(eps), _dev(absdot), absdot.stride(0),
                                       _dev(keep), keep.stride(0), _dev(count)))
    return absdot, keep, count


def eigvalsh_batched_band_desc(band, n: int, scale: float, *, n_samples: int, p_dim: int, k: int = 1,
                               stride: int = 1, mode: int = MODE_EIG, sigma2: float = 1.0,
                               sigma2_mode: int = SIGMA2_GIVEN, top_frac: float = 0.2, small_rel: float = 1e-2,
                               tail_frac: float = 0.7, w=None, keep_w: bool = True, info=None, out=None, ws=None,
                               to_host: bool = True):
    """Window spectra and their descriptors in one pass (spec_eigvalsh_batched_desc)
    from the band [S, T, n] of gram_window.  Returns (w or None, info, records)."""
    torch = _torch()
    S, T, N = band.shape
    if N != n or not band.is_contiguous():
        raise SpecError(-1, "band must be a contiguous [streams, T, n] tensor")
    batch = S * ((T - n) // stride + 1)
    src = BatchSrc(SRC_BAND, _dev(band), 0, 0, S, T, stride, float(scale))
    dev = band.device
    if w is None and keep_w:
        w = torch.empty((batch, n), dtype=torch.float32, device=dev)
    if info is None:
        info = torch.empty((batch,), dtype=torch.int32, device=dev)
    if out is None:
        out = torch.empty((batch, DESC_DTYPE.itemsize), dtype=torch.uint8, device=dev)
    if ws is None:
        ws = torch.empty((descriptors_workspace(n),), dtype=torch.uint8, device=dev)
    p = DescParams(mode, sigma2_mode, float(sigma2), int(n_samples), int(p_dim), int(k), float(top_frac),
                   float(small_rel), float(tail_frac))
    _check(lib().spec_eigvalsh_batched_desc(_stream(), ctypes.byref(src), batch, n,
                                            _dev(w) if w is not None else None, _dev(info), ctypes.byref(p),
                                            _dev(out), _dev(ws), ws.numel()))
    rec = out.cpu().numpy().view(DESC_DTYPE).reshape(batch) if to_host else out
    return w, info, rec


def eigvalsh_batched_dense_desc(A, *, n_samples: int, p_dim: int, k: int = 1, w=None, info=None, out=None,
                                ws=None, **kw):
    """Dense batch [batch, n, n] (lower read): spectra and descriptors in one pass."""
    torch = _torch()
    if A.dim() == 2:
        A = A.unsqueeze(0)
    batch, n, _ = A.shape
    src = BatchSrc(SRC_DENSE, _dev(A), A.stride(1), A.stride(0), 0, 0, 1, 1.0)
    dev = A.device
    if w is None:
        w = torch.empty((batch, n), dtype=torch.float32, device=dev)
    if info is None:
        info = torch.empty((batch,), dtype=torch.int32, device=dev)
    if out is None:
        out = torch.empty((batch, DESC_DTYPE.itemsize), dtype=torch.uint8, device=dev)
    if ws is None:
        ws = torch.empty((descriptors_workspace(n),), dtype=torch.uint8, device=dev)
    p = DescParams(kw.get("mode", MODE_EIG), kw.get("sigma2_mode", SIGMA2_GIVEN), float(kw.get("sigma2", 1.0)),
                   int(n_samples), int(p_dim), int(k), float(kw.get("top_frac", 0.2)),
                   float(kw.get("small_rel", 1e-2)), float(kw.get("tail_frac", 0.7)))
    _check(lib().spec_eigvalsh_batched_desc(_stream(), ctypes.byref(src), batch, n, _dev(w), _dev(info),
                                            ctypes.byref(p), _dev(out), _dev(ws), ws.numel()))
    return w, info, out.cpu().numpy().view(DESC_DTYPE).reshape(batch)


# ---------------------------------------------------------------- training a projected student
#
# Gradients are calls of their own: none of these is recorded by autograd, and what
# they return of tensors that require a gradient has none.

#: Five equal steps a s + b s^3 + c s^5 that take singular values from (0, 1] to
#: about 0.7 .. 1.2 (Muon's coefficients).
NS_COEFFS = ((3.4445, -4.7750, 2.0315),) * 5


def _ids(ids, n=None):
    torch = _torch()
    if ids.dtype not in (torch.int32, torch.int64):
        raise SpecError(-2, f"token ids must be int32 or int64, not {ids.dtype}")
    if ids.dim() != 1 or not ids.is_contiguous() or (n is not None and ids.shape[0] != n):
        raise SpecError(-1, "token ids must be a contiguous vector, one per row")
    return _dev(ids), I32 if ids.dtype == torch.int32 else I64


def _rows(*ts):
    for t in ts:
        if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] != 1):
            raise SpecError(-1, "matrices must be 2-D with a contiguous inner dimension")


def _ld(t):
    """Row stride; of a single row its length, whatever stride it carries."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _vec32(t, n):
    if t.dtype != _torch().float32 or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise SpecError(-1, "per-row values must be a contiguous float32 vector, one per row")
    return _dev(t)


def _matrix(t, shape, dtype):
    """An output the caller passed: its shape and type must be the result's."""
    _rows(t)
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype:
        raise SpecError(-1, f"output must be {tuple(shape)} of {dtype}")


def _bytes(query, *args):
    b = ctypes.c_size_t(0)
    _check(query(*args, ctypes.byref(b)))
    return b.value


def _ws(ws, size, device):
    return _torch().empty((size,), dtype=_torch().uint8, device=device) if ws is None else ws


def embed(E, ids, scale: float = 1.0, out=None):
    """scale * E[ids] [n, d] for token ids [n] (int32 or int64); a zero row where
    an id is no row of E [V, d]."""
    _rows(E)
    V, d = E.shape
    p, idt = _ids(ids)
    n = ids.shape[0]
    if out is None:
        out = _torch().empty((n, d), dtype=E.dtype, device=E.device)
    _matrix(out, (n, d), E.dtype)
    _check(lib().spec_embed(_stream(), _dev(E), _dt(E), V, d, _ld(E), p, idt, n, float(scale), _dev(out), _ld(out)))
    return out


def embed_grad_workspace(n: int, V: int, d: int) -> int:
    return _bytes(lib().spec_embed_grad_workspace, n, V, d)


def embed_grad(dY, ids, V: int, scale: float = 1.0, beta: float = 0.0, dE=None, ws=None):
    """dE[v] = beta dE[v] + scale * sum of the rows dY[i] with ids[i] = v, [V, d].
    beta 0 writes every row, beta 1 adds to the rows present.  dE is of dY's type,
    or float32 for a bfloat16 dY."""
    torch = _torch()
    _rows(dY)
    n, d = dY.shape
    p, idt = _ids(ids, n)
    if dE is None:
        if beta != 0.0:
            raise SpecError(-1, "beta needs the dE to add to")
        dE = torch.empty((V, d), dtype=dY.dtype, device=dY.device)
    _matrix(dE, (V, d), dE.dtype)
    ws = _ws(ws, embed_grad_workspace(n, V, d), dY.device)
    _check(lib().spec_embed_grad(_stream(), _dev(dY), _dt(dY), n, V, d, _ld(dY), p, idt, float(scale), float(beta),
                                 _dev(dE), _dt(dE), _ld(dE), _dev(ws), ws.numel()))
    return dE


def _head(H, W):
    _rows(H, W)
    if H.shape[1] != W.shape[1] or H.dtype != W.dtype:
        raise SpecError(-1, "H [T, d] and W [V, d] must agree in d and type")
    return H.shape[0], W.shape[0], W.shape[1]


def linear_xent_workspace(T: int, V: int, d: int, dtype) -> int:
    return _bytes(lib().spec_linear_xent_workspace, T, V, d, _dt(_torch().empty(0, dtype=dtype)))


def linear_xent(H, W, target, scale: float = 1.0, loss=None, lse=None, ws=None):
    """Softmax cross entropy of the logits scale * H W^T: (loss, lse), float32
    [T], both 0 where target is no row of W.  H [T, d], W [V, d]."""
    torch = _torch()
    T, V, d = _head(H, W)
    p, tt = _ids(target, T)
    if loss is None:
        loss = torch.empty((T,), dtype=torch.float32, device=H.device)
    if lse is None:
        lse = torch.empty((T,), dtype=torch.float32, device=H.device)
    t = _dt(H)
    ws = _ws(ws, _bytes(lib().spec_linear_xent_workspace, T, V, d, t), H.device)
    _check(lib().spec_linear_xent(_stream(), _dev(H), _dev(W), t, T, V, d, _ld(H), _ld(W), p, tt, float(scale),
                                  _vec32(loss, T), _vec32(lse, T), _dev(ws), ws.numel()))
    return loss, lse


def linear_xent_grad_workspace(T: int, V: int, d: int, dtype) -> int:
    return _bytes(lib().spec_linear_xent_grad_workspace, T, V, d, _dt(_torch().empty(0, dtype=dtype)))


def linear_xent_grad(H, W, target, lse, dloss, scale: float = 1.0, beta: float = 0.0, dH=None, dW=None, ws=None):
    """Gradients of sum(dloss * loss) of linear_xent, with its lse: dH [T, d] and
    dW = beta dW + ... [V, d].  dloss: float32 [T]."""
    torch = _torch()
    T, V, d = _head(H, W)
    p, tt = _ids(target, T)
    if dH is None:
        dH = torch.empty((T, d), dtype=H.dtype, device=H.device)
    if dW is None:
        if beta != 0.0:
            raise SpecError(-1, "beta needs the dW to add to")
        dW = torch.empty((V, d), dtype=W.dtype, device=W.device)
    _matrix(dH, (T, d), H.dtype)
    _matrix(dW, (V, d), W.dtype)
    t = _dt(H)
    ws = _ws(ws, _bytes(lib().spec_linear_xent_grad_workspace, T, V, d, t), H.device)
    _check(lib().spec_linear_xent_grad(_stream(), _dev(H), _dev(W), t, T, V, d, _ld(H), _ld(W), p, tt, float(scale),
                                       _vec32(lse, T), _vec32(dloss, T), float(beta), _dev(dH), _ld(dH), _dev(dW),
                                       _ld(dW), _dev(ws), ws.numel()))
    return dH, dW


def orthogonalize_workspace(batch: int, m: int, n: int, dtype) -> int:
    return _bytes(lib().spec_orthogonalize_workspace, batch, m, n, _dt(_torch().empty(0, dtype=dtype)))


def orthogonalize(G, coeffs=NS_COEFFS, eps: float = 1e-7, scale: float = 1.0, out=None, ws=None):
    """Newton-Schulz orthogonalisation of G [m, n] or [batch, m, n]: one step
    X <- a X + (b X X^T + c (X X^T)^2) X per (a, b, c) of coeffs, from
    X = G / (|G|_F + eps); returns scale * X in G's type (out may be G)."""
    torch = _torch()
    if out is None:
        out = torch.empty(G.shape, dtype=G.dtype, device=G.device)
    if G.dim() not in (2, 3) or out.shape != G.shape or out.dtype != G.dtype:
        raise SpecError(-1, "G must be [m, n] or [batch, m, n] and out of its shape and type")
    g, o = (G.unsqueeze(0), out.unsqueeze(0)) if G.dim() == 2 else (G, out)
    batch, m, n = g.shape
    if (g.stride(2) != 1 or o.stride(2) != 1) and n != 1:
        raise SpecError(-1, "inner dimension must be contiguous")

    def strides(t):
        ld = t.stride(1) if m > 1 else n
        return ld, (t.stride(0) if batch > 1 else m * ld)
    (ldg, sg), (ldo, so) = strides(g), strides(o)
    steps = len(coeffs)
    co = (ctypes.c_double * (3 * max(steps, 1)))(*[float(x) for c in coeffs for x in c])
    t = _dt(G)
    ws = _ws(ws, _bytes(lib().spec_orthogonalize_workspace, batch, m, n, t), G.device)
    _check(lib().spec_orthogonalize(_stream(), _dev(G), t, batch, m, n, ldg, sg, co, steps, float(eps), float(scale),
                                    _dev(out), ldo, so, _dev(ws), ws.numel()))
    return out


# ---------------------------------------------------------------- a student's residual blocks
#
# As above, gradients are calls of their own.  Tensors have to be on the current device.

class Mx(NamedTuple):
    """A microscaled matrix: codes uint8 [rows, ldq], scales uint8 [rows, lds] (contiguous
    rows, a row's bytes as mx_empty gives them or more), its columns and its format."""
    q: Any
    s: Any
    cols: int
    fmt: int


# The calls below are short on the GPU for a decode step, so their way there is kept
# short too: sizes are looked at once, and what the call itself made not again.

def _on(t):
    """The device of a tensor, which must be the current one."""
    if not t.is_cuda:
        raise SpecError(-1, "tensor must be on the GPU")
    dev = t.get_device()
    if dev != _torch()._C._cuda_getDevice():
        raise SpecError(-1, "tensor must be on the current device")
    return dev


def _at(t, dev):
    """The address of a tensor, which must be on this device."""
    if t.get_device() != dev:
        raise SpecError(-1, "tensors must be on the current device")
    return t.data_ptr()


def _mat(t, shape, dtype, dev):
    """(address, row stride) of a matrix of this shape and type with contiguous rows."""
    if t.shape != shape or t.dtype != dtype:
        raise SpecError(-1, f"matrix must be {tuple(shape)} of {dtype}")
    st = t.stride()
    if st[1] != 1 and shape[1] != 1:
        raise SpecError(-1, "matrices must have a contiguous inner dimension")
    return _at(t, dev), st[0] if shape[0] > 1 else shape[1]


def _shape(t):
    if t.dim() != 2:
        raise SpecError(-1, "matrices must be 2-D with a contiguous inner dimension")
    return t.shape


def _launch(f, dev, *args):
    status = f(_torch()._C._cuda_getCurrentRawStream(dev), *args)
    if status != 0:
        _check(status)


@functools.lru_cache(maxsize=1024)
def _workspace(query, *sizes):
    """Bytes of a workspace: a function of the sizes alone."""
    return _bytes(getattr(lib(), query), *sizes)


def _scratch(ws, size, dev):
    """(address, bytes, the tensor itself, which has to live until the call returns)."""
    if ws is None:
        torch = _torch()
        ws = torch.empty(size, dtype=torch.uint8, device=dev)
        return ws.data_ptr(), size, ws
    if not ws.is_contiguous():  # its elements would not be its bytes (expand)
        raise SpecError(-1, "a workspace must be contiguous")
    return _at(ws, dev), ws.numel() * ws.element_size(), ws


def _mx_rows(fmt, cols):
    if fmt not in (MX_INT8, MX_FP4):
        raise SpecError(-2, f"unsupported microscaled format {fmt}")
    if cols < 1:
        raise SpecError(-1, "a microscaled matrix has columns")
    blocks = (cols + 31) // 32
    return blocks * (32 if fmt == MX_INT8 else 16), (blocks + 15) // 16 * 16


def _mx(m, rows, cols, dev=None):
    """The C descriptor of a microscaled matrix of these sizes (None: any)."""
    if type(m) is not Mx:
        raise SpecError(-1, "a microscaled matrix (Mx) is needed")
    u8, (q, s, c, fmt) = _torch().uint8, m
    if q.dtype != u8 or s.dtype != u8 or q.dim() != 2 or s.dim() != 2:
        raise SpecError(-1, "codes and scales must be uint8 [rows, bytes]")
    (n, wq), (ns, wsc), (ldq, iq), (lds, isc) = q.shape, s.shape, q.stride(), s.stride()
    lq, ls = _mx_rows(fmt, c)
    if n != ns or wq < lq or wsc < ls or iq != 1 or isc != 1:
        raise SpecError(-1, f"rows of {c} columns are {lq} contiguous bytes of codes and {ls} of scales")
    if (rows is not None and n != rows) or (cols is not None and c != cols):
        raise SpecError(-1, f"the microscaled matrix must be {rows} x {cols}, not {n} x {c}")
    if dev is None:
        dev = _on(q)
    return MxMatrix(_at(q, dev), _at(s, dev), ldq if n > 1 else lq, lds if n > 1 else ls, fmt)


def mx_empty(rows: int, cols: int, fmt: int, device="cuda") -> Mx:
    """Uninitialised storage of a microscaled matrix (mx_quantize and block_norm fill it)."""
    torch = _torch()
    lq, ls = _mx_rows(fmt, cols)
    return Mx(torch.empty((rows, lq), dtype=torch.uint8, device=device),
              torch.empty((rows, ls), dtype=torch.uint8, device=device), cols, fmt)


def mx_quantize(X, fmt: int, out: Mx = None) -> Mx:
    """X [rows, cols] (bfloat16 or float32) in microscaled storage, MX_INT8 or MX_FP4."""
    shape = rows, cols = _shape(X)
    lq, ls = _mx_rows(fmt, cols)
    if out is not None and out.fmt != fmt:
        raise SpecError(-1, "out has another format")
    dev = _on(X)
    x, ldx = _mat(X, shape, X.dtype, dev)
    if out is None:
        out = mx_empty(rows, cols, fmt, dev)
        o = MxMatrix(out.q.data_ptr(), out.s.data_ptr(), lq, ls, fmt)
    else:
        o = _mx(out, rows, cols, dev)
    _launch(lib().spec_mx_quantize, dev, x, _dt(X), rows, cols, ldx, o)
    return out


def mx_dequantize(m: Mx, dtype=None, out=None):
    """The values of a microscaled matrix, bfloat16 (the default) or float32."""
    d = _mx(m, None, None)
    torch, dev, rows, cols = _torch(), m.q.get_device(), m.q.shape[0], m.cols
    if out is None:
        out = torch.empty((rows, cols), dtype=dtype or torch.bfloat16, device=dev)
        o = out.data_ptr(), cols
    else:
        o = _mat(out, (rows, cols), dtype or out.dtype, dev)
    _launch(lib().spec_mx_dequantize, dev, d, rows, cols, o[0], _dt(out), o[1])
    return out


def mx_plan(op: int, T: int, N: int, K: int, dtype):
    """(edge of the tiles, shares of the sums' dimension) that mx_linear (MX_OP_LINEAR), mx_product
    (MX_OP_PRODUCT) or mx_weight_grad (MX_OP_WEIGHT_GRAD) takes for these sizes."""
    edge, shares = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().spec_mx_plan(op, T, N, K, _dt(_torch().empty(0, dtype=dtype)), edge, shares))
    return edge.value, shares.value


def mx_linear_workspace(T: int, N: int, K: int, dtype) -> int:
    return _workspace("spec_mx_linear_workspace", T, N, K, _dt(_torch().empty(0, dtype=dtype)))


def mx_linear(X, W: Mx, out=None, ws=None):
    """X W^T [T, N] for X [T, K] (bfloat16 or float32) and W [N, K] in MX_FP4."""
    shape = T, K = _shape(X)
    t = _dt(X)
    if type(W) is not Mx or W.cols != K:
        raise SpecError(-1, f"W must be a microscaled matrix of {K} columns")
    dev = _on(X)
    w, N = _mx(W, None, K, dev), W.q.shape[0]
    x, ldx = _mat(X, shape, X.dtype, dev)
    if out is None:
        out = _torch().empty((T, N), dtype=X.dtype, device=dev)
        o = out.data_ptr(), N
    else:
        o = _mat(out, (T, N), X.dtype, dev)
    p, size, ws = _scratch(ws, _workspace("spec_mx_linear_workspace", T, N, K, t), dev)
    _launch(lib().spec_mx_linear, dev, x, t, T, N, K, ldx, w, *o, p, size)
    return out


def mx_product_workspace(T: int, N: int, K: int) -> int:
    return _workspace("spec_mx_product_workspace", T, N, K)


def mx_product(X: Mx, W: Mx, dtype=None, out=None, ws=None):
    """X W^T [T, N] in bfloat16 (the default) or float32 for X [T, K] and W [N, K] in MX_FP4."""
    x = _mx(X, None, None)
    torch, dev, T, K = _torch(), X.q.get_device(), X.q.shape[0], X.cols
    w, N = _mx(W, None, K, dev), W.q.shape[0]
    if out is None:
        out = torch.empty((T, N), dtype=dtype or torch.bfloat16, device=dev)
        o = out.data_ptr(), N
    else:
        o = _mat(out, (T, N), dtype or out.dtype, dev)
    p, size, ws = _scratch(ws, _workspace("spec_mx_product_workspace", T, N, K), dev)
    _launch(lib().spec_mx_product, dev, x, w, T, N, K, o[0], _dt(out), o[1], p, size)
    return out


def mx_weight_grad_workspace(T: int, N: int, K: int, dtype) -> int:
    return _workspace("spec_mx_weight_grad_workspace", T, N, K, _dt(_torch().empty(0, dtype=dtype)))


def mx_weight_grad(dY, X: Mx, beta: float = 0.0, dW=None, ws=None):
    """dW = beta dW + dY^T X [N, K] in dY's type, for dY [T, N] (bfloat16 or float32) and
    X [T, K] in MX_INT8."""
    shape = T, N = _shape(dY)
    t = _dt(dY)
    if type(X) is not Mx or X.q.shape[0] != T:
        raise SpecError(-1, f"X must be a microscaled matrix of {T} rows")
    dev = _on(dY)
    x, K = _mx(X, T, None, dev), X.cols
    y, ldy = _mat(dY, shape, dY.dtype, dev)
    if dW is None:
        if beta != 0.0:
            raise SpecError(-1, "beta needs the dW to add to")
        dW = _torch().empty((N, K), dtype=dY.dtype, device=dev)
        o = dW.data_ptr(), K
    else:
        o = _mat(dW, (N, K), dY.dtype, dev)
    p, size, ws = _scratch(ws, _workspace("spec_mx_weight_grad_workspace", T, N, K, t), dev)
    _launch(lib().spec_mx_weight_grad, dev, y, t, T, N, K, ldy, x, float(beta), *o, p, size)
    return dW


def _block(n, d, dtype, t, dev, post, w_post, w_pre, gate, gate_rows, alpha, beta, eps):
    """The C descriptor of a block's norms: (Block, gate rows)."""
    def vec(w):
        if w is None:
            return None
        if w.dtype != dtype or w.shape != (d,) or (w.stride(0) != 1 and d > 1):
            raise SpecError(-1, f"weights must be contiguous [{d}] of {dtype}")
        return _at(w, dev)
    ldg, gates, g = d, 0, None
    if gate is not None:
        if gate.dim() == 1:
            gate, gate_rows = gate.unsqueeze(0), max(n, 1)
        gates = (n + gate_rows - 1) // gate_rows if gate_rows >= 1 else -1
        if gate.dim() != 2 or gate.dtype != dtype or gate.shape[1] != d or gates < 0 or gate.shape[0] < gates:
            raise SpecError(-1, f"gate must be [rows / gate_rows, {d}] of {dtype}, or [{d}]")
        g, ldg = _mat(gate, gate.shape, dtype, dev)
    return Block(n, d, t, 1 if post else 0, alpha, beta, eps, vec(w_post), vec(w_pre), g, ldg, gate_rows), gates


def block_norm(H, Y=None, post: bool = True, w_post=None, w_pre=None, gate=None, gate_rows: int = 1, alpha: float = 1.0,
               beta: float = 1.0, eps: float = 1e-6, Hout=None, X=None, y8: Mx = None, h8: Mx = None, x8: Mx = None):
    """The norms around a residual block: u = norm(Y) w_post (post) or Y, Hout = alpha H + beta gate u,
    X = norm(Hout) w_pre.  Returns (Hout, X, r_post, r_pre), r the rows' factors of the two norms
    (None where there is none); without Y, Hout is H (and cannot be passed).  gate: [d], or
    [rows, d] of which one row serves gate_rows rows of Y.  y8, h8, x8: MX_INT8 storage that
    receives Y, Hout and X.  Hout may be H, X may be Y."""
    torch, dtype, t = _torch(), H.dtype, _dt(H)
    shape = n, d = _shape(H)
    if Y is None and not (Hout is None and y8 is None and h8 is None):
        raise SpecError(-1, "without Y there is no Hout, y8 or h8 to write")
    dev = _on(H)
    h, ldh = _mat(H, shape, dtype, dev)
    b, _ = _block(n, d, dtype, t, dev, post, w_post, w_pre, gate, gate_rows, alpha, beta, eps)
    y = ho = (None, 0)
    r_post = p_post = None
    if Y is None:
        Hout = H
    else:
        y = _mat(Y, shape, dtype, dev)
        if Hout is None:
            Hout = torch.empty(shape, dtype=dtype, device=dev)
            ho = Hout.data_ptr(), d
        else:
            ho = _mat(Hout, shape, dtype, dev)
        if post:
            r_post = torch.empty(n, dtype=torch.float32, device=dev)
            p_post = r_post.data_ptr()
    if X is None:
        X = torch.empty(shape, dtype=dtype, device=dev)
        x = X.data_ptr(), d
    else:
        x = _mat(X, shape, dtype, dev)
    r_pre = torch.empty(n, dtype=torch.float32, device=dev)
    y8, h8, x8 = (None if m is None else _mx(m, n, d, dev) for m in (y8, h8, x8))
    _launch(lib().spec_block_norm, dev, b, *y, h, ldh, *ho, *x, p_post, r_pre.data_ptr(), y8, h8, x8)
    return Hout, X, r_post, r_pre


@functools.lru_cache(maxsize=1024)
def _block_grad_workspace(n, d, t, gates, gate_rows):
    b = Block(n, d, t, 0, 1.0, 1.0, 1e-6, None, None, 256 if gates else None, d, gate_rows)
    return _bytes(lib().spec_block_norm_grad_workspace, b)


def block_norm_grad_workspace(n: int, d: int, dtype, gates: int = 0, gate_rows: int = 1) -> int:
    """Workspace of block_norm_grad, with `gates` gate rows (0: no gate) of gate_rows rows each."""
    return _block_grad_workspace(n, d, _dt(_torch().empty(0, dtype=dtype)), gates, gate_rows)


def block_norm_grad(dX, dHout, Hout, Y, r_pre, r_post=None, post: bool = True, w_post=None, w_pre=None, gate=None,
                    gate_rows: int = 1, alpha: float = 1.0, beta: float = 1.0, dH=None, dY=None, ws=None):
    """Gradients of block_norm from those of its X and (otherwise than through X) of its Hout; one
    of them may be None: zero.  Hout and Y as they were, or as stored in MX_INT8; Y None: no block,
    the gradients of the norm of Hout itself.
    Returns (dH, dY, dw_post, dw_pre, dgate), the last three float32, None for what was not given.
    dH may be dHout, dY may be dX."""
    torch = _torch()
    like = dX if dX is not None else dHout
    if like is None:
        raise SpecError(-1, "a gradient of X or of Hout is needed")
    dtype, t = like.dtype, _dt(like)
    shape = n, d = _shape(like)
    if Y is None:
        if dY is not None:
            raise SpecError(-1, "without Y there is no dY to write")
        post, w_post, gate = False, None, None
    dev = _on(like)
    b, gates = _block(n, d, dtype, t, dev, post, w_post, w_pre, gate, gate_rows, alpha, beta, 1e-6)
    none = (None, 0)

    def given(m):
        """(address, stride, descriptor) of a matrix or of its checkpoint."""
        if type(m) is Mx:
            return None, 0, _mx(m, n, d, dev)
        return (*(none if m is None else _mat(m, shape, dtype, dev)), None)

    def result(m):
        if m is None:
            m = torch.empty(shape, dtype=dtype, device=dev)
            return m, (m.data_ptr(), d)
        return m, _mat(m, shape, dtype, dev)

    def sums(wanted, *size):
        if not wanted:
            return None, None
        m = torch.empty(size, dtype=torch.float32, device=dev)
        return m, m.data_ptr()

    def factors(r):
        if r.dtype != torch.float32 or r.shape != (n,) or (n > 1 and r.stride(0) != 1):
            raise SpecError(-1, "per-row values must be a contiguous float32 vector, one per row")
        return _at(r, dev)
    y, ho = given(Y), given(Hout) if dX is not None else (None, 0, None)
    dx, do = (none if m is None else _mat(m, shape, dtype, dev) for m in (dX, dHout))
    dH, dh = result(dH)
    dY, dy = (None, none) if Y is None else result(dY)
    dw_post, p_post = sums(w_post is not None, d)
    dw_pre, p_pre = sums(dX is not None and w_pre is not None, d)
    dgate, p_gate = sums(gate is not None, gates, d)
    r1 = factors(r_post) if post and r_post is not None else None
    r2 = factors(r_pre) if dX is not None and r_pre is not None else None
    # (a single gate row serves all rows)
    p, size, ws = _scratch(ws, _block_grad_workspace(n, d, t, gates, b.gate_rows if gates else 1), dev)
    _launch(lib().spec_block_norm_grad, dev, b, *y, *ho, r1, r2, *do, *dx, *dh, *dy, p_post, p_pre, p_gate, p, size)
    if gate is not None and gate.dim() == 1:
        dgate = dgate.view(d) if n > 0 else torch.zeros(d, dtype=torch.float32, device=dev)  # (a sum over no rows)
    return dH, dY, dw_post, dw_pre, dgate
