"""Thin ctypes binding of libmhc (include/mhc.h).

Argument marshalling only: every step of the forward runs in the HIP kernels
of libmhc.  Tensors are torch tensors used as device-memory handles; the
current torch HIP stream is passed unless a stream is given.  There is no CPU
fallback: if the library is missing or fails to load, every call raises.
"""

import ctypes
import functools
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmhc.so")

MHC_OK = 0
MHC_ERR_INVALID_ARG = 1
MHC_ERR_UNSUPPORTED = 2
MHC_ERR_WORKSPACE = 3
MHC_ERR_HIP = 4
MHC_ERR_INCOMPLETE = 5
MHC_SINKHORN_ITERS = 20
MHC_ROUTE_SOFTMAX = 1
MHC_ROUTE_RENORM = 2
MHC_ROUTE_BF16 = 4

EXPORTED = ("mhc_status_string", "mhc_coeffs_workspace_size", "mhc_coeffs_split_k",
            "mhc_coeffs", "mhc_pre", "mhc_post_res", "mhc_post_res_coeffs_workspace_size",
            "mhc_post_res_coeffs", "mhc_coeffs_fp8_workspace_size", "mhc_coeffs_fp8",
            "mhc_pre_fp8", "mhc_post_res_fp8", "mhc_post_res_coeffs_fp8_workspace_size",
            "mhc_post_res_coeffs_fp8", "mhc_coeffs_phi32_workspace_size", "mhc_coeffs_phi32",
            "mhc_post_res_coeffs_phi32_workspace_size", "mhc_post_res_coeffs_phi32",
            "mhc_lazy_prenorm_gemm", "mhc_post_res_coeffs_pre_workspace_size",
            "mhc_post_res_coeffs_pre", "mhc_post_res_coeffs_pre_one_pass",
            "mhc_post_res_coeffs_pre_fp8_workspace_size", "mhc_post_res_coeffs_pre_fp8",
            "mhc_post_res_coeffs_pre_fp8_one_pass", "mhc_post_res_coeffs_pre_check",
            "mhc_tuning_set", "mhc_tuning_reset", "mhc_post_res_coeffs_pre_noalloc",
            "mhc_coeffs_pre_workspace_size", "mhc_coeffs_pre", "mhc_coeffs_pre_one_pass",
            "mhc_coeffs_pre_check", "mhc_coeffs_pre_fp8_workspace_size", "mhc_coeffs_pre_fp8",
            "mhc_coeffs_pre_fp8_one_pass", "mhc_ckpt_scales_per_row", "mhc_ckpt_pack", "mhc_ckpt_unpack",
            "mhc_post_res_bwd", "mhc_post_res_bwd_ckpt", "mhc_coeffs_pre_bwd_workspace_size",
            "mhc_coeffs_pre_bwd", "mhc_coeffs_pre_bwd_ckpt", "mhc_embed", "mhc_embed_bwd_workspace_size",
            "mhc_embed_bwd", "mhc_rmsnorm", "mhc_rmsnorm_bwd_workspace_size", "mhc_rmsnorm_bwd", "mhc_route",
            "mhc_route_bwd", "mhc_experts_order_workspace_size", "mhc_experts_order", "mhc_experts_gather",
            "mhc_experts_gather_ckpt", "mhc_experts_combine", "mhc_experts_combine_bwd")

MHC_NOALLOC_SCRATCH_BYTES = 32 << 20

_lib = None


class MhcError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {mhc_status_string(status)} (status {status})")


def load():
    """Load libmhc.so once and declare the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run `python -m manifold_constrained_hyper_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    i64, i32, vp, f32, sz = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float, ctypes.c_size_t
    lib.mhc_status_string.argtypes = [ctypes.c_int]
    lib.mhc_status_string.restype = ctypes.c_char_p
    lib.mhc_coeffs_workspace_size.argtypes = [i64, i32, i64]
    lib.mhc_coeffs_workspace_size.restype = sz
    lib.mhc_coeffs_split_k.argtypes = [i64, i32, i64]
    lib.mhc_coeffs_split_k.restype = i32
    lib.mhc_coeffs.argtypes = [i64, i32, i64, vp, vp, f32, f32, f32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.mhc_coeffs.restype = ctypes.c_int
    lib.mhc_pre.argtypes = [i64, i32, i64, vp, vp, vp, vp]
    lib.mhc_pre.restype = ctypes.c_int
    lib.mhc_post_res.argtypes = [i64, i32, i64, vp, vp, vp, vp, vp]
    lib.mhc_post_res.restype = ctypes.c_int
    lib.mhc_post_res_coeffs_workspace_size.argtypes = [i64, i32, i64]
    lib.mhc_post_res_coeffs_workspace_size.restype = sz
    lib.mhc_post_res_coeffs.argtypes = [i64, i32, i64, vp, vp, vp, vp, vp, f32, f32, f32,
                                        vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.mhc_post_res_coeffs.restype = ctypes.c_int
    for suffix in ("", "_fp8", "_phi32"):
        if suffix:
            getattr(lib, "mhc_coeffs" + suffix).argtypes = lib.mhc_coeffs.argtypes
            getattr(lib, "mhc_coeffs" + suffix).restype = ctypes.c_int
            if suffix == "_fp8":
                getattr(lib, "mhc_pre" + suffix).argtypes = lib.mhc_pre.argtypes
                getattr(lib, "mhc_pre" + suffix).restype = ctypes.c_int
                getattr(lib, "mhc_post_res" + suffix).argtypes = lib.mhc_post_res.argtypes
                getattr(lib, "mhc_post_res" + suffix).restype = ctypes.c_int
            getattr(lib, "mhc_post_res_coeffs" + suffix).argtypes = lib.mhc_post_res_coeffs.argtypes
            getattr(lib, "mhc_post_res_coeffs" + suffix).restype = ctypes.c_int
    lib.mhc_coeffs_fp8_workspace_size.argtypes = [i64, i32, i64]
    lib.mhc_coeffs_fp8_workspace_size.restype = sz
    lib.mhc_post_res_coeffs_fp8_workspace_size.argtypes = [i64, i32, i64]
    lib.mhc_post_res_coeffs_fp8_workspace_size.restype = sz
    lib.mhc_coeffs_phi32_workspace_size.argtypes = [i64, i32, i64]
    lib.mhc_coeffs_phi32_workspace_size.restype = sz
    lib.mhc_post_res_coeffs_phi32_workspace_size.argtypes = [i64, i32, i64]
    lib.mhc_post_res_coeffs_phi32_workspace_size.restype = sz
    lib.mhc_lazy_prenorm_gemm.argtypes = [i64, i64, i64, vp, vp, f32, vp, vp, vp]
    lib.mhc_lazy_prenorm_gemm.restype = ctypes.c_int
    lib.mhc_post_res_coeffs_pre_workspace_size.argtypes = [i64, i32, i64]
    lib.mhc_post_res_coeffs_pre_workspace_size.restype = sz
    lib.mhc_post_res_coeffs_pre.argtypes = [i64, i32, i64, vp, vp, vp, vp, vp, f32, f32, f32,
                                            vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.mhc_post_res_coeffs_pre.restype = ctypes.c_int
    lib.mhc_post_res_coeffs_pre_one_pass.argtypes = [i64, i32, i64]
    lib.mhc_post_res_coeffs_pre_one_pass.restype = i32
    lib.mhc_post_res_coeffs_pre_fp8_workspace_size.argtypes = [i64, i32, i64]
    lib.mhc_post_res_coeffs_pre_fp8_workspace_size.restype = sz
    lib.mhc_post_res_coeffs_pre_fp8.argtypes = [i64, i32, i64, vp, vp, vp, vp, vp, f32, f32, f32,
                                                vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.mhc_post_res_coeffs_pre_fp8.restype = ctypes.c_int
    lib.mhc_post_res_coeffs_pre_fp8_one_pass.argtypes = [i64, i32, i64]
    lib.mhc_post_res_coeffs_pre_fp8_one_pass.restype = i32
    lib.mhc_post_res_coeffs_pre_check.argtypes = [i64, i32, i64, i32, vp, sz, vp]
    lib.mhc_post_res_coeffs_pre_check.restype = ctypes.c_int
    lib.mhc_tuning_set.argtypes = [ctypes.c_char_p, i64]
    lib.mhc_tuning_set.restype = ctypes.c_int
    lib.mhc_post_res_coeffs_pre_noalloc.argtypes = [i64, i32, i64, vp, vp, vp, vp, vp, f32, f32, f32,
                                                    vp, vp, vp, vp, vp, vp, vp, vp]
    lib.mhc_post_res_coeffs_pre_noalloc.restype = ctypes.c_int
    for suffix in ("", "_fp8"):
        getattr(lib, f"mhc_coeffs_pre{suffix}_workspace_size").argtypes = [i64, i32, i64]
        getattr(lib, f"mhc_coeffs_pre{suffix}_workspace_size").restype = sz
        getattr(lib, f"mhc_coeffs_pre{suffix}").argtypes = [i64, i32, i64, vp, vp, f32, f32, f32, vp, vp,
                                                           vp, vp, vp, vp, vp, vp, sz, vp]
        getattr(lib, f"mhc_coeffs_pre{suffix}").restype = ctypes.c_int
        getattr(lib, f"mhc_coeffs_pre{suffix}_one_pass").argtypes = [i64, i32, i64]
        getattr(lib, f"mhc_coeffs_pre{suffix}_one_pass").restype = i32
    lib.mhc_coeffs_pre_check.argtypes = [i64, i32, i64, i32, vp, sz, vp]
    lib.mhc_coeffs_pre_check.restype = ctypes.c_int
    lib.mhc_ckpt_scales_per_row.argtypes = [i32, i64]
    lib.mhc_ckpt_scales_per_row.restype = i64
    lib.mhc_coeffs_pre_bwd_workspace_size.argtypes = [i64, i32, i64]
    lib.mhc_coeffs_pre_bwd_workspace_size.restype = sz
    lib.mhc_embed_bwd_workspace_size.argtypes = [i64, i32, i64, i64]
    lib.mhc_embed_bwd_workspace_size.restype = sz
    shape, bwd = [i64, i32, i64], [vp, f32, f32, f32] + [vp] * 16 + [sz, vp]
    for name, args in (("mhc_ckpt_pack", [vp] * 4), ("mhc_ckpt_unpack", [vp] * 4), ("mhc_post_res_bwd", [vp] * 7),
                       ("mhc_post_res_bwd_ckpt", [vp] * 8), ("mhc_coeffs_pre_bwd", [vp] + bwd),
                       ("mhc_coeffs_pre_bwd_ckpt", [vp] * 2 + bwd), ("mhc_embed", [i64, vp, vp, f32, vp, vp]),
                       ("mhc_embed_bwd", [i64, vp, vp, f32, i32, vp, vp, sz, vp])):
        getattr(lib, name).argtypes = shape + args
        getattr(lib, name).restype = ctypes.c_int
    lib.mhc_rmsnorm_bwd_workspace_size.argtypes = [i64, i64]
    lib.mhc_rmsnorm_bwd_workspace_size.restype = sz
    lib.mhc_experts_order_workspace_size.argtypes = [i64, i32, i32]
    lib.mhc_experts_order_workspace_size.restype = sz
    for name, args in (("mhc_rmsnorm", [i64, i64] + [vp] * 3 + [f32] + [vp] * 6),
                       ("mhc_rmsnorm_bwd", [i64, i64] + [vp] * 8 + [sz, vp]),
                       ("mhc_route", [i64] + [i32] * 5 + [f32] + [vp] * 5),
                       ("mhc_route_bwd", [i64] + [i32] * 3 + [f32] + [vp] * 5),
                       ("mhc_experts_order", [i64, i32, i32] + [vp] * 4 + [sz, vp]),
                       ("mhc_experts_gather", [i64, i32, i64] + [vp] * 4),
                       ("mhc_experts_gather_ckpt", [i64, i32, i64] + [vp] * 6),
                       ("mhc_experts_combine", [i64, i32, i64] + [vp] * 6),
                       ("mhc_experts_combine_bwd", [i64, i32, i64] + [vp] * 7)):
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = ctypes.c_int
    lib.mhc_tuning_reset.argtypes = []
    lib.mhc_tuning_reset.restype = None
    _lib = lib
    return lib


def _ptr(t, nbytes=None, esize=None, name="tensor"):
    """Device pointer of a tensor (None -> NULL; an int is taken as a raw
    address).  Raises ValueError on host or non-contiguous tensors and, when
    the call's sizes are given, on a tensor of another element size (uint8
    tensors are taken as raw bytes) or smaller than the nbytes the library
    will touch, before anything runs."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        return int(t)  # raw address
    if esize is not None and t.numel() > 0 and t.element_size() != esize and t.dtype != torch.uint8:
        raise ValueError(f"{name}: element size {t.element_size()} bytes, the call takes {esize}")
    if nbytes is not None and t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{name}: {t.numel() * t.element_size()} bytes, the call needs {nbytes}")
    if not t.is_contiguous():
        raise ValueError("libmhc takes contiguous tensors")
    if t.numel() > 0 and not t.is_cuda:
        raise ValueError("libmhc takes device tensors")
    return t.data_ptr() or None


class _Sizes:
    """Byte counts of the tensors of one (B, n, C) call: eb bytes per
    residual-stream element (2 bf16, 1 E4M3), pb per phi element."""

    def __init__(self, B, n, C, eb=2, pb=2):
        B, n, C = int(B), int(n), int(C)
        N = n * n + 2 * n
        self.eb, self.pb = eb, pb
        self.x = max(B, 0) * n * C * eb       # X_t, X_next
        self.f = max(B, 0) * C * eb           # F_out, F_pre
        self.phi = n * C * N * pb
        self.coef = max(B, 0) * N * 4         # logits, H
        self.r = max(B, 0) * 4
        self.nb = n * 4                       # b_pre, b_post
        self.nr = n * n * 4                   # b_res
        if B <= 0:  # B == 0 touches nothing (and B < 0 is the library's error to report)
            self.x = self.f = self.phi = self.coef = self.r = self.nb = self.nr = 0


def _coeff_args(z, phi, b_pre, b_post, b_res, logits, r, H):
    return (_ptr(phi, z.phi, z.pb, "phi"), _ptr(b_pre, z.nb, 4, "b_pre"), _ptr(b_post, z.nb, 4, "b_post"),
            _ptr(b_res, z.nr, 4, "b_res"), _ptr(logits, z.coef, 4, "logits"), _ptr(r, z.r, 4, "r"),
            _ptr(H, z.coef, 4, "H"))


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(status, where):
    if status != MHC_OK:
        raise MhcError(status, where)


def mhc_status_string(status):
    return load().mhc_status_string(int(status)).decode()


def mhc_tuning_set(name, value):
    """Override a route or launch-shape choice process-wide (tests and tuning;
    value < 0 restores the default).  See include/mhc.h."""
    _check(load().mhc_tuning_set(str(name).encode(), int(value)), f"mhc_tuning_set({name})")


def mhc_tuning_reset():
    """Restore every route and launch-shape choice to its default."""
    load().mhc_tuning_reset()


def _ws_bytes(workspace, workspace_bytes):
    if workspace_bytes is not None:
        return int(workspace_bytes)
    return workspace.numel() * workspace.element_size() if isinstance(workspace, torch.Tensor) else 0


def mhc_coeffs_workspace_size(B, n, C):
    return int(load().mhc_coeffs_workspace_size(int(B), int(n), int(C)))


def mhc_coeffs_split_k(B, n, C):
    return int(load().mhc_coeffs_split_k(int(B), int(n), int(C)))


def _coeffs(fn, name, eb, pb, B, n, C, X_t, phi, alpha_pre, alpha_post, alpha_res, b_pre, b_post,
            b_res, logits, r, H, workspace, workspace_bytes, stream, check):
    z = _Sizes(B, n, C, eb, pb)
    pp, bp, bq, br, lg, rr, hh = _coeff_args(z, phi, b_pre, b_post, b_res, logits, r, H)
    wb = _ws_bytes(workspace, workspace_bytes)
    st = fn(int(B), int(n), int(C), _ptr(X_t, z.x, eb, "X_t"), pp, float(alpha_pre), float(alpha_post),
            float(alpha_res), bp, bq, br, lg, rr, hh, _ptr(workspace, wb, None, "workspace"), wb,
            _stream(stream))
    if check:
        _check(st, name)
    return st


def mhc_coeffs(B, n, C, X_t, phi, alpha_pre, alpha_post, alpha_res, b_pre, b_post, b_res,
               logits, r, H, workspace, workspace_bytes=None, stream=None, check=True):
    """Steps (1)-(3): logits, r and H from X_t and phi (see include/mhc.h)."""
    return _coeffs(load().mhc_coeffs, "mhc_coeffs", 2, 2, B, n, C, X_t, phi, alpha_pre, alpha_post,
                   alpha_res, b_pre, b_post, b_res, logits, r, H, workspace, workspace_bytes, stream, check)


def _coeffs_pre(fn, name, eb, B, n, C, X_t, phi, alpha_pre, alpha_post, alpha_res, b_pre, b_post,
                b_res, logits, r, H, F_pre, workspace, workspace_bytes, stream, check):
    z = _Sizes(B, n, C, eb, 2)
    pp, bp, bq, br, lg, rr, hh = _coeff_args(z, phi, b_pre, b_post, b_res, logits, r, H)
    wb = _ws_bytes(workspace, workspace_bytes)
    st = fn(int(B), int(n), int(C), _ptr(X_t, z.x, eb, "X_t"), pp, float(alpha_pre), float(alpha_post),
            float(alpha_res), bp, bq, br, lg, rr, hh, _ptr(F_pre, z.f, eb, "F_pre"),
            _ptr(workspace, wb, None, "workspace"), wb, _stream(stream))
    if check:
        _check(st, name)
    return st


def mhc_coeffs_pre_workspace_size(B, n, C):
    return int(load().mhc_coeffs_pre_workspace_size(int(B), int(n), int(C)))


def mhc_coeffs_pre_one_pass(B, n, C):
    return bool(load().mhc_coeffs_pre_one_pass(int(B), int(n), int(C)))


def mhc_coeffs_pre(B, n, C, X_t, phi, alpha_pre, alpha_post, alpha_res, b_pre, b_post, b_res,
                   logits, r, H, F_pre, workspace, workspace_bytes=None, stream=None, check=True):
    """Steps (1)-(3) and (4a) of one layer: logits, r, H and F_pre from X_t, in
    one pass where the shape allows (see include/mhc.h)."""
    return _coeffs_pre(load().mhc_coeffs_pre, "mhc_coeffs_pre", 2, B, n, C, X_t, phi, alpha_pre,
                       alpha_post, alpha_res, b_pre, b_post, b_res, logits, r, H, F_pre, workspace,
                       workspace_bytes, stream, check)


def mhc_coeffs_pre_check(B, n, C, workspace, fp8=False, workspace_bytes=None, stream=None):
    """Status of the last one-pass mhc_coeffs_pre(_fp8) call of shape (B, n, C)
    on `workspace`: MHC_OK, or MHC_ERR_INCOMPLETE if one of its waits gave up
    (synchronises the stream).  Returns the status, never raises on it."""
    wb = _ws_bytes(workspace, workspace_bytes)
    return int(load().mhc_coeffs_pre_check(int(B), int(n), int(C), 1 if fp8 else 0,
                                            _ptr(workspace, wb, None, "workspace"), wb, _stream(stream)))


def mhc_coeffs_pre_fp8_workspace_size(B, n, C):
    return int(load().mhc_coeffs_pre_fp8_workspace_size(int(B), int(n), int(C)))


def mhc_coeffs_pre_fp8_one_pass(B, n, C):
    return bool(load().mhc_coeffs_pre_fp8_one_pass(int(B), int(n), int(C)))


def mhc_coeffs_pre_fp8(B, n, C, X_t, phi, alpha_pre, alpha_post, alpha_res, b_pre, b_post, b_res,
                       logits, r, H, F_pre, workspace, workspace_bytes=None, stream=None, check=True):
    """mhc_coeffs_pre on an E4M3 X_t (see include/mhc.h)."""
    return _coeffs_pre(load().mhc_coeffs_pre_fp8, "mhc_coeffs_pre_fp8", 1, B, n, C, X_t, phi,
                       alpha_pre, alpha_post, alpha_res, b_pre, b_post, b_res, logits, r, H, F_pre,
                       workspace, workspace_bytes, stream, check)


def _pre(fn, name, eb, B, n, C, X_t, H, F_pre, stream, check):
    z = _Sizes(B, n, C, eb)
    st = fn(int(B), int(n), int(C), _ptr(X_t, z.x, eb, "X_t"), _ptr(H, z.coef, 4, "H"),
            _ptr(F_pre, z.f, eb, "F_pre"), _stream(stream))
    if check:
        _check(st, name)
    return st


def mhc_pre(B, n, C, X_t, H, F_pre, stream=None, check=True):
    """Step (4a): F_pre = sum_i H_pre[i] X_t[i] (see include/mhc.h)."""
    return _pre(load().mhc_pre, "mhc_pre", 2, B, n, C, X_t, H, F_pre, stream, check)


def _post_res(fn, name, eb, B, n, C, X_t, F_out, H, X_next, stream, check):
    z = _Sizes(B, n, C, eb)
    st = fn(int(B), int(n), int(C), _ptr(X_t, z.x, eb, "X_t"), _ptr(F_out, z.f, eb, "F_out"),
            _ptr(H, z.coef, 4, "H"), _ptr(X_next, z.x, eb, "X_next"), _stream(stream))
    if check:
        _check(st, name)
    return st


def mhc_post_res(B, n, C, X_t, F_out, H, X_next, stream=None, check=True):
    """Step (4b): X_next = H_res X_t + H_post^T F_out (see include/mhc.h)."""
    return _post_res(load().mhc_post_res, "mhc_post_res", 2, B, n, C, X_t, F_out, H, X_next, stream, check)


def _fused(fn, name, eb, pb, B, n, C, X_t, F_out, H, X_next, phi_next, alpha_pre, alpha_post,
           alpha_res, b_pre, b_post, b_res, logits_next, r_next, H_next, F_pre_next, workspace,
           workspace_bytes, stream, check, with_pre):
    z = _Sizes(B, n, C, eb, pb)
    pp, bp, bq, br, lg, rr, hh = _coeff_args(z, phi_next, b_pre, b_post, b_res, logits_next, r_next, H_next)
    wb = _ws_bytes(workspace, workspace_bytes)
    args = [int(B), int(n), int(C), _ptr(X_t, z.x, eb, "X_t"), _ptr(F_out, z.f, eb, "F_out"),
            _ptr(H, z.coef, 4, "H"), _ptr(X_next, z.x, eb, "X_next"), pp, float(alpha_pre),
            float(alpha_post), float(alpha_res), bp, bq, br, lg, rr, hh]
    if with_pre:
        args.append(_ptr(F_pre_next, z.f, eb, "F_pre_next"))
    args += [_ptr(workspace, wb, None, "workspace"), wb, _stream(stream)]
    st = fn(*args)
    if check:
        _check(st, name)
    return st


def mhc_post_res_coeffs_workspace_size(B, n, C):
    return int(load().mhc_post_res_coeffs_workspace_size(int(B), int(n), int(C)))


def mhc_post_res_coeffs(B, n, C, X_t, F_out, H, X_next, phi_next, alpha_pre, alpha_post,
                        alpha_res, b_pre, b_post, b_res, logits_next, r_next, H_next, workspace,
                        workspace_bytes=None, stream=None, check=True):
    """Step (4b) of this layer fused with steps (1)-(3) of the next (see include/mhc.h)."""
    return _fused(load().mhc_post_res_coeffs, "mhc_post_res_coeffs", 2, 2, B, n, C, X_t, F_out, H,
                  X_next, phi_next, alpha_pre, alpha_post, alpha_res, b_pre, b_post, b_res,
                  logits_next, r_next, H_next, None, workspace, workspace_bytes, stream, check, False)


def mhc_post_res_coeffs_pre_workspace_size(B, n, C):
    return int(load().mhc_post_res_coeffs_pre_workspace_size(int(B), int(n), int(C)))


def mhc_post_res_coeffs_pre_one_pass(B, n, C):
    return bool(load().mhc_post_res_coeffs_pre_one_pass(int(B), int(n), int(C)))


def mhc_post_res_coeffs_pre(B, n, C, X_t, F_out, H, X_next, phi_next, alpha_pre, alpha_post,
                            alpha_res, b_pre, b_post, b_res, logits_next, r_next, H_next,
                            F_pre_next, workspace, workspace_bytes=None, stream=None, check=True):
    """Step (4b) of this layer, then steps (1)-(3) and (4a) of the next, in
    one pass where the shape allows (see include/mhc.h)."""
    return _fused(load().mhc_post_res_coeffs_pre, "mhc_post_res_coeffs_pre", 2, 2, B, n, C, X_t,
                  F_out, H, X_next, phi_next, alpha_pre, alpha_post, alpha_res, b_pre, b_post, b_res,
                  logits_next, r_next, H_next, F_pre_next, workspace, workspace_bytes, stream, check,
                  True)


def mhc_post_res_coeffs_pre_noalloc(B, n, C, X_t, F_out, H, X_next, phi_next, alpha_pre,
                                    alpha_post, alpha_res, b_pre, b_post, b_res, logits_next,
                                    r_next, H_next, F_pre_next, stream=None, check=True):
    """mhc_post_res_coeffs_pre with its workspace in the library's own device
    array (no allocation; see include/mhc.h)."""
    z = _Sizes(B, n, C, 2, 2)
    pp, bp, bq, br, lg, rr, hh = _coeff_args(z, phi_next, b_pre, b_post, b_res, logits_next, r_next, H_next)
    st = load().mhc_post_res_coeffs_pre_noalloc(
        int(B), int(n), int(C), _ptr(X_t, z.x, 2, "X_t"), _ptr(F_out, z.f, 2, "F_out"),
        _ptr(H, z.coef, 4, "H"), _ptr(X_next, z.x, 2, "X_next"), pp, float(alpha_pre),
        float(alpha_post), float(alpha_res), bp, bq, br, lg, rr, hh,
        _ptr(F_pre_next, z.f, 2, "F_pre_next"), _stream(stream))
    if check:
        _check(st, "mhc_post_res_coeffs_pre_noalloc")
    return st


def mhc_post_res_coeffs_pre_check(B, n, C, workspace, fp8=False, workspace_bytes=None, stream=None):
    """Status of the last one-pass call of shape (B, n, C) on `workspace`:
    MHC_OK, or MHC_ERR_INCOMPLETE if one of its waits gave up (synchronises
    the stream; see include/mhc.h).  Returns the status, never raises on it."""
    wb = _ws_bytes(workspace, workspace_bytes)
    return int(load().mhc_post_res_coeffs_pre_check(int(B), int(n), int(C), 1 if fp8 else 0,
                                                     _ptr(workspace, wb, None, "workspace"), wb,
                                                     _stream(stream)))


def mhc_post_res_coeffs_pre_fp8_workspace_size(B, n, C):
    return int(load().mhc_post_res_coeffs_pre_fp8_workspace_size(int(B), int(n), int(C)))


def mhc_post_res_coeffs_pre_fp8_one_pass(B, n, C):
    return bool(load().mhc_post_res_coeffs_pre_fp8_one_pass(int(B), int(n), int(C)))


def mhc_post_res_coeffs_pre_fp8(B, n, C, X_t, F_out, H, X_next, phi_next, alpha_pre, alpha_post,
                                alpha_res, b_pre, b_post, b_res, logits_next, r_next, H_next,
                                F_pre_next, workspace, workspace_bytes=None, stream=None,
                                check=True):
    """mhc_post_res_coeffs_pre on the E4M3 residual stream (see include/mhc.h)."""
    return _fused(load().mhc_post_res_coeffs_pre_fp8, "mhc_post_res_coeffs_pre_fp8", 1, 2, B, n, C,
                  X_t, F_out, H, X_next, phi_next, alpha_pre, alpha_post, alpha_res, b_pre, b_post,
                  b_res, logits_next, r_next, H_next, F_pre_next, workspace, workspace_bytes, stream,
                  check, True)


# FP8 (E4M3) residual-stream variant: same arguments, with X_t, F_out, F_pre
# and X_next as E4M3 tensors (torch.float8_e4m3fn or raw uint8 codes).

def mhc_coeffs_fp8_workspace_size(B, n, C):
    return int(load().mhc_coeffs_fp8_workspace_size(int(B), int(n), int(C)))


def mhc_coeffs_fp8(B, n, C, X_t, phi, alpha_pre, alpha_post, alpha_res, b_pre, b_post, b_res,
                   logits, r, H, workspace, workspace_bytes=None, stream=None, check=True):
    """Steps (1)-(3) on an E4M3 X_t (see include/mhc.h)."""
    return _coeffs(load().mhc_coeffs_fp8, "mhc_coeffs_fp8", 1, 2, B, n, C, X_t, phi, alpha_pre,
                   alpha_post, alpha_res, b_pre, b_post, b_res, logits, r, H, workspace,
                   workspace_bytes, stream, check)


def mhc_pre_fp8(B, n, C, X_t, H, F_pre, stream=None, check=True):
    """Step (4a) on the E4M3 residual stream (see include/mhc.h)."""
    return _pre(load().mhc_pre_fp8, "mhc_pre_fp8", 1, B, n, C, X_t, H, F_pre, stream, check)


def mhc_post_res_fp8(B, n, C, X_t, F_out, H, X_next, stream=None, check=True):
    """Step (4b) on the E4M3 residual stream (see include/mhc.h)."""
    return _post_res(load().mhc_post_res_fp8, "mhc_post_res_fp8", 1, B, n, C, X_t, F_out, H, X_next,
                     stream, check)


def mhc_post_res_coeffs_fp8_workspace_size(B, n, C):
    return int(load().mhc_post_res_coeffs_fp8_workspace_size(int(B), int(n), int(C)))


def mhc_post_res_coeffs_fp8(B, n, C, X_t, F_out, H, X_next, phi_next, alpha_pre, alpha_post,
                            alpha_res, b_pre, b_post, b_res, logits_next, r_next, H_next,
                            workspace, workspace_bytes=None, stream=None, check=True):
    """mhc_post_res_coeffs on the E4M3 residual stream (see include/mhc.h)."""
    return _fused(load().mhc_post_res_coeffs_fp8, "mhc_post_res_coeffs_fp8", 1, 2, B, n, C, X_t, F_out,
                  H, X_next, phi_next, alpha_pre, alpha_post, alpha_res, b_pre, b_post, b_res,
                  logits_next, r_next, H_next, None, workspace, workspace_bytes, stream, check, False)


def mhc_coeffs_phi32_workspace_size(B, n, C):
    return int(load().mhc_coeffs_phi32_workspace_size(int(B), int(n), int(C)))


def mhc_coeffs_phi32(B, n, C, X_t, phi, alpha_pre, alpha_post, alpha_res, b_pre, b_post, b_res,
                     logits, r, H, workspace, workspace_bytes=None, stream=None, check=True):
    """Steps (1)-(3) with an fp32 phi (see include/mhc.h)."""
    return _coeffs(load().mhc_coeffs_phi32, "mhc_coeffs_phi32", 2, 4, B, n, C, X_t, phi, alpha_pre,
                   alpha_post, alpha_res, b_pre, b_post, b_res, logits, r, H, workspace,
                   workspace_bytes, stream, check)


def mhc_post_res_coeffs_phi32_workspace_size(B, n, C):
    return int(load().mhc_post_res_coeffs_phi32_workspace_size(int(B), int(n), int(C)))


def mhc_post_res_coeffs_phi32(B, n, C, X_t, F_out, H, X_next, phi_next, alpha_pre, alpha_post,
                              alpha_res, b_pre, b_post, b_res, logits_next, r_next, H_next,
                              workspace, workspace_bytes=None, stream=None, check=True):
    """mhc_post_res_coeffs with an fp32 phi_next (see include/mhc.h)."""
    return _fused(load().mhc_post_res_coeffs_phi32, "mhc_post_res_coeffs_phi32", 2, 4, B, n, C, X_t,
                  F_out, H, X_next, phi_next, alpha_pre, alpha_post, alpha_res, b_pre, b_post, b_res,
                  logits_next, r_next, H_next, None, workspace, workspace_bytes, stream, check, False)


def mhc_lazy_prenorm_gemm(M, N, K, A, W, C, rstd=None, eps=1e-5, stream=None, check=True):
    """C = rmsnorm(A) @ W^T (A bf16 [M, K], W bf16 [N, K], C bf16 [M, N]); rstd
    fp32 [M] if given (see include/mhc.h)."""
    M, N, K = int(M), int(N), int(K)
    m = max(M, 0)
    st = load().mhc_lazy_prenorm_gemm(M, N, K, _ptr(A, m * K * 2, 2, "A"), _ptr(W, max(N, 0) * K * 2, 2, "W"),
                                      float(eps), _ptr(C, m * max(N, 0) * 2, 2, "C"),
                                      _ptr(rstd, m * 4, 4, "rstd"), _stream(stream))
    if check:
        _check(st, "mhc_lazy_prenorm_gemm")
    return st


# Training: the stream's 8-bit checkpoint, the gradients of the calls above,
# the embeddings.  These calls launch on the current device, so they take
# tensors of that device only.

def _device():
    """The current device's index, -1 where no device is in use yet."""
    return torch._C._cuda_getDevice() if torch.cuda.is_initialized() else -1


def _dev_ptrs(dev, tensors, sizes):
    """_ptr of each tensor, with its (nbytes, esize, name), on the current
    device (index dev).  A tensor of another device is refused, not launched on
    (the kernels would run on another device than the tensor's).  Where a type
    stands for esize, a tensor of other numbers of its size is refused."""
    out = []
    for t, (nbytes, esize, name) in zip(tensors, sizes):
        if t is not None:
            # What nearly every tensor is, decided in a few attribute reads (a
            # raw address has none of them).
            try:
                usual = (t.get_device() == dev >= 0 and (t.dtype is esize or t.itemsize == esize or esize is None)
                         and t.nbytes >= nbytes and t.is_contiguous())
            except AttributeError:
                usual = False
            t = t.data_ptr() if usual else _dev_ptr(t, dev, nbytes, esize, name)
        out.append(t)
    return out


# What holds a type's values besides it and raw bytes (uint8).
_SAME = {torch.bfloat16: (torch.uint16, torch.int16), "codes": (torch.float8_e4m3fn,),
         "scales": (torch.float8_e8m0fnu,)}


def _dev_ptr(t, dev, nbytes, esize, name):
    if isinstance(esize, torch.dtype):
        if (isinstance(t, torch.Tensor) and t.numel() > 0 and t.itemsize == esize.itemsize
                and t.dtype not in (esize, torch.uint8, *_SAME.get(esize, ()), *_SAME.get(name, ()))):
            raise ValueError(f"{name}: {t.dtype}, the call takes {esize}")
        esize = esize.itemsize
    p = _ptr(t, nbytes, esize, name)
    if isinstance(t, torch.Tensor) and t.is_cuda and t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{dev}")
    return p


def _dev_stream(stream, dev):
    if stream is None and dev >= 0:
        return torch._C._cuda_getCurrentRawStream(dev)
    return _stream(stream)


def mhc_ckpt_scales_per_row(n, C):
    """Scale bytes a row of the checkpoint has: n * ceil(C / 32)."""
    return int(load().mhc_ckpt_scales_per_row(int(n), int(C)))


# What each call's tensors have to be, in their order: (bytes, element size,
# name).  They depend on the sizes alone and are worked out once for each.

def _x_sizes(B, n, C, ckpt):
    return (((B * n * C, 1, "codes"), (B * n * -(-C // 32), 1, "scales")) if ckpt else ((B * n * C * 2, 2, "X_t"),))


@functools.lru_cache(maxsize=256)
def _ckpt_sizes(B, n, C, pack):
    x, held = (_x_sizes(max(B, 0), n, C, ckpt) for ckpt in (False, True))
    return x + held if pack else held + x


@functools.lru_cache(maxsize=256)
def _post_res_bwd_sizes(B, n, C, ckpt):
    B, N = max(B, 0), n * n + 2 * n
    return _x_sizes(B, n, C, ckpt) + (
        (B * C * 2, 2, "F_out"), (B * N * 4, 4, "H"), (B * n * C * 2, 2, "dX_next"), (B * C * 2, 2, "dF_out"),
        (B * N * 4, 4, "dH"))


@functools.lru_cache(maxsize=256)
def _coeffs_pre_bwd_sizes(B, n, C, ckpt):
    B, N = max(B, 0), n * n + 2 * n
    some = 1 if B > 0 else 0  # at B == 0 only the parameters' gradients are touched
    return _x_sizes(B, n, C, ckpt) + (
        (some * n * C * N * 2, 2, "phi"), (some * n * 4, 4, "b_pre"), (some * n * 4, 4, "b_post"),
        (some * n * n * 4, 4, "b_res"), (B * N * 4, 4, "logits"), (B * 4, 4, "r"), (B * N * 4, 4, "H"),
        (B * n * C * 2, 2, "dX_next"), (B * N * 4, 4, "dH"), (B * C * 2, 2, "dF_pre"), (B * n * C * 2, 2, "dX_t"),
        (n * C * N * 4, 4, "dphi"), (12, 4, "dalpha"), (n * 4, 4, "db_pre"), (n * 4, 4, "db_post"),
        (n * n * 4, 4, "db_res"))


def mhc_ckpt_pack(B, n, C, X_t, codes, scales, stream=None, check=True):
    """The 8-bit checkpoint of X_t: codes (E4M3 or uint8 [B, n*C]) and scales
    (uint8 [B, mhc_ckpt_scales_per_row(n, C)]); see include/mhc.h."""
    B, n, C, dev = int(B), int(n), int(C), _device()
    st = load().mhc_ckpt_pack(B, n, C, *_dev_ptrs(dev, (X_t, codes, scales), _ckpt_sizes(B, n, C, True)),
                              _dev_stream(stream, dev))
    if check:
        _check(st, "mhc_ckpt_pack")
    return st


def mhc_ckpt_unpack(B, n, C, codes, scales, X_t, stream=None, check=True):
    """X_t in bf16 from its checkpoint (see include/mhc.h)."""
    B, n, C, dev = int(B), int(n), int(C), _device()
    st = load().mhc_ckpt_unpack(B, n, C, *_dev_ptrs(dev, (codes, scales, X_t), _ckpt_sizes(B, n, C, False)),
                                _dev_stream(stream, dev))
    if check:
        _check(st, "mhc_ckpt_unpack")
    return st


def _post_res_bwd(fn, name, held, B, n, C, F_out, H, dX_next, dF_out, dH, stream, check):
    B, n, C, dev = int(B), int(n), int(C), _device()
    st = fn(B, n, C, *_dev_ptrs(dev, (*held, F_out, H, dX_next, dF_out, dH),
                                _post_res_bwd_sizes(B, n, C, len(held) == 2)), _dev_stream(stream, dev))
    if check:
        _check(st, name)
    return st


def mhc_post_res_bwd(B, n, C, X_t, F_out, H, dX_next, dF_out, dH, stream=None, check=True):
    """Gradients of step (4b) with respect to F_out and H (see include/mhc.h)."""
    return _post_res_bwd(load().mhc_post_res_bwd, "mhc_post_res_bwd", (X_t,), B, n, C, F_out, H, dX_next, dF_out, dH,
                         stream, check)


def mhc_post_res_bwd_ckpt(B, n, C, codes, scales, F_out, H, dX_next, dF_out, dH, stream=None, check=True):
    """mhc_post_res_bwd with X_t as its checkpoint (see include/mhc.h)."""
    return _post_res_bwd(load().mhc_post_res_bwd_ckpt, "mhc_post_res_bwd_ckpt", (codes, scales), B, n, C, F_out, H,
                         dX_next, dF_out, dH, stream, check)


def mhc_coeffs_pre_bwd_workspace_size(B, n, C):
    return int(load().mhc_coeffs_pre_bwd_workspace_size(int(B), int(n), int(C)))


def _coeffs_pre_bwd(fn, name, held, B, n, C, alphas, tensors, workspace, workspace_bytes, stream, check):
    B, n, C, dev = int(B), int(n), int(C), _device()
    p = _dev_ptrs(dev, (*held, *tensors), _coeffs_pre_bwd_sizes(B, n, C, len(held) == 2))
    wb = _ws_bytes(workspace, workspace_bytes)
    p += _dev_ptrs(dev, (workspace,), ((wb, None, "workspace"),))
    k = len(held) + 1  # the alphas follow phi
    st = fn(B, n, C, *p[:k], *alphas, *p[k:], wb, _dev_stream(stream, dev))
    if check:
        _check(st, name)
    return st


def mhc_coeffs_pre_bwd(B, n, C, X_t, phi, alpha_pre, alpha_post, alpha_res, b_pre, b_post, b_res, logits, r, H,
                       dX_next, dH, dF_pre, dX_t, dphi, dalpha, db_pre, db_post, db_res, workspace,
                       workspace_bytes=None, stream=None, check=True):
    """Gradients of steps (1)-(4a) and of X_t through the apply (see include/mhc.h)."""
    return _coeffs_pre_bwd(load().mhc_coeffs_pre_bwd, "mhc_coeffs_pre_bwd", (X_t,), B, n, C,
                           (float(alpha_pre), float(alpha_post), float(alpha_res)),
                           (phi, b_pre, b_post, b_res, logits, r, H, dX_next, dH, dF_pre, dX_t, dphi, dalpha, db_pre,
                            db_post, db_res), workspace, workspace_bytes, stream, check)


def mhc_coeffs_pre_bwd_ckpt(B, n, C, codes, scales, phi, alpha_pre, alpha_post, alpha_res, b_pre, b_post, b_res,
                            logits, r, H, dX_next, dH, dF_pre, dX_t, dphi, dalpha, db_pre, db_post, db_res,
                            workspace, workspace_bytes=None, stream=None, check=True):
    """mhc_coeffs_pre_bwd with X_t as its checkpoint (see include/mhc.h)."""
    return _coeffs_pre_bwd(load().mhc_coeffs_pre_bwd_ckpt, "mhc_coeffs_pre_bwd_ckpt", (codes, scales), B, n, C,
                           (float(alpha_pre), float(alpha_post), float(alpha_res)),
                           (phi, b_pre, b_post, b_res, logits, r, H, dX_next, dH, dF_pre, dX_t, dphi, dalpha, db_pre,
                            db_post, db_res), workspace, workspace_bytes, stream, check)


def mhc_embed(B, n, C, V, tokens, table, scale, X_0, stream=None, check=True):
    """X_0: the scaled embeddings of the tokens (int64) in every stream (see include/mhc.h)."""
    B, n, C, V, dev = int(B), int(n), int(C), int(V), _device()
    rows = max(B, 0)
    tokens, table, X_0 = _dev_ptrs(dev, (tokens, table, X_0), (
        (rows * 8, 8, "tokens"), (max(V, 0) * C * 2 if B > 0 else 0, 2, "table"), (rows * n * C * 2, 2, "X_0")))
    st = load().mhc_embed(B, n, C, V, tokens, table, float(scale), X_0, _dev_stream(stream, dev))
    if check:
        _check(st, "mhc_embed")
    return st


def mhc_embed_bwd_workspace_size(B, n, C, V):
    return int(load().mhc_embed_bwd_workspace_size(int(B), int(n), int(C), int(V)))


def mhc_embed_bwd(B, n, C, V, tokens, dX_0, scale, dtable, workspace, accumulate=False, workspace_bytes=None,
                  stream=None, check=True):
    """The embedding table's gradient (fp32 [V, C]), overwritten or, with
    accumulate, added to (see include/mhc.h)."""
    B, n, C, V, dev = int(B), int(n), int(C), int(V), _device()
    rows, wb = max(B, 0), _ws_bytes(workspace, workspace_bytes)
    tokens, dX_0, dtable, workspace = _dev_ptrs(dev, (tokens, dX_0, dtable, workspace), (
        (rows * 8, 8, "tokens"), (rows * n * C * 2, 2, "dX_0"), (max(V, 0) * C * 4, 4, "dtable"),
        (wb, None, "workspace")))
    st = load().mhc_embed_bwd(B, n, C, V, tokens, dX_0, float(scale), int(bool(accumulate)), dtable, workspace, wb,
                              _dev_stream(stream, dev))
    if check:
        _check(st, "mhc_embed_bwd")
    return st


# Around a layer of experts: norm, choice of experts, rows into the experts'
# order and back.  On the current device, as the training calls; tensors are of
# the types that include/mhc.h names (the gather copies any of their size).

_BF16, _FP32, _INT32, _BYTE = torch.bfloat16, torch.float32, torch.int32, torch.uint8


@functools.lru_cache(maxsize=256)
def _rmsnorm_sizes(B, C):
    B = max(B, 0)
    some = 4 * C if B > 0 else 0  # at B == 0 nothing is touched
    return ((B * C * 2, _BF16, "x"), (B * C * 2, _BF16, "shortcut"), (some, _FP32, "weight"), (B * C * 2, _BF16, "sum"),
            (B * C * 2, _BF16, "y"), (B * C, _BYTE, "codes"), (B * -(-C // 32), _BYTE, "scales"),
            (B * 4, _FP32, "rstd"))


def mhc_rmsnorm(B, C, x, weight, y=None, codes=None, scales=None, shortcut=None, sum=None, rstd=None, eps=1e-5,
                stream=None, check=True):
    """Root-mean-square norm of x (plus the shortcut, kept in sum), times weight
    (fp32 [C] or None): y in bf16, or codes and scales in 8 bits, or all three
    (see include/mhc.h)."""
    B, C, dev = int(B), int(C), _device()
    x, shortcut, weight, *out = _dev_ptrs(dev, (x, shortcut, weight, sum, y, codes, scales, rstd), _rmsnorm_sizes(B, C))
    st = load().mhc_rmsnorm(B, C, x, shortcut, weight, float(eps), *out, _dev_stream(stream, dev))
    if check:
        _check(st, "mhc_rmsnorm")
    return st


def mhc_rmsnorm_bwd_workspace_size(B, C):
    return int(load().mhc_rmsnorm_bwd_workspace_size(int(B), int(C)))


@functools.lru_cache(maxsize=256)
def _rmsnorm_bwd_sizes(B, C):
    B = max(B, 0)
    some = 4 * C if B > 0 else 0
    return ((B * C * 2, _BF16, "sum"), (some, _FP32, "weight"), (B * 4, _FP32, "rstd"), (B * C * 2, _BF16, "dy"),
            (B * C * 2, _BF16, "dsum"), (B * C * 2, _BF16, "dx"), (4 * C, _FP32, "dweight"))


def mhc_rmsnorm_bwd(B, C, sum, weight, rstd, dy, dx, dweight=None, workspace=None, dsum=None, workspace_bytes=None,
                    stream=None, check=True):
    """Gradients of mhc_rmsnorm: dx (with dsum, what arrives at the sum on its
    other path) and, with a workspace, dweight (see include/mhc.h)."""
    B, C, dev = int(B), int(C), _device()
    p = _dev_ptrs(dev, (sum, weight, rstd, dy, dsum, dx, dweight), _rmsnorm_bwd_sizes(B, C))
    wb = _ws_bytes(workspace, workspace_bytes)
    p += _dev_ptrs(dev, (workspace,), ((wb, None, "workspace"),))
    st = load().mhc_rmsnorm_bwd(B, C, *p, wb, _dev_stream(stream, dev))
    if check:
        _check(st, "mhc_rmsnorm_bwd")
    return st


def _logits_type(logits, softmax, renorm, bf16):
    """Type and flags: the logits' type is the tensor's (bf16 says it for raw addresses)."""
    if bf16 is None:
        bf16 = isinstance(logits, torch.Tensor) and logits.dtype == torch.bfloat16
    if isinstance(logits, torch.Tensor) and logits.dtype not in (torch.bfloat16, torch.float32, torch.uint8):
        raise ValueError(f"logits: {logits.dtype}, the call takes float32 or bfloat16")
    return (_BF16 if bf16 else _FP32,
            (MHC_ROUTE_SOFTMAX if softmax else 0) | (MHC_ROUTE_RENORM if renorm else 0) | (MHC_ROUTE_BF16 if bf16 else 0))


def mhc_route(B, E, k, logits, ids, weights, bias=None, groups=1, top_groups=1, softmax=False, renorm=True, scale=1.0,
              bf16=None, stream=None, check=True):
    """The k experts of each row of logits (fp32 or bf16 [B, E]): ids (int32)
    and weights (fp32), both [B, k] (see include/mhc.h)."""
    B, E, k, dev = int(B), int(E), int(k), _device()
    kind, flags = _logits_type(logits, softmax, renorm, bf16)
    rows, one = max(B, 0), kind.itemsize
    logits, bias, ids, weights = _dev_ptrs(dev, (logits, bias, ids, weights), (
        (rows * E * one, kind, "logits"), (4 * E if rows else 0, _FP32, "bias"), (rows * k * 4, _INT32, "ids"),
        (rows * k * 4, _FP32, "weights")))
    st = load().mhc_route(B, E, k, int(groups), int(top_groups), flags, float(scale), logits, bias, ids, weights,
                          _dev_stream(stream, dev))
    if check:
        _check(st, "mhc_route")
    return st


def mhc_route_bwd(B, E, k, logits, ids, dweights, dlogits, softmax=False, renorm=True, scale=1.0, bf16=None,
                  stream=None, check=True):
    """Gradient of mhc_route's weights with respect to the logits, in their
    type (see include/mhc.h)."""
    B, E, k, dev = int(B), int(E), int(k), _device()
    kind, flags = _logits_type(logits, softmax, renorm, bf16)
    rows, one = max(B, 0), kind.itemsize
    logits, ids, dweights, dlogits = _dev_ptrs(dev, (logits, ids, dweights, dlogits), (
        (rows * E * one, kind, "logits"), (rows * k * 4, _INT32, "ids"), (rows * k * 4, _FP32, "dweights"),
        (rows * E * one, kind, "dlogits")))
    st = load().mhc_route_bwd(B, E, k, flags, float(scale), logits, ids, dweights, dlogits, _dev_stream(stream, dev))
    if check:
        _check(st, "mhc_route_bwd")
    return st


def mhc_experts_order_workspace_size(B, k, E):
    return int(load().mhc_experts_order_workspace_size(int(B), int(k), int(E)))


def mhc_experts_order(B, k, E, ids, slots, offsets, workspace, workspace_bytes=None, stream=None, check=True):
    """Places (int32 [B, k]) of the pairs (row, ids[row, j]) in the order of
    their experts, and the experts' first places (int32 [E + 1]; see
    include/mhc.h)."""
    B, k, E, dev = int(B), int(k), int(E), _device()
    rows, wb = max(B, 0), _ws_bytes(workspace, workspace_bytes)
    ids, slots, offsets, workspace = _dev_ptrs(dev, (ids, slots, offsets, workspace), (
        (rows * k * 4, _INT32, "ids"), (rows * k * 4, _INT32, "slots"), ((max(E, 0) + 1) * 4, _INT32, "offsets"),
        (wb, None, "workspace")))
    st = load().mhc_experts_order(B, k, E, ids, slots, offsets, workspace, wb, _dev_stream(stream, dev))
    if check:
        _check(st, "mhc_experts_order")
    return st


# Tensors of B rows and of their B * k pairs.

@functools.lru_cache(maxsize=256)
def _gather_sizes(B, k, C, ckpt):
    B = max(B, 0)
    if not ckpt:
        return ((B * C * 2, 2, "X"), (B * k * 4, _INT32, "slots"), (B * k * C * 2, 2, "rows"))
    blocks = -(-C // 32)
    return ((B * C, 1, "codes"), (B * blocks, 1, "scales"), (B * k * 4, _INT32, "slots"),
            (B * k * C, 1, "row_codes"), (B * k * blocks, 1, "row_scales"))


@functools.lru_cache(maxsize=256)
def _combine_sizes(B, k, C, bwd):
    B = max(B, 0)
    rows, pairs, row = B * k * C * 2, B * k * 4, B * C * 2
    sizes = ((rows, _BF16, "Y"), (pairs, _INT32, "slots"), (pairs, _FP32, "weights"))
    if bwd:
        return sizes + ((row, _BF16, "dF_out"), (rows, _BF16, "dY"), (pairs, _FP32, "dweights"))
    return sizes + ((row, _BF16, "shared"), (row, _BF16, "F_out"))


def mhc_experts_gather(B, k, C, X, slots, rows, stream=None, check=True):
    """rows[slots[b, j]] = X[b] (bf16; see include/mhc.h)."""
    B, k, C, dev = int(B), int(k), int(C), _device()
    st = load().mhc_experts_gather(B, k, C, *_dev_ptrs(dev, (X, slots, rows), _gather_sizes(B, k, C, False)),
                                   _dev_stream(stream, dev))
    if check:
        _check(st, "mhc_experts_gather")
    return st


def mhc_experts_gather_ckpt(B, k, C, codes, scales, slots, row_codes, row_scales, stream=None, check=True):
    """mhc_experts_gather of rows held in 8 bits, codes and scales (see include/mhc.h)."""
    B, k, C, dev = int(B), int(k), int(C), _device()
    p = _dev_ptrs(dev, (codes, scales, slots, row_codes, row_scales), _gather_sizes(B, k, C, True))
    st = load().mhc_experts_gather_ckpt(B, k, C, *p, _dev_stream(stream, dev))
    if check:
        _check(st, "mhc_experts_gather_ckpt")
    return st


def mhc_experts_combine(B, k, C, Y, slots, weights, F_out, shared=None, stream=None, check=True):
    """F_out[b] = shared[b] + sum_j weights[b, j] Y[slots[b, j]]; weights None:
    1, the gradient of mhc_experts_gather (see include/mhc.h)."""
    B, k, C, dev = int(B), int(k), int(C), _device()
    p = _dev_ptrs(dev, (Y, slots, weights, shared, F_out), _combine_sizes(B, k, C, False))
    st = load().mhc_experts_combine(B, k, C, *p, _dev_stream(stream, dev))
    if check:
        _check(st, "mhc_experts_combine")
    return st


def mhc_experts_combine_bwd(B, k, C, Y, slots, weights, dF_out, dY, dweights, stream=None, check=True):
    """Gradients of mhc_experts_combine with respect to Y and the weights (see include/mhc.h)."""
    B, k, C, dev = int(B), int(k), int(C), _device()
    p = _dev_ptrs(dev, (Y, slots, weights, dF_out, dY, dweights), _combine_sizes(B, k, C, True))
    st = load().mhc_experts_combine_bwd(B, k, C, *p, _dev_stream(stream, dev))
    if check:
        _check(st, "mhc_experts_combine_bwd")
    return st


def alloc_outputs(B, n, C, device="cuda"):
    """Caller-side buffers for one forward of shape (B, n, C): logits, r, H,
    F_pre, X_next and the coefficient workspace (uint8, 16-byte aligned)."""
    N = n * n + 2 * n
    ws_bytes = mhc_coeffs_workspace_size(B, n, C)
    return {
        "logits": torch.empty(B, N, dtype=torch.float32, device=device),
        "r": torch.empty(B, dtype=torch.float32, device=device),
        "H": torch.empty(B, N, dtype=torch.float32, device=device),
        "F_pre": torch.empty(B, C, dtype=torch.bfloat16, device=device),
        "X_next": torch.empty(B, n * C, dtype=torch.bfloat16, device=device),
        "workspace": torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=device),
    }
