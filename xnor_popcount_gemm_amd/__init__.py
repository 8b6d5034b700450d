"""Python binding of libbnn.so, the MI355X (gfx950) binary-network hot path.

Argument marshalling only: every step of the path (sign + bit-pack,
XNOR-popcount GEMM/GEMV, alpha / residual / folded-BatchNorm epilogues, the FP
first and last layers) runs in the HIP kernels behind the C ABI declared in
``include/bnn.h``.  PyTorch provides device memory and the current stream;
there is no CPU or PyTorch fallback: if the library is missing, importing the
binding's calls raises.

The functions keep the C names without the ``bnn_`` prefix.  Tensors passed
in must live on a HIP device; outputs are allocated here (or given with
``out=`` style arguments) with the layouts the C ABI documents:
packed matrices are uint32 ``[rows, ld]`` stored as ``torch.int32`` (same
bits), ``ld`` a multiple of 4, bit 0 = +1, bit 1 = -1, pad bits and words 0.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

__all__ = [
    "BnnError", "lib", "packed_words", "padded_ld", "pack_weights", "pack_activations",
    "xnor_gemm", "xnor_gemm_mfma", "linear_fused", "fold_bn_thresholds", "dense_f32_sign_pack",
    "dense_binact_f32", "EPI_DOT_I32", "EPI_SCALE_F32", "EPI_RESIDUAL_F32",
    "EPI_THRESH_PACK", "EPI_ALPHA_TENSOR", "EPI_BIAS_F32", "LIB_PATH",
    "weight_scale_tensor", "weight_scale_tensor_noalloc", "NOALLOC_MAX_ROWS", "quantize_act_i8", "pack_act_i8", "bwn_i8_linear", "MAX_K_I8", "bwn_f16_gemv", "MAX_K_F16",
    "W_TERNARY", "pack_weights_ternary", "EPI_SIGN_PACK", "pack_activations_rsign", "conv3x3_fused",
    "KVCache", "qk_norm_rope", "rope_turns", "tree_mask", "tree_attention", "tree_attention_workspace",
    "cache_score_add", "cache_evict", "cache_evict_workspace",
    "block_norm", "expert_route", "expert_route_workspace", "ExpertWeights", "expert_linear", "MAX_NORM_D", "MAX_EXPERTS",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libbnn.so")

EPI_DOT_I32 = 1
EPI_SCALE_F32 = 2
EPI_RESIDUAL_F32 = 4
EPI_THRESH_PACK = 8
EPI_ALPHA_TENSOR = 16
EPI_BIAS_F32 = 32
W_TERNARY = 64
EPI_SIGN_PACK = 128
MAX_K_I8 = 1 << 17
MAX_K_F16 = 16384
NOALLOC_MAX_ROWS = 1 << 16

_STATUS = {
    0: "BNN_OK", 1: "BNN_ERR_NULL", 2: "BNN_ERR_SHAPE", 3: "BNN_ERR_LD",
    4: "BNN_ERR_ALIGN", 5: "BNN_ERR_UNSUPPORTED", 6: "BNN_ERR_HIP",
}


class BnnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {_STATUS.get(status, status)}")


class _ConvGeom(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("B", "H", "W", "C", "R", "S", "stride", "pad")]


class _FusedArgs(ctypes.Structure):
    _fields_ = [
        ("Xp", ctypes.c_void_p), ("ldXp", ctypes.c_int64),
        ("Wp", ctypes.c_void_p), ("ldWp", ctypes.c_int64),
        ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
        ("epilogue", ctypes.c_uint32),
        ("D", ctypes.c_void_p), ("ldD", ctypes.c_int64),
        ("alpha", ctypes.c_void_p),
        ("Y", ctypes.c_void_p), ("ldY", ctypes.c_int64),
        ("R", ctypes.c_void_p), ("ldR", ctypes.c_int64),
        ("tau", ctypes.c_void_p), ("dir", ctypes.c_void_p),
        ("Op", ctypes.c_void_p), ("ldOp", ctypes.c_int64),
        ("bias", ctypes.c_void_p),
        ("Zp", ctypes.c_void_p), ("nnz", ctypes.c_void_p),
        ("beta", ctypes.c_void_p),
    ]


class _I8Args(ctypes.Structure):
    _fields_ = [
        ("Xb", ctypes.c_void_p), ("ldXb", ctypes.c_int64),
        ("xsum", ctypes.c_void_p),
        ("Xq", ctypes.c_void_p), ("ldXq", ctypes.c_int64),
        ("xscale", ctypes.c_void_p),
        ("Wp", ctypes.c_void_p), ("ldWp", ctypes.c_int64),
        ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
        ("epilogue", ctypes.c_uint32),
        ("D", ctypes.c_void_p), ("ldD", ctypes.c_int64),
        ("alpha", ctypes.c_void_p),
        ("Y", ctypes.c_void_p), ("ldY", ctypes.c_int64),
        ("Zp", ctypes.c_void_p),
    ]


class _KvCache(ctypes.Structure):
    _fields_ = [
        ("K", ctypes.c_void_p), ("k_page", ctypes.c_int64), ("k_slot", ctypes.c_int64), ("k_head", ctypes.c_int64),
        ("V", ctypes.c_void_p), ("v_page", ctypes.c_int64), ("v_slot", ctypes.c_int64), ("v_head", ctypes.c_int64),
        ("table", ctypes.c_void_p), ("ld_table", ctypes.c_int64),
        ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int64),
        ("kv_heads", ctypes.c_int64), ("dim", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
    ]


class _KvBatch(ctypes.Structure):
    _fields_ = [
        ("indptr", ctypes.c_void_p), ("ctx", ctypes.c_void_p),
        ("B", ctypes.c_int64), ("rows", ctypes.c_int64),
        ("max_nodes", ctypes.c_int64), ("max_ctx", ctypes.c_int64),
    ]


class _RopeArgs(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("q_row", ctypes.c_int64), ("q_head", ctypes.c_int64),
        ("k", ctypes.c_void_p), ("k_row", ctypes.c_int64), ("k_head", ctypes.c_int64),
        ("v", ctypes.c_void_p), ("v_row", ctypes.c_int64), ("v_head", ctypes.c_int64),
        ("src_dtype", ctypes.c_int32),
        ("heads", ctypes.c_int64),
        ("q_out", ctypes.c_void_p), ("qo_row", ctypes.c_int64), ("qo_head", ctypes.c_int64),
        ("positions", ctypes.c_void_p),
        ("turns", ctypes.c_void_p), ("max_pos", ctypes.c_int64), ("rot", ctypes.c_int64),
        ("interleaved", ctypes.c_int32),
        ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
        ("eps", ctypes.c_float),
        ("pos", ctypes.c_void_p), ("score", ctypes.c_void_p),
        ("ld_slots", ctypes.c_int64),
    ]


class _AttnArgs(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("q_row", ctypes.c_int64), ("q_head", ctypes.c_int64),
        ("heads", ctypes.c_int64),
        ("mask", ctypes.c_void_p), ("ld_mask", ctypes.c_int64),
        ("scale", ctypes.c_float),
        ("out", ctypes.c_void_p), ("o_row", ctypes.c_int64), ("o_head", ctypes.c_int64),
        ("out_dtype", ctypes.c_int32),
        ("lse", ctypes.c_void_p), ("ld_lse", ctypes.c_int64),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64),
    ]


class _ScoreArgs(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p), ("q_row", ctypes.c_int64), ("q_head", ctypes.c_int64),
        ("heads", ctypes.c_int64),
        ("lse", ctypes.c_void_p), ("ld_lse", ctypes.c_int64),
        ("mask", ctypes.c_void_p), ("ld_mask", ctypes.c_int64),
        ("accept", ctypes.c_void_p), ("ld_accept", ctypes.c_int64),
        ("scale", ctypes.c_float),
        ("score_in", ctypes.c_void_p), ("score_out", ctypes.c_void_p),
        ("ld_slots", ctypes.c_int64),
    ]


class _EvictArgs(ctypes.Structure):
    _fields_ = [
        ("accept", ctypes.c_void_p), ("ld_accept", ctypes.c_int64),
        ("budget", ctypes.c_int64), ("recent", ctypes.c_int64),
        ("pos_in", ctypes.c_void_p), ("pos_out", ctypes.c_void_p),
        ("score_in", ctypes.c_void_p), ("score_out", ctypes.c_void_p),
        ("ld_slots", ctypes.c_int64),
        ("ctx_out", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64),
    ]


class _NormArgs(ctypes.Structure):
    _fields_ = [
        ("M", ctypes.c_int64), ("D", ctypes.c_int64), ("used", ctypes.c_void_p),
        ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("x_dtype", ctypes.c_int32),
        ("branch", ctypes.c_void_p), ("ldb", ctypes.c_int64), ("b_dtype", ctypes.c_int32), ("b_rows", ctypes.c_int64),
        ("place", ctypes.c_void_p), ("weight", ctypes.c_void_p), ("parts", ctypes.c_int64),
        ("post", ctypes.c_int32), ("post_weight", ctypes.c_void_p), ("post_bias", ctypes.c_void_p),
        ("gate", ctypes.c_void_p), ("ld_gate", ctypes.c_int64),
        ("x_scale", ctypes.c_float), ("branch_scale", ctypes.c_float),
        ("pre", ctypes.c_int32), ("pre_weight", ctypes.c_void_p), ("pre_bias", ctypes.c_void_p),
        ("eps", ctypes.c_float),
        ("x_out", ctypes.c_void_p), ("ldxo", ctypes.c_int64),
        ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64), ("y_dtype", ctypes.c_int32),
        ("Xq", ctypes.c_void_p), ("ldXq", ctypes.c_int64), ("Xb", ctypes.c_void_p), ("ldXb", ctypes.c_int64),
        ("xsum", ctypes.c_void_p), ("xscale", ctypes.c_void_p),
    ]


class _RouteArgs(ctypes.Structure):
    _fields_ = [
        ("logits", ctypes.c_void_p), ("ld", ctypes.c_int64), ("dtype", ctypes.c_int32),
        ("rows", ctypes.c_int64), ("experts", ctypes.c_int64), ("top", ctypes.c_int64),
        ("used", ctypes.c_void_p), ("score", ctypes.c_int32), ("bias", ctypes.c_void_p),
        ("renorm", ctypes.c_int32), ("scale", ctypes.c_float),
        ("expert", ctypes.c_void_p), ("weight", ctypes.c_void_p), ("offsets", ctypes.c_void_p),
        ("order", ctypes.c_void_p), ("place", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64),
    ]


class _ExpertMatrix(ctypes.Structure):
    _fields_ = [
        ("W", ctypes.c_void_p), ("alpha", ctypes.c_void_p), ("ld_alpha", ctypes.c_int64),
        ("bias", ctypes.c_void_p), ("ld_bias", ctypes.c_int64),
    ]


class _ExpertArgs(ctypes.Structure):
    _fields_ = [
        ("Xq", ctypes.c_void_p), ("ldXq", ctypes.c_int64), ("xscale", ctypes.c_void_p), ("rows", ctypes.c_int64),
        ("order", ctypes.c_void_p), ("per_row", ctypes.c_int64), ("offsets", ctypes.c_void_p),
        ("experts", ctypes.c_int64), ("positions", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
        ("ternary", ctypes.c_int32), ("main", _ExpertMatrix), ("up", _ExpertMatrix), ("act", ctypes.c_int32),
        ("residual", ctypes.c_void_p), ("ldr", ctypes.c_int64),
        ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64), ("y_dtype", ctypes.c_int32),
    ]


_lib = None
_i64 = ctypes.c_int64
_vp = ctypes.c_void_p


def lib() -> ctypes.CDLL:
    """Load libbnn.so (built in-tree by ``xnor_popcount_gemm_amd.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -m xnor_popcount_gemm_amd.build` "
                "(there is no fallback path)")
        L = ctypes.CDLL(LIB_PATH)
        L.bnn_packed_words.argtypes = [_i64]
        L.bnn_packed_words.restype = _i64
        L.bnn_status_string.argtypes = [ctypes.c_int]
        L.bnn_status_string.restype = ctypes.c_char_p
        sigs = {
            "bnn_pack_weights": [_vp, _i64, _i64, _i64, _vp, _i64, _vp, _vp],
            "bnn_pack_activations": [_vp, _i64, _i64, _i64, _vp, _vp, _i64, _vp],
            "bnn_xnor_gemm": [_vp, _i64, _vp, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _vp, _i64, _vp],
            "bnn_xnor_gemm_mfma": [_vp, _i64, _vp, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _vp, _i64, _vp],
            "bnn_linear_fused": [ctypes.POINTER(_FusedArgs), _vp],
            "bnn_fold_bn_thresholds_host": [_vp, _vp, _vp, _vp, ctypes.c_float, _vp, _i64, _vp, _vp],
            "bnn_dense_f32_sign_pack": [_vp, _i64, _vp, _i64, _i64, _i64, _i64, _vp, _i64, _vp],
            "bnn_dense_binact_f32": [_vp, _i64, _vp, _i64, _i64, _i64, _i64, _vp, _i64, _vp],
            "bnn_weight_scale_tensor": [_vp, _i64, _i64, _i64, _vp, _vp, _vp],
            "bnn_weight_scale_tensor_noalloc": [_vp, _i64, _i64, _i64, _vp, _vp],
            "bnn_quantize_act_i8": [_vp, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp],
            "bnn_pack_act_i8": [_vp, _i64, _i64, _i64, _vp, _i64, _vp, _vp],
            "bnn_bwn_i8_linear": [ctypes.POINTER(_I8Args), _vp],
            "bnn_bwn_f16_gemv": [_vp, _i64, _vp, _i64, _i64, _i64, _i64, ctypes.c_uint32, _vp, _vp, _i64, _vp],
            "bnn_pack_weights_ternary": [_vp, _i64, _i64, _i64, _vp, ctypes.c_float, _vp, _vp, _i64, _vp, _vp],
            "bnn_pack_activations_rsign": [_vp, _i64, _i64, _i64, _vp, _vp, _i64, _vp],
            "bnn_conv3x3_fused": [ctypes.POINTER(_FusedArgs), ctypes.POINTER(_ConvGeom), _vp],
            "bnn_qk_norm_rope": [_vp, _vp, _vp, _vp],
            "bnn_rope_turns_host": [_i64, _i64, ctypes.c_double, ctypes.c_int32, ctypes.c_double, ctypes.c_double,
                                    ctypes.c_double, ctypes.c_double, _vp],
            "bnn_tree_mask_host": [_vp, _i64, _vp, _i64],
            "bnn_tree_attention": [_vp, _vp, _vp, _vp],
            "bnn_cache_score_add": [_vp, _vp, _vp, _vp],
            "bnn_cache_evict": [_vp, _vp, _vp, _vp],
            "bnn_block_norm": [_vp, _vp],
            "bnn_expert_route": [_vp, _vp],
            "bnn_expert_pack": [_vp, _vp, _i64, _i64, _i64, _i64, _i64, _vp, _i64, _vp],
            "bnn_expert_linear": [_vp, _vp],
        }
        for name, args in sigs.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        L.bnn_tree_attention_workspace.argtypes = [_vp, _vp, _i64]
        L.bnn_tree_attention_workspace.restype = _i64
        L.bnn_cache_evict_workspace.argtypes = [_vp, _i64]
        L.bnn_cache_evict_workspace.restype = _i64
        L.bnn_expert_route_workspace.argtypes = [_i64, _i64, _i64]
        L.bnn_expert_route_workspace.restype = _i64
        L.bnn_expert_pack_bytes.argtypes = [_i64, _i64, _i64, ctypes.c_int32]
        L.bnn_expert_pack_bytes.restype = _i64
        _lib = L
    return _lib


def _check(status: int, where: str) -> None:
    if status != 0:
        raise BnnError(status, where)


def packed_words(K: int) -> int:
    """ceil(K / 32)."""
    return int(lib().bnn_packed_words(int(K)))


def padded_ld(K: int) -> int:
    """Smallest valid leading dimension of a packed matrix: ceil(K/32) rounded
    up to a multiple of 4 words (16-byte rows)."""
    kw = (int(K) + 31) // 32
    return (kw + 3) // 4 * 4


def _dev(t: torch.Tensor, dtype, name: str) -> torch.Tensor:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a HIP device (got {t.device})")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    return t


def _ld(t: torch.Tensor) -> int:
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError("expected a 2-D tensor with unit column stride")
    return t.stride(0)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _packed_empty(rows: int, K: int, device, ld: int | None = None) -> torch.Tensor:
    ld = padded_ld(K) if ld is None else ld
    return torch.empty((rows, ld), dtype=torch.int32, device=device)


def pack_weights(W: torch.Tensor, *, alpha: bool = True, out: torch.Tensor | None = None,
                 alpha_out: torch.Tensor | None = None):
    """Sign + bit-pack fp32 weights [N, K]; returns (Wp [N, ld], alpha [N] or None)."""
    _dev(W, torch.float32, "W")
    N, K = W.shape
    Wp = _packed_empty(N, K, W.device) if out is None else out
    a = None
    if alpha:
        a = torch.empty(N, dtype=torch.float32, device=W.device) if alpha_out is None else alpha_out
    _check(lib().bnn_pack_weights(_ptr(W), N, K, _ld(W), _ptr(Wp), _ld(Wp), _ptr(a),
                                  _stream(W.device)), "bnn_pack_weights")
    return Wp, a


def pack_activations(X: torch.Tensor, *, conv3x3: bool = False, out: torch.Tensor | None = None):
    """Sign + bit-pack activations.

    Dense: X fp32 [M, K] -> packed [M, ld].  ``conv3x3=True``: X is an NHWC
    fp32 image [B, H, W, C] (contiguous) and the result is its packed 3x3 /
    stride 1 / pad 1 im2col matrix [B*H*W, ld] with K = 9*C, pad pixels +1.
    """
    _dev(X, torch.float32, "X")
    if conv3x3:
        if X.dim() != 4 or not X.is_contiguous():
            raise ValueError("conv3x3 input must be a contiguous NHWC tensor")
        B, H, Wd, C = X.shape
        M, K = B * H * Wd, 9 * C
        g = _ConvGeom(B, H, Wd, C, 3, 3, 1, 1)
        Xp = _packed_empty(M, K, X.device) if out is None else out
        _check(lib().bnn_pack_activations(_ptr(X), M, K, C, ctypes.byref(g), _ptr(Xp), _ld(Xp),
                                          _stream(X.device)), "bnn_pack_activations")
        return Xp
    M, K = X.shape
    Xp = _packed_empty(M, K, X.device) if out is None else out
    _check(lib().bnn_pack_activations(_ptr(X), M, K, _ld(X), None, _ptr(Xp), _ld(Xp),
                                      _stream(X.device)), "bnn_pack_activations")
    return Xp


def xnor_gemm(Xp: torch.Tensor, Wp: torch.Tensor, K: int, *, alpha: torch.Tensor | None = None,
              want_dot: bool = True, want_scaled: bool = False,
              D: torch.Tensor | None = None, Y: torch.Tensor | None = None):
    """D = K - 2 popcount(Xp xor Wp) (int32 [M, N]) and/or Y = alpha * D (fp32)."""
    _dev(Xp, torch.int32, "Xp")
    _dev(Wp, torch.int32, "Wp")
    M, N = Xp.shape[0], Wp.shape[0]
    if want_dot and D is None:
        D = torch.empty((M, N), dtype=torch.int32, device=Xp.device)
    if want_scaled and Y is None:
        Y = torch.empty((M, N), dtype=torch.float32, device=Xp.device)
    if not want_dot:
        D = None
    if not want_scaled:
        Y = None
    _check(lib().bnn_xnor_gemm(_ptr(Xp), _ld(Xp), _ptr(Wp), _ld(Wp), M, N, int(K),
                               _ptr(D), _ld(D) if D is not None else 0, _ptr(alpha),
                               _ptr(Y), _ld(Y) if Y is not None else 0,
                               _stream(Xp.device)), "bnn_xnor_gemm")
    return D, Y


def xnor_gemm_mfma(Xp: torch.Tensor, Wp: torch.Tensor, K: int, *, alpha: torch.Tensor | None = None,
                   want_dot: bool = True, want_scaled: bool = False,
                   D: torch.Tensor | None = None, Y: torch.Tensor | None = None):
    """The same D and Y as ``xnor_gemm``, computed on the fp4 matrix cores
    (bnn_xnor_gemm_mfma: exact +-1 products)."""
    _dev(Xp, torch.int32, "Xp")
    _dev(Wp, torch.int32, "Wp")
    M, N = Xp.shape[0], Wp.shape[0]
    if want_dot and D is None:
        D = torch.empty((M, N), dtype=torch.int32, device=Xp.device)
    if want_scaled and Y is None:
        Y = torch.empty((M, N), dtype=torch.float32, device=Xp.device)
    if not want_dot:
        D = None
    if not want_scaled:
        Y = None
    _check(lib().bnn_xnor_gemm_mfma(_ptr(Xp), _ld(Xp), _ptr(Wp), _ld(Wp), M, N, int(K),
                                    _ptr(D), _ld(D) if D is not None else 0, _ptr(alpha),
                                    _ptr(Y), _ld(Y) if Y is not None else 0,
                                    _stream(Xp.device)), "bnn_xnor_gemm_mfma")
    return D, Y


def _fused_struct(Xp, Wp, K, epilogue, M, *, alpha=None, R=None, tau=None, dir=None, D=None, Y=None,
                  Op=None, bias=None, Zp=None, nnz=None, beta=None):
    N = Wp.shape[0]
    dev = Xp.device
    if epilogue & EPI_DOT_I32 and D is None:
        D = torch.empty((M, N), dtype=torch.int32, device=dev)
    if epilogue & (EPI_SCALE_F32 | EPI_RESIDUAL_F32) and Y is None:
        Y = torch.empty((M, N), dtype=torch.float32, device=dev)
    if epilogue & (EPI_THRESH_PACK | EPI_SIGN_PACK) and Op is None:
        Op = _packed_empty(M, N, dev)
    a = _FusedArgs()
    a.Xp, a.ldXp = Xp.data_ptr(), _ld(Xp)
    a.Wp, a.ldWp = Wp.data_ptr(), _ld(Wp)
    a.M, a.N, a.K = M, N, int(K)
    a.epilogue = int(epilogue)
    if D is not None:
        a.D, a.ldD = D.data_ptr(), _ld(D)
    if alpha is not None:
        a.alpha = alpha.data_ptr()
    if Y is not None:
        a.Y, a.ldY = Y.data_ptr(), _ld(Y)
    if R is not None:
        a.R, a.ldR = R.data_ptr(), _ld(R)
    if tau is not None:
        a.tau = tau.data_ptr()
    if dir is not None:
        a.dir = dir.data_ptr()
    if Op is not None:
        a.Op, a.ldOp = Op.data_ptr(), _ld(Op)
    if bias is not None:
        a.bias = bias.data_ptr()
    if Zp is not None:
        a.Zp = Zp.data_ptr()
    if nnz is not None:
        a.nnz = nnz.data_ptr()
    if beta is not None:
        a.beta = beta.data_ptr()
    return a, {"D": D, "Y": Y, "Op": Op}


def linear_fused(Xp: torch.Tensor, Wp: torch.Tensor, K: int, epilogue: int, *,
                 alpha=None, R=None, tau=None, dir=None, D=None, Y=None, Op=None,
                 bias=None, Zp=None, nnz=None, beta=None, M: int | None = None):
    """XNOR-popcount GEMM with a fused epilogue (OR of EPI_* flags).

    Returns a dict with the outputs the flags ask for: ``D`` (int32 [M, N]),
    ``Y`` (fp32 [M, N]), ``Op`` (packed [M, ld] of the output signs).
    """
    _dev(Xp, torch.int32, "Xp")
    _dev(Wp, torch.int32, "Wp")
    M = Xp.shape[0] if M is None else M
    a, out = _fused_struct(Xp, Wp, K, epilogue, M, alpha=alpha, R=R, tau=tau, dir=dir, D=D, Y=Y, Op=Op,
                           bias=bias, Zp=Zp, nnz=nnz, beta=beta)
    _check(lib().bnn_linear_fused(ctypes.byref(a), _stream(Xp.device)), "bnn_linear_fused")
    return out


def conv3x3_fused(Ximg: torch.Tensor, Wp: torch.Tensor, geom, epilogue: int, **kw):
    """Binary 3x3 conv with implicit im2col: Ximg is the packed NHWC image
    [B*H*W, ld] (C bits per pixel), Wp the packed OHWI weights; geom =
    (B, H, W, C).  Epilogue keywords as for linear_fused."""
    _dev(Ximg, torch.int32, "Ximg")
    _dev(Wp, torch.int32, "Wp")
    B, H, W, C = geom
    M = B * H * W
    a, out = _fused_struct(Ximg, Wp, 9 * C, epilogue, M, **kw)
    g = _ConvGeom(B, H, W, C, 3, 3, 1, 1)
    _check(lib().bnn_conv3x3_fused(ctypes.byref(a), ctypes.byref(g), _stream(Ximg.device)), "bnn_conv3x3_fused")
    return out


def pack_activations_rsign(X: torch.Tensor, beta: torch.Tensor, *, out: torch.Tensor | None = None):
    """Packed RSign of fp32 rows [M, K]: bit = (x >= beta_k) ? 0 : 1."""
    _dev(X, torch.float32, "X")
    _dev(beta, torch.float32, "beta")
    M, K = X.shape
    Xp = _packed_empty(M, K, X.device) if out is None else out
    _check(lib().bnn_pack_activations_rsign(_ptr(X), M, K, _ld(X), _ptr(beta), _ptr(Xp), _ld(Xp),
                                            _stream(X.device)), "bnn_pack_activations_rsign")
    return Xp


def fold_bn_thresholds(gamma, beta, mean, var, eps, alpha):
    """Host-side BatchNorm fold -> (tau fp32 [N], dir int8 [N]) as numpy arrays."""
    import numpy as np
    g, b, mu, v, a = (np.ascontiguousarray(x, dtype=np.float32) for x in (gamma, beta, mean, var, alpha))
    N = a.shape[0]
    tau = np.empty(N, dtype=np.float32)
    d = np.empty(N, dtype=np.int8)
    P = lambda x: x.ctypes.data_as(ctypes.c_void_p)
    _check(lib().bnn_fold_bn_thresholds_host(P(g), P(b), P(mu), P(v), ctypes.c_float(float(eps)),
                                             P(a), N, P(tau), P(d)), "bnn_fold_bn_thresholds_host")
    return tau, d


def dense_f32_sign_pack(X: torch.Tensor, W: torch.Tensor, *, out: torch.Tensor | None = None):
    """FP first layer: packed signs of X W^T (double accumulation)."""
    _dev(X, torch.float32, "X")
    _dev(W, torch.float32, "W")
    M, K = X.shape
    N = W.shape[0]
    Op = _packed_empty(M, N, X.device) if out is None else out
    _check(lib().bnn_dense_f32_sign_pack(_ptr(X), _ld(X), _ptr(W), _ld(W), M, N, K,
                                         _ptr(Op), _ld(Op), _stream(X.device)),
           "bnn_dense_f32_sign_pack")
    return Op


def dense_binact_f32(Xp: torch.Tensor, W: torch.Tensor, K: int, *, out: torch.Tensor | None = None):
    """FP last layer on packed +1/-1 activations: fp32 [M, N]."""
    _dev(Xp, torch.int32, "Xp")
    _dev(W, torch.float32, "W")
    M, N = Xp.shape[0], W.shape[0]
    Y = torch.empty((M, N), dtype=torch.float32, device=Xp.device) if out is None else out
    _check(lib().bnn_dense_binact_f32(_ptr(Xp), _ld(Xp), _ptr(W), _ld(W), M, N, int(K),
                                      _ptr(Y), _ld(Y), _stream(Xp.device)), "bnn_dense_binact_f32")
    return Y


def weight_scale_tensor(W: torch.Tensor, *, out: torch.Tensor | None = None) -> torch.Tensor:
    """One scale for the whole matrix, ||W||_1 / (N K) (fp32 [1])."""
    _dev(W, torch.float32, "W")
    N, K = W.shape
    work = torch.empty(N, dtype=torch.float64, device=W.device)
    a = torch.empty(1, dtype=torch.float32, device=W.device) if out is None else out
    _check(lib().bnn_weight_scale_tensor(_ptr(W), N, K, _ld(W), _ptr(work), _ptr(a),
                                         _stream(W.device)), "bnn_weight_scale_tensor")
    return a


def weight_scale_tensor_noalloc(W: torch.Tensor, *, out: torch.Tensor) -> torch.Tensor:
    """The scale of weight_scale_tensor through the entry point that allocates
    nothing: the caller passes the output, the library's static per-GPU
    scratch holds the row sums (N <= NOALLOC_MAX_ROWS; overlapping calls on
    one GPU race)."""
    _dev(W, torch.float32, "W")
    _dev(out, torch.float32, "out")
    N, K = W.shape
    _check(lib().bnn_weight_scale_tensor_noalloc(_ptr(W), N, K, _ld(W), _ptr(out), _stream(W.device)),
           "bnn_weight_scale_tensor_noalloc")
    return out


def i8_ld(K: int) -> int:
    """Row stride of an int8 activation matrix: K rounded up to 16 bytes."""
    return (int(K) + 15) // 16 * 16


def _planes_ld(Xb: torch.Tensor) -> int:
    if Xb.dim() != 3 or Xb.shape[1] != 8 or Xb.stride(2) != 1 or Xb.stride(0) != 8 * Xb.stride(1):
        raise ValueError("bit planes must be an int32 tensor [M, 8, ld] with row stride 8*ld")
    return Xb.stride(1)


def quantize_act_i8(X: torch.Tensor, *, want_int8: bool = True, want_planes: bool = True,
                    want_xsum: bool | None = None):
    """Absmax INT8 quantization per row of fp32 X [M, K].

    Returns a dict: ``Xq`` int8 [M, K] (row stride a multiple of 16) or None,
    ``Xb`` int32 bit planes [M, 8, ld] (or None), ``xsum`` int32 [M] row
    sums (always with planes; else when ``want_xsum``), and ``xscale`` fp32
    [M] (X ~= xscale * Xq)."""
    _dev(X, torch.float32, "X")
    M, K = X.shape
    dev = X.device
    if want_xsum is None:
        want_xsum = want_planes
    if want_planes and not want_xsum:
        raise ValueError("bit planes come with their row sums")
    Xq = torch.empty((M, i8_ld(K)), dtype=torch.int8, device=dev)[:, :K] if want_int8 else None
    Xb = torch.empty((M, 8, padded_ld(K)), dtype=torch.int32, device=dev) if want_planes else None
    xsum = torch.empty(M, dtype=torch.int32, device=dev) if want_xsum else None
    xscale = torch.empty(M, dtype=torch.float32, device=dev)
    _check(lib().bnn_quantize_act_i8(_ptr(X), M, K, _ld(X),
                                     _ptr(Xq), Xq.stride(0) if Xq is not None else 0,
                                     _ptr(Xb), _planes_ld(Xb) if Xb is not None else 0, _ptr(xsum),
                                     _ptr(xscale), _stream(dev)), "bnn_quantize_act_i8")
    return {"Xq": Xq, "Xb": Xb, "xsum": xsum, "xscale": xscale}


def pack_act_i8(Xq: torch.Tensor):
    """Bit planes [M, 8, ld] and row sums [M] of int8 activations [M, K]."""
    _dev(Xq, torch.int8, "Xq")
    M, K = Xq.shape
    Xb = torch.empty((M, 8, padded_ld(K)), dtype=torch.int32, device=Xq.device)
    xsum = torch.empty(M, dtype=torch.int32, device=Xq.device)
    _check(lib().bnn_pack_act_i8(_ptr(Xq), M, K, _ld(Xq), _ptr(Xb), _planes_ld(Xb), _ptr(xsum),
                                 _stream(Xq.device)), "bnn_pack_act_i8")
    return Xb, xsum


def bwn_i8_linear(Wp: torch.Tensor, K: int, epilogue: int, *, Xb=None, xsum=None, Xq=None,
                  xscale=None, alpha=None, D=None, Y=None, Zp=None, M: int | None = None):
    """Binary weights x INT8 activations: D = sum q * s (int32) and/or
    Y = alpha * D (* xscale) (fp32), from bit planes (GEMV, M <= 2) or int8
    rows (MFMA GEMM).  Returns a dict with ``D`` and ``Y``.  expert_linear is
    the faster one for Y alone, from weights laid out once."""
    _dev(Wp, torch.int32, "Wp")
    if M is None:
        M = (Xb if Xb is not None else Xq).shape[0]
    N = Wp.shape[0]
    dev = Wp.device
    if epilogue & EPI_DOT_I32 and D is None:
        D = torch.empty((M, N), dtype=torch.int32, device=dev)
    if epilogue & EPI_SCALE_F32 and Y is None:
        Y = torch.empty((M, N), dtype=torch.float32, device=dev)
    a = _I8Args()
    if Xb is not None:
        _dev(Xb, torch.int32, "Xb")
        a.Xb, a.ldXb = Xb.data_ptr(), _planes_ld(Xb)
    if xsum is not None:
        a.xsum = xsum.data_ptr()
    if Xq is not None:
        _dev(Xq, torch.int8, "Xq")
        a.Xq, a.ldXq = Xq.data_ptr(), _ld(Xq)
    if xscale is not None:
        a.xscale = xscale.data_ptr()
    a.Wp, a.ldWp = Wp.data_ptr(), _ld(Wp)
    a.M, a.N, a.K = M, N, int(K)
    a.epilogue = int(epilogue)
    if D is not None:
        a.D, a.ldD = D.data_ptr(), _ld(D)
    if alpha is not None:
        a.alpha = alpha.data_ptr()
    if Y is not None:
        a.Y, a.ldY = Y.data_ptr(), _ld(Y)
    if Zp is not None:
        a.Zp = Zp.data_ptr()
    _check(lib().bnn_bwn_i8_linear(ctypes.byref(a), _stream(dev)), "bnn_bwn_i8_linear")
    return {"D": D, "Y": Y}


def bwn_f16_gemv(Wp: torch.Tensor, K: int, X: torch.Tensor, alpha: torch.Tensor, *,
                 alpha_tensor: bool = False, Y: torch.Tensor | None = None):
    """Binary weights x fp16 activations: Y = fl32(alpha * sum_k s x_k) with
    an fp32 sum (bnn_bwn_f16_gemv).  X float16 [M, ldX >= K] (ldX % 8 == 0),
    alpha fp32 [N] (or [1] with ``alpha_tensor``).  Returns Y fp32 [M, N]."""
    _dev(Wp, torch.int32, "Wp")
    _dev(X, torch.float16, "X")
    _dev(alpha, torch.float32, "alpha")
    M, N = X.shape[0], Wp.shape[0]
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float32, device=Wp.device)
    fl = EPI_SCALE_F32 | (EPI_ALPHA_TENSOR if alpha_tensor else 0)
    _check(lib().bnn_bwn_f16_gemv(X.data_ptr(), _ld(X), Wp.data_ptr(), _ld(Wp), M, N, int(K), fl,
                                  alpha.data_ptr(), Y.data_ptr(), _ld(Y), _stream(Wp.device)), "bnn_bwn_f16_gemv")
    return Y


def pack_weights_ternary(W: torch.Tensor, *, gamma: torch.Tensor | None = None, delta: float = 0.0):
    """Ternary weights as (sign plane Sp [N, ld], nonzero plane Zp [N, ld],
    nnz int32 [N]): RoundClip(W / gamma) (eq. (9)) when ``gamma`` (a device
    fp32 [1]) is given, else the threshold ``delta`` (eq. (7))."""
    _dev(W, torch.float32, "W")
    N, K = W.shape
    Sp = _packed_empty(N, K, W.device)
    Zp = _packed_empty(N, K, W.device)
    nnz = torch.empty(N, dtype=torch.int32, device=W.device)
    _check(lib().bnn_pack_weights_ternary(_ptr(W), N, K, _ld(W), _ptr(gamma), ctypes.c_float(float(delta)),
                                          _ptr(Sp), _ptr(Zp), _ld(Sp), _ptr(nnz), _stream(W.device)),
           "bnn_pack_weights_ternary")
    return Sp, Zp, nnz


# ---- the decoder's key/value cache
#
# These calls take a few microseconds on the GPU for a single token, so the
# argument structs are packed in one go (the layouts of the ctypes classes
# above) and the checks test what is right first.

def _layout(struct_type) -> struct.Struct:
    codes = {ctypes.c_void_p: "P", ctypes.c_int64: "q", ctypes.c_int32: "i", ctypes.c_float: "f"}
    s = struct.Struct("@" + "".join(codes[t] for _, t in struct_type._fields_))
    last, _ = struct_type._fields_[-1]
    assert s.size == getattr(struct_type, last).offset + getattr(struct_type, last).size
    return s


_pack_batch, _pack_rope, _pack_attn, _pack_score, _pack_evict = (
    _layout(t).pack for t in (_KvBatch, _RopeArgs, _AttnArgs, _ScoreArgs, _EvictArgs))


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda index: torch.cuda.current_stream(index).cuda_stream)


# Address of tensors without elements (a step without new tokens, a batch
# without sequences): torch gives them none, and the C calls want one though
# they do not read it.
_EMPTY = 256

BF16, F16, F32 = 1, 2, 3
_KV_TYPES = {torch.bfloat16: BF16, torch.float16: F16}
ROPE_KINDS = {"plain": 0, "linear": 1, "base": 2, "ramp": 3, "bands": 4}


def _workspace(t: torch.Tensor, index: int):
    """Address and bytes of a workspace on device `index`."""
    if t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"workspace must be contiguous on cuda:{index} (got strides {t.stride()} on {t.device})")
    return t.data_ptr(), t.numel() * t.element_size()


class KVCache:
    """A paged key/value cache over the caller's tensors (bnn_kv_cache).

    ``k``, ``v``: [pages, page_size, kv_heads, dim] in bfloat16 or float16,
    any strides with a unit last one (a head-major cache is passed
    transposed).  ``table``: int32 [B, pages per sequence], or None where
    sequence b owns page b.  ``pos`` int32 and ``score`` float32
    [B, kv_heads, slots]: the position and the running attention weight of
    each slot, for the calls that keep or read them; with a table a row for
    each of its sequences, without one their rows bound the sequences.  The tensors are kept
    alive by this object and used in place."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor | None = None, *,
                 pos: torch.Tensor | None = None, score: torch.Tensor | None = None):
        if k.dtype not in _KV_TYPES:
            raise TypeError(f"k must be torch.bfloat16 or torch.float16 (got {k.dtype})")
        _dev(k, k.dtype, "k")
        _dev(v, k.dtype, "v")
        if k.dim() != 4 or k.shape != v.shape or k.stride(3) != 1 or v.stride(3) != 1:
            raise ValueError("k and v must be [pages, page_size, kv_heads, dim] alike, with a unit last stride")
        pages, page, heads, dim = k.shape
        self.k, self.v, self.table, self.pos, self.score = k, v, table, pos, score
        self.device, self.dtype = k.device, k.dtype
        self._index = k.device.index
        self.kv_heads, self.dim, self.page_size = heads, dim, page
        c = self._c = _KvCache()
        c.K, c.k_page, c.k_slot, c.k_head = k.data_ptr() or _EMPTY, k.stride(0), k.stride(1), k.stride(2)
        c.V, c.v_page, c.v_slot, c.v_head = v.data_ptr() or _EMPTY, v.stride(0), v.stride(1), v.stride(2)
        if table is not None:
            _dev(table, torch.int32, "table")
            if table.dim() != 2 or not table.is_contiguous():
                raise ValueError("table must be a contiguous [B, pages per sequence] tensor")
            c.table, c.ld_table = table.data_ptr() or _EMPTY, table.shape[1]
        c.num_pages, c.page_size, c.kv_heads, c.dim, c.dtype = pages, page, heads, dim, _KV_TYPES[k.dtype]
        self.sequences = pages if table is None else table.shape[0]
        self.slots = page if table is None else table.shape[1] * page
        for t, dtype, name in ((pos, torch.int32, "pos"), (score, torch.float32, "score")):
            if t is not None:
                self._check_slots(_dev(t, dtype, name), name)
                self.sequences = min(self.sequences, t.shape[0])   # without a table there may be more pages than sequences
        self._ref = ctypes.addressof(c)

    def _check_slots(self, t, name):
        if t.dim() != 3 or t.shape[1] != self.kv_heads or t.shape[2] < self.slots or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [B, kv_heads, slots] tensor of at least {self.slots} slots")
        if self.table is not None and t.shape[0] < self.table.shape[0]:
            raise ValueError(f"{name} must have a row for each of the table's {self.table.shape[0]} sequences (got {t.shape[0]})")
        return t


def _batch(cache: KVCache, indptr, ctx, rows: int, max_nodes: int, max_ctx: int) -> bytes:
    n = ctx.numel()
    if not (indptr.dtype is torch.int32 and ctx.dtype is torch.int32 and indptr.is_cuda and ctx.is_cuda and indptr.numel() == n + 1
            and n <= cache.sequences and indptr.is_contiguous() and ctx.is_contiguous()):
        _dev(indptr, torch.int32, "indptr")
        _dev(ctx, torch.int32, "ctx")
        raise ValueError("indptr must be [B + 1] and ctx [B], contiguous, for at most the cache's sequences")
    return _pack_batch(indptr.data_ptr(), ctx.data_ptr() or _EMPTY, n, rows, max_nodes, max_ctx)


def _token_rows(t: torch.Tensor, dtype, name: str, rows, heads, dim):
    """Address, row stride and head stride of a token tensor."""
    st = t.stride()
    if not (t.dtype is dtype and t.is_cuda and t.shape == (rows, heads, dim) and st[2] == 1):
        _dev(t, dtype, name)
        raise ValueError(f"{name} must be [{rows}, {heads}, {dim}] with a unit last stride (got {tuple(t.shape)})")
    return t.data_ptr() or _EMPTY, st[0], st[1]


def _flat(t: torch.Tensor, dtype, name: str, n: int) -> int:
    if not (t.dtype is dtype and t.is_cuda and t.numel() == n and t.is_contiguous()):
        _dev(t, dtype, name)
        raise ValueError(f"{name} must be contiguous, with {n} elements")
    return t.data_ptr() or _EMPTY


def _row_floats(t: torch.Tensor, name: str, rows: int, heads: int):
    if not (t.dtype is torch.float32 and t.is_cuda and t.shape == (rows, heads) and t.stride(1) == 1):
        _dev(t, torch.float32, name)
        raise ValueError(f"{name} must be [{rows}, {heads}] with a unit last stride")
    return t.data_ptr() or _EMPTY, t.stride(0)


def _bit_rows(t: torch.Tensor | None, name: str, rows: int):
    if t is None:
        return 0, 0
    if not (t.dtype is torch.int32 and t.is_cuda and t.dim() == 2 and t.shape[0] == rows and t.is_contiguous()):
        _dev(t, torch.int32, name)
        raise ValueError(f"{name} must be a contiguous packed int32 [{rows}, words] tensor")
    return t.data_ptr() or _EMPTY, t.shape[1]


def rope_turns(max_pos: int, rot: int, *, base: float = 10000.0, kind: str = "plain", factor: float = 1.0,
               old_ctx: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0, device=None) -> torch.Tensor:
    """The table of qk_norm_rope, float32 [max_pos, rot]: rot/2 cosines, then
    rot/2 sines, computed in double (bnn_rope_turns_host).  ``kind``: "plain",
    "linear", "base", "ramp" or "bands", the ways to stretch positions to
    longer contexts that the header lists."""
    t = torch.empty((int(max_pos), int(rot)), dtype=torch.float32)
    if kind not in ROPE_KINDS:
        raise ValueError(f"kind must be one of {sorted(ROPE_KINDS)}")
    _check(lib().bnn_rope_turns_host(max_pos, rot, base, ROPE_KINDS[kind], factor, old_ctx, beta_fast, beta_slow, _ptr(t) or _EMPTY),
           "bnn_rope_turns_host")
    return t if device is None else t.to(device)


def tree_mask(parents, words: int | None = None) -> torch.Tensor:
    """Packed visibility rows of one tree of drafts, int32 [T, words] on the
    host: bit j of row i where node j is i or an ancestor of i.
    ``parents[i]`` < i, or -1 for a child of the last committed token."""
    p = torch.as_tensor(parents, dtype=torch.int32).contiguous()
    T = p.numel()
    words = max(1, (T + 31) // 32) if words is None else int(words)
    m = torch.zeros((T, words), dtype=torch.int32)
    if T:
        _check(lib().bnn_tree_mask_host(_ptr(p), T, _ptr(m), words), "bnn_tree_mask_host")
    return m


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cache: KVCache, indptr: torch.Tensor,
                 ctx: torch.Tensor, positions: torch.Tensor, turns: torch.Tensor | None, *,
                 q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                 interleaved: bool = False, q_out: torch.Tensor | None = None) -> torch.Tensor:
    """Norm and rotate the new tokens' queries and keys, append keys and
    values to the cache at the slots after each sequence's ``ctx``
    (bnn_qk_norm_rope).

    ``q`` [rows, heads, dim], ``k``, ``v`` [rows, kv_heads, dim]: float32 or
    the cache's type, views of one fused projection if wanted.  ``indptr``
    int32 [B + 1], ``ctx`` int32 [B], ``positions`` int32 [rows].  ``turns``:
    rope_turns, or None for no rotation.  Also fills the slots' ``cache.pos``
    and clears their ``cache.score`` where the cache has them.  Returns the
    queries in the cache's type, [rows, heads, dim]."""
    rows, heads, dim = q.shape
    src = q.dtype
    if src is not torch.float32 and src is not cache.dtype:
        raise TypeError(f"q must be torch.float32 or {cache.dtype} (got {src})")
    dim = cache.dim
    kv = cache.kv_heads
    if q_out is None:
        q_out = q.new_empty((rows, heads, dim), dtype=cache.dtype)
    table, max_pos, rot = 0, 0, 0
    if turns is not None:
        if turns.dim() != 2:
            raise ValueError("turns must be a contiguous [max_pos, rot] tensor")
        max_pos, rot = turns.shape
        table = _flat(turns, torch.float32, "turns", max_pos * rot)
    pos, score, slots = 0, 0, 0
    if cache.pos is not None:
        pos, slots = cache.pos.data_ptr() or _EMPTY, cache.pos.shape[2]
    if cache.score is not None:
        if pos and slots != cache.score.shape[2]:
            raise ValueError("cache.pos and cache.score must have the same number of slots")
        score, slots = cache.score.data_ptr() or _EMPTY, cache.score.shape[2]
    a = _pack_rope(*_token_rows(q, src, "q", rows, heads, dim), *_token_rows(k, src, "k", rows, kv, dim),
                   *_token_rows(v, src, "v", rows, kv, dim), F32 if src is torch.float32 else _KV_TYPES[src], heads,
                   *_token_rows(q_out, cache.dtype, "q_out", rows, heads, dim),
                   _flat(positions, torch.int32, "positions", rows), table, max_pos, rot, 1 if interleaved else 0,
                   0 if q_weight is None else _flat(q_weight, torch.float32, "q_weight", dim),
                   0 if k_weight is None else _flat(k_weight, torch.float32, "k_weight", dim), eps, pos, score, slots)
    _check((_lib or lib()).bnn_qk_norm_rope(cache._ref, _batch(cache, indptr, ctx, rows, rows, 0), a, _raw_stream(cache._index)),
           "bnn_qk_norm_rope")
    return q_out


def tree_attention_workspace(cache: KVCache, rows: int, heads: int, max_nodes: int, max_ctx: int) -> torch.Tensor:
    """A workspace for tree_attention calls of up to these sizes over up to all
    of this cache's sequences."""
    b = _pack_batch(0, 0, cache.sequences, rows, max_nodes, max_ctx)
    n = lib().bnn_tree_attention_workspace(cache._ref, b, heads)
    if n < 0:
        raise ValueError("tree_attention_workspace: sizes out of range")
    return torch.empty(n, dtype=torch.uint8, device=cache.device)


def tree_attention(q: torch.Tensor, cache: KVCache, indptr: torch.Tensor, ctx: torch.Tensor, *, max_nodes: int,
                   max_ctx: int, mask: torch.Tensor | None = None, scale: float | None = None,
                   out: torch.Tensor | None = None, lse: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                   workspace: torch.Tensor | None = None):
    """Attention of the new tokens' queries over the cache (bnn_tree_attention).

    ``q`` [rows, heads, dim] in the cache's type; ``mask``: packed int32
    [rows, words] (tree_mask), None for a causal run.  ``max_nodes`` and
    ``max_ctx`` bound the new and committed tokens of a sequence.  Returns
    (out [rows, heads, dim] in ``out_dtype``: float32, or the cache's type by
    default; lse float32 [rows, heads], the logarithm of each row's sum).
    ``workspace``: tree_attention_workspace, made here where it is None; with
    a smaller one long sequences are shared by fewer workgroups."""
    rows, heads, dim = q.shape
    b = _batch(cache, indptr, ctx, rows, max_nodes, max_ctx)
    if out is None:
        out = q.new_empty((rows, heads, dim), dtype=out_dtype or cache.dtype)
    if lse is None:
        lse = q.new_empty((rows, heads), dtype=torch.float32)
    kind = out.dtype
    if kind is not torch.float32 and kind is not cache.dtype:
        raise TypeError(f"out must be torch.float32 or {cache.dtype} (got {kind})")
    L = _lib or lib()
    if workspace is None:
        workspace = torch.empty(max(0, L.bnn_tree_attention_workspace(cache._ref, b, heads)), dtype=torch.uint8, device=q.device)
    a = _pack_attn(*_token_rows(q, cache.dtype, "q", rows, heads, cache.dim), heads, *_bit_rows(mask, "mask", rows),
                   dim ** -0.5 if scale is None else scale, *_token_rows(out, kind, "out", rows, heads, dim),
                   F32 if kind is torch.float32 else _KV_TYPES[kind], *_row_floats(lse, "lse", rows, heads), *_workspace(workspace, cache._index))
    _check(L.bnn_tree_attention(cache._ref, b, a, _raw_stream(cache._index)), "bnn_tree_attention")
    return out, lse


def cache_score_add(q: torch.Tensor, lse: torch.Tensor, cache: KVCache, indptr: torch.Tensor, ctx: torch.Tensor, *,
                    max_nodes: int, max_ctx: int, mask: torch.Tensor | None = None, accept: torch.Tensor | None = None,
                    scale: float | None = None, score_out: torch.Tensor | None = None) -> torch.Tensor:
    """Add to ``cache.score`` the attention weight that each slot received
    from the accepted new tokens (bnn_cache_score_add).  ``q``, ``mask``,
    ``scale``: as given to tree_attention; ``lse``: as it returned it;
    ``accept``: packed int32 [B, words], None where all tokens count.  Writes
    the sums in place, or into ``score_out``, and returns them."""
    rows, heads, dim = q.shape
    if cache.score is None:
        raise ValueError("the cache has no score tensor")
    if score_out is None:
        score_out = cache.score
    elif _dev(score_out, torch.float32, "score_out").shape != cache.score.shape or not score_out.is_contiguous():
        raise ValueError("score_out must be laid out as cache.score")
    a = _pack_score(*_token_rows(q, cache.dtype, "q", rows, heads, cache.dim), heads, *_row_floats(lse, "lse", rows, heads),
                    *_bit_rows(mask, "mask", rows), *_bit_rows(accept, "accept", ctx.numel()), dim ** -0.5 if scale is None else scale,
                    cache.score.data_ptr() or _EMPTY, score_out.data_ptr() or _EMPTY, cache.score.shape[2])
    _check((_lib or lib()).bnn_cache_score_add(cache._ref, _batch(cache, indptr, ctx, rows, max_nodes, max_ctx), a, _raw_stream(cache._index)),
           "bnn_cache_score_add")
    return score_out


def cache_evict_workspace(cache: KVCache) -> torch.Tensor:
    """A workspace for cache_evict calls on this cache."""
    n = lib().bnn_cache_evict_workspace(cache._ref, cache.sequences)
    if n < 0:
        raise ValueError("cache_evict_workspace: sizes out of range")
    return torch.empty(n, dtype=torch.uint8, device=cache.device)


def cache_evict(cache: KVCache, indptr: torch.Tensor, ctx: torch.Tensor, *, budget: int, recent: int, max_nodes: int,
                max_ctx: int, accept: torch.Tensor | None = None, ctx_out: torch.Tensor | None = None,
                pos_out: torch.Tensor | None = None, score_out: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Drop the new tokens that were not accepted and cut every sequence to
    ``budget`` tokens per key head by ``cache.score``, keeping the last
    ``recent`` positions first (bnn_cache_evict).  K and V are compacted in
    place; ``cache.pos``, ``cache.score`` and ``ctx`` too unless outputs are
    given.  Returns the new ctx, int32 [B]."""
    if cache.pos is None or cache.score is None:
        raise ValueError("the cache has no pos or no score tensor")
    if cache.pos.shape != cache.score.shape:
        raise ValueError("cache.pos and cache.score must have the same shape")
    pos_out = cache.pos if pos_out is None else _dev(pos_out, torch.int32, "pos_out")
    score_out = cache.score if score_out is None else _dev(score_out, torch.float32, "score_out")
    ctx_out = ctx if ctx_out is None else _dev(ctx_out, torch.int32, "ctx_out")
    slots = cache.pos.shape
    if pos_out.shape != slots or score_out.shape != slots or not (pos_out.is_contiguous() and score_out.is_contiguous()):
        raise ValueError("pos_out and score_out must be laid out as cache.pos")
    if ctx_out.shape != ctx.shape or not ctx_out.is_contiguous():
        raise ValueError("ctx_out must be laid out as ctx")
    if workspace is None:
        workspace = cache_evict_workspace(cache)
    a = _pack_evict(*_bit_rows(accept, "accept", ctx.numel()), budget, recent, cache.pos.data_ptr() or _EMPTY, pos_out.data_ptr() or _EMPTY,
                    cache.score.data_ptr() or _EMPTY, score_out.data_ptr() or _EMPTY, slots[2], ctx_out.data_ptr() or _EMPTY,
                    *_workspace(workspace, cache._index))
    _check((_lib or lib()).bnn_cache_evict(cache._ref, _batch(cache, indptr, ctx, 1 << 30, max_nodes, max_ctx), a, _raw_stream(cache._index)),
           "bnn_cache_evict")
    return ctx_out


# ---- the decoder's feed-forward half
#
# Also calls of a few microseconds: packed argument structs, checks that test
# what is right first.

_pack_norm, _pack_route = (_layout(t).pack for t in (_NormArgs, _RouteArgs))
# bnn_expert_args with its two matrices in line; each member of both is 8 bytes
_pack_expert = struct.Struct("@PqPqPqPqqqqiPPqPqPPqPqiPqPqi").pack
assert struct.calcsize("@PqPqPqPqqqqiPPqPqPPqPqiPqPqi") == _ExpertArgs.y_dtype.offset + 4

NORMS = {"none": 0, "rms": 1, "layer": 2}
SCORES = {"softmax": 0, "sigmoid": 1}
ACTIVATIONS = {"none": 0, "relu": 1, "relu2": 2, "silu": 3, "gelu": 4, "gelu_tanh": 5}
_TYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
_NORM_OUT = {"x", "y", "Xq", "Xb", "xsum", "xscale"}
MAX_NORM_D = 16384
MAX_EXPERTS = 1024


def _one_of(kinds: dict, value: str, name: str) -> int:
    if value not in kinds:
        raise ValueError(f"{name} must be one of {sorted(kinds)} (got {value!r})")
    return kinds[value]


def _float_type(t: torch.Tensor, name: str) -> int:
    kind = _TYPES.get(t.dtype)
    if kind is None:
        raise TypeError(f"{name} must be torch.float32, torch.bfloat16 or torch.float16 (got {t.dtype})")
    return kind


def _matrix(t: torch.Tensor, dtype, name: str, rows: int, cols: int, index: int):
    """Address and row stride of a [rows, cols] matrix on device `index`."""
    if not (t.dtype is dtype and t.shape == (rows, cols) and t.get_device() == index):
        _dev(t, dtype, name)
        raise ValueError(f"{name} must be [{rows}, {cols}] on cuda:{index} (got {tuple(t.shape)} on {t.device})")
    row, col = t.stride()
    if col != 1 and cols > 1 and rows > 0:
        raise ValueError(f"{name} must have a unit column stride")
    return t.data_ptr() or _EMPTY, row if rows > 1 else max(row, cols)


def _vector(t: torch.Tensor | None, dtype, name: str, n: int, index: int) -> int:
    """Address of a vector of n elements on device `index`; 0 for None."""
    if t is None:
        return 0
    if not (t.dtype is dtype and t.numel() == n and t.get_device() == index and t.is_contiguous()):
        _dev(t, dtype, name)
        raise ValueError(f"{name} must be contiguous on cuda:{index}, with {n} elements (got {tuple(t.shape)} on {t.device})")
    return t.data_ptr() or _EMPTY


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _on(index: int, call, *args) -> int:
    """The status of a call that launches on device `index`, on its current stream."""
    if index == _current_device():
        return call(*args, _raw_stream(index))
    with torch.cuda.device(index):
        return call(*args, _raw_stream(index))


def block_norm(x: torch.Tensor | None = None, branch: torch.Tensor | None = None, *, place: torch.Tensor | None = None,
               weight: torch.Tensor | None = None, post: str = "none", post_weight: torch.Tensor | None = None,
               post_bias: torch.Tensor | None = None, gate: torch.Tensor | None = None, x_scale: float = 1.0,
               branch_scale: float = 1.0, pre: str = "rms", pre_weight: torch.Tensor | None = None,
               pre_bias: torch.Tensor | None = None, eps: float = 1e-6, used: torch.Tensor | None = None,
               y_dtype: torch.dtype | None = None, int8: bool = True, planes: bool = False, out: dict | None = None) -> dict:
    """What lies between two linear layers of a block, in one pass
    (bnn_block_norm):

        b = sum_j weight[:, j] * branch[place[:, j]]       (or branch)
        x = x_scale * x + branch_scale * gate * post(b);   y = pre(x);   INT8 rows of y

    ``x`` [M, D] (the residual stream) and ``branch`` [M, D], or [rows, D]
    with ``place`` int32 and ``weight`` float32 [M, parts] (as expert_route
    gives them): float32, bfloat16 or float16, either may be left out.
    ``post``, ``pre``: "none", "rms" or "layer", with float32 [D] weights and
    biases (None: 1 and 0).  ``gate``: float32 [D] or [M, D].  ``used``: int32
    [1], the rows from there on are left alone.

    Returns a dict: ``x`` (the new stream, where x and branch are given),
    ``y`` in ``y_dtype`` (where given), with ``int8`` ``Xq``, with ``planes``
    ``Xb`` and ``xsum``, with either ``xscale``, laid out as by
    quantize_act_i8.  Codes are ``rint(y * (127.0 / amax))`` as torch computes
    it on the GPU (127 times the reciprocal); quantize_act_i8, of ``y`` in
    float32, rounds the factor once: about 2.5 of 10^7 codes, next to a border,
    differ by one.  ``out``: such a dict of tensors to write instead; it then says by
    itself which outputs there are (``out["x"]`` may be ``x``)."""
    first = x if x is not None else branch
    if first is None:
        raise ValueError("x or branch must be given")
    index = _dev(first, first.dtype, "x or branch").get_device()
    D = first.shape[-1]
    M = x.shape[0] if x is not None else place.shape[0] if place is not None else branch.shape[0]
    if out is None:
        dev = first.device
        out = {}
        if x is not None and branch is not None:
            out["x"] = torch.empty((M, D), dtype=x.dtype, device=dev)
        if y_dtype is not None:
            out["y"] = torch.empty((M, D), dtype=y_dtype, device=dev)
        if int8:
            out["Xq"] = torch.empty((M, i8_ld(D)), dtype=torch.int8, device=dev)[:, :D]
        if planes:
            out["Xb"] = torch.empty((M, 8, padded_ld(D)), dtype=torch.int32, device=dev)
            out["xsum"] = torch.empty(M, dtype=torch.int32, device=dev)
        if int8 or planes:
            out["xscale"] = torch.empty(M, dtype=torch.float32, device=dev)
    elif not out.keys() <= _NORM_OUT:
        raise ValueError(f"out may hold {sorted(_NORM_OUT)} (got {sorted(out)})")
    get = out.get
    xo, y, Xq, Xb, xsum, xscale = get("x"), get("y"), get("Xq"), get("Xb"), get("xsum"), get("xscale")
    xp, bp, op, yp, qp, gp = (0, 0), (0, 0), (0, 0), (0, 0), (0, 0), (0, 0)
    xt = bt = yt = b_rows = parts = 0
    if x is not None:
        xt = _float_type(x, "x")
        xp = _matrix(x, x.dtype, "x", M, D, index)
    if branch is not None:
        bt = _float_type(branch, "branch")
        b_rows = branch.shape[0] if place is not None else M
        bp = _matrix(branch, branch.dtype, "branch", b_rows, D, index)
    if xo is not None:
        if x is not None and xo.dtype is not x.dtype:
            raise TypeError(f"out['x'] must be {x.dtype} (got {xo.dtype})")
        xt = _float_type(xo, "out['x']")
        op = _matrix(xo, xo.dtype, "out['x']", M, D, index)
    if y is not None:
        yt = _float_type(y, "out['y']")
        yp = _matrix(y, y.dtype, "out['y']", M, D, index)
    if Xq is not None:
        qp = _matrix(Xq, torch.int8, "out['Xq']", M, D, index)
    bits = (0, 0)
    if Xb is not None:
        if _dev(Xb, torch.int32, "out['Xb']").dim() != 3 or Xb.shape[0] != M or Xb.get_device() != index:
            raise ValueError(f"out['Xb'] must be [{M}, 8, ld] on cuda:{index}")
        bits = Xb.data_ptr() or _EMPTY, _planes_ld(Xb)
        if Xb.shape[2] != bits[1]:   # all ld words of a plane are written
            raise ValueError(f"out['Xb'] must have no words between its rows (got {Xb.shape[2]} words at a stride of {bits[1]})")
    if place is not None:
        if place.dim() != 2 or place.shape[0] != M or (weight is not None and weight.shape != place.shape):
            raise ValueError(f"place and weight must be [{M}, parts] alike")
        parts = place.shape[1]
    elif weight is not None:
        raise ValueError("weight goes with place")
    if gate is not None:
        gp = (_vector(gate, torch.float32, "gate", D, index), 0) if gate.dim() == 1 else _matrix(gate, torch.float32, "gate", M, D, index)
    f32, i32 = torch.float32, torch.int32

    a = _pack_norm(M, D, _vector(used, i32, "used", 1, index), *xp, xt, *bp, bt, b_rows, _vector(place, i32, "place", M * parts, index),
                   _vector(weight, f32, "weight", M * parts, index), parts, _one_of(NORMS, post, "post"),
                   _vector(post_weight, f32, "post_weight", D, index), _vector(post_bias, f32, "post_bias", D, index), *gp, x_scale, branch_scale,
                   _one_of(NORMS, pre, "pre"), _vector(pre_weight, f32, "pre_weight", D, index), _vector(pre_bias, f32, "pre_bias", D, index), eps,
                   *op, *yp, yt, *qp, *bits, _vector(xsum, i32, "out['xsum']", M, index), _vector(xscale, f32, "out['xscale']", M, index))
    _check(_on(index, (_lib or lib()).bnn_block_norm, a), "bnn_block_norm")
    return out


def expert_route_workspace(rows: int, experts: int, top: int, *, device="cuda") -> torch.Tensor:
    """A workspace for expert_route calls of up to these rows and experts."""
    n = lib().bnn_expert_route_workspace(rows, experts, top)
    if n < 0:
        raise ValueError("expert_route_workspace: sizes out of range")
    return torch.empty(n, dtype=torch.uint8, device=device)


def expert_route(logits: torch.Tensor, top: int, *, score: str = "softmax", bias: torch.Tensor | None = None, renorm: bool = False,
                 scale: float = 1.0, used: torch.Tensor | None = None, out: dict | None = None, workspace: torch.Tensor | None = None) -> dict:
    """The experts of every token and the tokens sorted by expert
    (bnn_expert_route).

    ``logits`` [rows, experts] in float32, bfloat16 or float16.  ``score``:
    "softmax" (over all experts) or "sigmoid".  ``bias`` float32 [experts] is
    added to the scores for the choice only.  ``renorm``: weights divided by
    their sum.  ``used``: int32 [1], rows from there on have no experts.

    Returns a dict: ``expert`` int32 and ``weight`` float32 [rows, top],
    ``offsets`` int32 [experts + 1] (expert e has the positions offsets[e] ..
    offsets[e + 1] - 1), ``order`` int32 [rows * top] (row * top + choice of
    each position), ``place`` int32 [rows, top] (its inverse; -1: none).
    ``out``: such a dict of tensors to write instead.  ``workspace``:
    expert_route_workspace on the device of ``logits``, made here where it is
    None."""
    rows, experts = logits.shape
    index = _dev(logits, logits.dtype, "logits").get_device()
    L = _lib or lib()
    if out is None:
        pair = dict(dtype=torch.int32, device=logits.device)
        out = {"expert": torch.empty((rows, top), **pair), "weight": torch.empty((rows, top), dtype=torch.float32, device=logits.device),
               "offsets": torch.empty(experts + 1, **pair), "order": torch.empty(rows * top, **pair), "place": torch.empty((rows, top), **pair)}
    if workspace is None:
        workspace = torch.empty(max(0, L.bnn_expert_route_workspace(rows, experts, top)), dtype=torch.uint8, device=logits.device)
    n, i32 = rows * top, torch.int32
    a = _pack_route(*_matrix(logits, logits.dtype, "logits", rows, experts, index), _float_type(logits, "logits"), rows, experts, top,
                    _vector(used, i32, "used", 1, index), _one_of(SCORES, score, "score"), _vector(bias, torch.float32, "bias", experts, index),
                    1 if renorm else 0, scale, _vector(out["expert"], i32, "out['expert']", n, index),
                    _vector(out["weight"], torch.float32, "out['weight']", n, index), _vector(out["offsets"], i32, "out['offsets']", experts + 1, index),
                    _vector(out["order"], i32, "out['order']", n, index), _vector(out["place"], i32, "out['place']", n, index),
                    *_workspace(workspace, index))
    _check(_on(index, L.bnn_expert_route, a), "bnn_expert_route")
    return out


class ExpertWeights:
    """One matrix for each expert as expert_linear reads it, laid out once
    from packed planes (bnn_expert_pack).

    ``Wp``, ``Zp``: the planes of pack_weights (``Zp`` None) or
    pack_weights_ternary, [N, ld] of a single layer or [experts, N, ld]
    stacked.  ``alpha`` float32 [experts, N] ([N] of a single layer), or
    [experts] with one scale for a whole matrix; ``bias`` float32 like
    [experts, N], or None.  A row of either that experts share, as by
    ``expand``, is copied for each.  The planes are not needed afterwards; ``alpha`` and ``bias`` are
    kept and read by each call."""

    def __init__(self, Wp: torch.Tensor, K: int, *, Zp: torch.Tensor | None = None, alpha: torch.Tensor, bias: torch.Tensor | None = None):
        _dev(Wp, torch.int32, "Wp")
        if Wp.dim() == 2:
            Wp = Wp[None]
            Zp = Zp[None] if Zp is not None and Zp.dim() == 2 else Zp
        if Wp.dim() != 3 or Wp.stride(2) != 1:
            raise ValueError("Wp must be [N, ld] or [experts, N, ld] with a unit last stride")
        if Zp is not None and (_dev(Zp, torch.int32, "Zp").shape != Wp.shape or Zp.stride() != Wp.stride() or Zp.get_device() != Wp.get_device()):
            raise ValueError("Zp must be laid out as Wp, on its device")
        self.experts, self.N, self.K, self.ternary = Wp.shape[0], Wp.shape[1], int(K), Zp is not None
        self.device = Wp.device
        n = lib().bnn_expert_pack_bytes(self.experts, self.N, self.K, self.ternary)
        if n < 0:
            raise ValueError("ExpertWeights: sizes out of range")
        if Wp.shape[2] < (self.K + 31) // 32:   # a stride of so many words is not enough: a narrow view ends before
            raise ValueError(f"Wp must have the {(self.K + 31) // 32} words of K = {self.K} (got {Wp.shape[2]})")
        W = torch.empty(n, dtype=torch.uint8, device=Wp.device)
        index = self._index = Wp.get_device()
        _check(_on(index, lib().bnn_expert_pack, Wp.data_ptr() or _EMPTY, 0 if Zp is None else Zp.data_ptr() or _EMPTY, Wp.stride(1), Wp.stride(0),
                   self.experts, self.N, self.K, W.data_ptr() or _EMPTY, n), "bnn_expert_pack")
        _dev(alpha, torch.float32, "alpha")
        if alpha.shape == (self.N,) and self.experts == 1 and self.N != 1:
            alpha = alpha[None]
        if alpha.shape == (self.experts,):
            scale = _vector(alpha, torch.float32, "alpha", self.experts, index), 0
        else:
            alpha = self._rows(alpha)
            scale = _matrix(alpha, torch.float32, "alpha", self.experts, self.N, index)
        shift = 0, 0
        if bias is not None:
            bias = self._rows(_dev(bias, torch.float32, "bias"))
            shift = _matrix(bias[None] if bias.dim() == 1 else bias, torch.float32, "bias", self.experts, self.N, index)
        self._held = W, alpha, bias
        self._c = (W.data_ptr() or _EMPTY, *scale, *shift)

    def _rows(self, t: torch.Tensor) -> torch.Tensor:
        """A row that experts share laid out for each: a stride of 0 says that each has a single scale, and no bias can have it."""
        return t.contiguous() if t.dim() == 2 and self.experts > 1 and t.stride(0) < self.N else t

    # Their addresses are in _c: they can be written in place, not replaced.
    W = property(lambda self: self._held[0])
    alpha = property(lambda self: self._held[1])
    bias = property(lambda self: self._held[2])


def expert_linear(Xq: torch.Tensor, weights: ExpertWeights, *, xscale: torch.Tensor | None = None, offsets: torch.Tensor | None = None,
                  order: torch.Tensor | None = None, per_row: int = 1, up: ExpertWeights | None = None, act: str = "none",
                  residual: torch.Tensor | None = None, out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """INT8 rows times the matrix of each row's expert (bnn_expert_linear):

        y = act(alpha * D * xscale + bias) [* (the same of ``up``)] [+ residual],   D = Xq W^T

    ``Xq`` int8 [rows, K] with a row stride of a multiple of 16 and ``xscale``
    float32 [rows], as quantize_act_i8 and block_norm give them.
    ``offsets``: int32 [experts + 1], the positions of each expert (None with a
    single matrix: all).  ``order`` int32 [positions]: position p reads row
    order[p] // per_row (expert_route's order and top); None: row p.  ``act``:
    "none", "relu", "relu2", "silu", "gelu" or "gelu_tanh".  ``residual``:
    [positions, N] in the output's type.  Returns ``out`` [positions, N] in
    ``out_dtype`` (float32, bfloat16 or float16); positions past the last
    expert's are left alone.

    A single matrix is what bwn_i8_linear takes too, from the packed planes as
    they are, with int32 sums or from bit planes of the rows; where scaled
    values are wanted this call is the faster one (measured from 1 to 8192 rows)."""
    rows = Xq.shape[0]
    K, N, experts = weights.K, weights.N, weights.experts
    positions = rows if order is None else order.numel()
    if out is None:
        out = Xq.new_empty((positions, N), dtype=out_dtype)
    if up is not None and (up._index != weights._index or up.K != K or up.N != N or up.experts != experts or up.ternary != weights.ternary):
        raise ValueError("up must have the sizes, the kind and the device of weights")
    kind = out.dtype
    index = weights._index
    a = _pack_expert(*_matrix(Xq, torch.int8, "Xq", rows, K, index), _vector(xscale, torch.float32, "xscale", rows, index), rows,
                     _vector(order, torch.int32, "order", positions, index), per_row, _vector(offsets, torch.int32, "offsets", experts + 1, index),
                     experts, positions, N, K, 1 if weights.ternary else 0, *weights._c, *(up._c if up is not None else (0, 0, 0, 0, 0)),
                     _one_of(ACTIVATIONS, act, "act"), *((0, 0) if residual is None else _matrix(residual, kind, "residual", positions, N, index)),
                     *_matrix(out, kind, "out", positions, N, index), _float_type(out, "out"))
    _check(_on(index, (_lib or lib()).bnn_expert_linear, a), "bnn_expert_linear")
    return out
