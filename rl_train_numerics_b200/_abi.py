"""Thin Python binding of libgdn_cpr.so (the C ABI in include/gdn_cpr.h,
gdn_pik.h, gdn_qk_norm.h and gdn_glr.h).

Argument marshalling only: torch provides device memory and the current CUDA
stream; every step of the layer runs in the library's CUDA kernels.  There is
no CPU or PyTorch fallback: if the shared library is missing, importing this
module raises, and every call checks that its tensors live on a CUDA device.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgdn_cpr.so")

GDN_OK = 0
GDN_ERR_INVALID_ARG = -1
GDN_ERR_UNSUPPORTED = -2
GDN_ERR_WORKSPACE = -3
GDN_ERR_CUDA = -4
GDN_ERR_DEVICE_DATA = -5
GDN_ERR_TIMEOUT = -6
GDN_ERR_CONTRACT = -7
GDN_DIGEST_SEMANTIC = 0
GDN_DIGEST_POLICY = 1
GDN_DIGEST_DEPLOYMENT = 2
GDN_BF16 = 0
GDN_F32 = 1
GDN_DEVERR_CU_SEQLENS = 1
GDN_DEVERR_POS = 2
GDN_DEVERR_TIMEOUT = 4
GDN_BWD_REUSE_FORWARD = 1
GDN_QK_NORM_L2 = 0
GDN_QK_NORM_RMS = 1
GDN_GLR_INPUT_PLAIN = 0
GDN_GLR_INPUT_COMPLEMENT = 1
CHUNK = 64
GLR_CHUNK = 16


class GdnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}")


class DecodeStateStruct(ctypes.Structure):
    _fields_ = [("s_run", ctypes.c_void_p), ("s_scale", ctypes.c_void_p),
                ("s_bnd", ctypes.c_void_p),
                ("buf_k", ctypes.c_void_p), ("buf_v", ctypes.c_void_p),
                ("buf_beta", ctypes.c_void_p), ("buf_g", ctypes.c_void_p),
                ("pos", ctypes.c_void_p), ("error", ctypes.c_void_p),
                ("resync", ctypes.c_void_p), ("n_slots", ctypes.c_int)]


class GlrStateStruct(ctypes.Structure):
    _fields_ = [("h", ctypes.c_void_p), ("a", ctypes.c_void_p), ("b", ctypes.c_void_p),
                ("pos", ctypes.c_void_p), ("error", ctypes.c_void_p),
                ("n_slots", ctypes.c_int)]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() or "
                          "python -m rl_train_numerics_b200.build_lib")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                             ctypes.c_size_t)
    sigs = {
        "gdn_cpr_abi_version": (i32, []),
        "gdn_status_string": (ctypes.c_char_p, [i32]),
        "gdn_cpr_forward_workspace_bytes": (sz, [i32, i64, i32, i32, i32, i32, i32]),
        "gdn_cpr_forward": (i32, [vp, vp, vp, i32, vp, vp, vp, i32, i64, i32, i32, i32, i32, f32,
                                  vp, vp, i32, vp, vp, vp, vp, sz, vp]),
        "gdn_cpr_forward_ex": (i32, [vp, vp, vp, i32, vp, vp, vp, i32, i64, i32, i32, i32, i32,
                                     f32, vp, vp, i32, vp, vp, vp, vp, sz, vp, vp]),
        "gdn_cpr_forward_noalloc": (i32, [vp, vp, vp, i32, vp, vp, vp, i32, i64, i32, i32, i32,
                                          i32, f32, vp, vp, i32, vp, vp, vp, vp, vp]),
        "gdn_cpr_decode_state_from_prefill": (i32, [vp, vp, i32, vp, vp, vp, i32, i64, i32, i32,
                                                    i32, i32, vp, vp, vp, vp,
                                                    DecodeStateStruct, vp]),
        "gdn_cpr_decode_step": (i32, [vp, vp, vp, i32, vp, vp, vp, i32, i32, i32, i32, i32, f32,
                                      DecodeStateStruct, vp, i32, vp]),
        "gdn_chunk_boundary": (i32, [vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, i32, vp, vp]),
        "gdn_recurrent_forward": (i32, [vp, vp, vp, i32, vp, vp, vp, i32, i64, i32, i32, i32, f32,
                                        vp, vp, i32, vp, vp, vp, vp]),
        "gdn_recurrent_decode_step": (i32, [vp, vp, vp, i32, vp, vp, i32, i32, i32, i32, f32, vp,
                                            vp, vp, i32, vp]),
        "gdn_native_forward": (i32, [vp, vp, vp, i32, vp, vp, vp, i32, i64, i32, i32, i32, i32,
                                     f32, vp, vp, i32, vp, vp, vp, sz, vp, vp]),
        "gdn_cpr_backward_workspace_bytes": (sz, [i32, i64, i32, i32, i32, i32, i32]),
        "gdn_cpr_backward": (i32, [vp, vp, vp, i32, vp, vp, vp, i32, i64, i32, i32, i32, i32,
                                   f32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, i32, vp]),
        "gdn_cpr_backward_ex": (i32, [vp, vp, vp, i32, vp, vp, vp, i32, i64, i32, i32, i32,
                                      i32, f32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, i32,
                                      vp, vp]),
        "gdn_pik_workspace_bytes": (sz, [i64, i64, i64, i32, i32]),
        "gdn_pik_gemm": (i32, [vp, vp, vp, i64, i64, i64, i32, i32, vp, sz, vp, vp]),
        "gdn_check_error": (i32, [vp, vp, vp]),
        "gdn_cpr_contract_descriptor": (i32, [i32, i32, i32, i32, i32, i32, ctypes.c_char_p, sz,
                                              ctypes.POINTER(ctypes.c_size_t)]),
        "gdn_cpr_contract_digest": (i32, [i32, i32, i32, i32, i32, i32, ctypes.c_char_p]),
        "gdn_cpr_contract_check": (i32, [ctypes.c_char_p, i32, i32, i32, i32, i32]),
        "gdn_sha256": (i32, [ctypes.c_char_p, sz, ctypes.c_char_p]),
        "gdn_selftest_bounded_wait": (i32, [i32, vp, vp]),
        "gdn_qk_norm_forward": (i32, [vp, i64, vp, i64, i32, i64, i32, i32, i32, i32, f32, vp, vp,
                                      vp, vp, i32, i32, vp, i64, vp, i64, i32, vp]),
        "gdn_qk_norm_backward_workspace_bytes": (sz, [i64, i32, i32, i32]),
        "gdn_qk_norm_backward": (i32, [vp, i64, vp, i64, i32, i64, i32, i32, i32, i32, f32, vp,
                                       vp, vp, vp, i32, i32, vp, i64, vp, i64, i32, vp, i64, vp,
                                       i64, vp, vp, vp, sz, vp]),
        "gdn_glr_carry_rows": (i64, [i32, i64]),
        "gdn_glr_forward": (i32, [vp, i64, i32, vp, i64, i32, vp, i32, i64, i32, i32, vp, vp, i64,
                                  i32, vp, ctypes.POINTER(GlrStateStruct), vp, vp, vp, vp]),
        "gdn_glr_backward": (i32, [vp, i64, i32, vp, i64, i32, vp, i32, i64, i32, i32, vp, vp,
                                   i64, i32, vp, vp, i64, vp, i64, vp, vp, vp]),
        "gdn_glr_decode_step": (i32, [vp, i64, i32, vp, i64, i32, vp, i32, i32, i32,
                                      GlrStateStruct, vp, i64, i32, vp]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


def status_string(status: int) -> str:
    return lib.gdn_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status != GDN_OK:
        raise GdnError(status, what)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("gdn_cpr: tensors must be on a CUDA device (there is no CPU path)")
    if not t.is_contiguous():
        raise ValueError("gdn_cpr: tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return GDN_BF16
    if t.dtype == torch.float32:
        return GDN_F32
    raise ValueError(f"gdn_cpr: unsupported dtype {t.dtype}")


def _out_code(in_code: int, out_dtype, o) -> int:
    """Output dtype code: from `o` when given (must agree with out_dtype), else
    out_dtype, else the input dtype."""
    if o is not None:
        code = _dtype_code(o)
        if out_dtype is not None and _dtype_code(torch.empty(0, dtype=out_dtype)) != code:
            raise ValueError("gdn_cpr: out_dtype disagrees with the dtype of o")
        return code
    if out_dtype is None:
        return in_code
    return _dtype_code(torch.empty(0, dtype=out_dtype))


def _torch_dtype(code: int):
    return torch.bfloat16 if code == GDN_BF16 else torch.float32


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def forward_workspace_bytes(n_seqs: int, total_tokens: int, H: int, dk: int, dv: int,
                            C: int = CHUNK, in_dtype=torch.bfloat16) -> int:
    code = GDN_BF16 if in_dtype == torch.bfloat16 else GDN_F32
    return int(lib.gdn_cpr_forward_workspace_bytes(n_seqs, total_tokens, H, dk, dv, C, code))


def forward(q, k, v, beta, g, cu_seqlens, *, n_seqs: Optional[int] = None, h0=None,
            C: int = CHUNK, scale: float = 1.0, out_dtype=None, o=None, s_run_final=None,
            s_bnd_final=None, s_run_scale=None, want_states: bool = True, workspace=None,
            stream=None, kernel_events=None):
    """gdn_cpr_forward (gdn_cpr_forward_ex when ``kernel_events``, a list of 5
    recorded torch.cuda.Event objects, is given).
    Returns (o, s_run_final, s_bnd_final, workspace).  s_run_final is the
    running state itself, unless an ``s_run_scale`` tensor [N, H] fp32 is
    passed: then s_run_final holds the mantissa and s_run_scale the scale (the
    pair decode needs to continue bit for bit)."""
    T, H, dk = q.shape
    dv = v.shape[2]
    N = (cu_seqlens.numel() - 1) if n_seqs is None else int(n_seqs)
    in_code = _dtype_code(q)
    out_code = _out_code(in_code, out_dtype, o)
    dev = q.device
    if o is None:
        o = torch.empty((T, H, dv), dtype=_torch_dtype(out_code), device=dev)
    if want_states:
        if s_run_final is None:
            s_run_final = torch.empty((N, H, dv, dk), dtype=torch.float32, device=dev)
        if s_bnd_final is None:
            s_bnd_final = torch.empty((N, H, dv, dk), dtype=torch.float32, device=dev)
    need = forward_workspace_bytes(N, T, H, dk, dv, C, q.dtype)
    if workspace is None:
        workspace = torch.zeros(max(need, 256), dtype=torch.uint8, device=dev)
    ev = None
    if kernel_events is not None:
        if len(kernel_events) != 5 or any(e.cuda_event == 0 for e in kernel_events):
            raise ValueError("kernel_events: 5 torch.cuda.Event objects, each recorded once")
        ev = (ctypes.c_void_p * 5)(*[e.cuda_event for e in kernel_events])
    st = lib.gdn_cpr_forward_ex(_ptr(q), _ptr(k), _ptr(v), in_code, _ptr(beta), _ptr(g),
                                _ptr(cu_seqlens), N, T, H, dk, dv, C, float(scale), _ptr(h0),
                                _ptr(o), out_code, _ptr(s_run_final), _ptr(s_run_scale),
                                _ptr(s_bnd_final), _ptr(workspace), workspace.numel(), ev,
                                _stream(stream))
    _check(st, "gdn_cpr_forward")
    return o, s_run_final, s_bnd_final, workspace


def native_forward(q, k, v, beta, g, cu_seqlens, *, n_seqs: Optional[int] = None, h0=None,
                   C: int = CHUNK, scale: float = 1.0, out_dtype=None, o=None, s_final=None,
                   s_bnd_final=None, want_states: bool = True, workspace=None, stream=None,
                   kernel_events=None):
    """gdn_native_forward (the chunked, "native mixed" forward; d = 128, bf16).
    Returns (o, s_final, s_bnd_final, workspace); the workspace is the CPR
    forward's (same size).  kernel_events: 5 recorded torch.cuda.Event objects."""
    T, H, dk = q.shape
    dv = v.shape[2]
    N = (cu_seqlens.numel() - 1) if n_seqs is None else int(n_seqs)
    in_code = _dtype_code(q)
    out_code = _out_code(in_code, out_dtype, o)
    dev = q.device
    if o is None:
        o = torch.empty((T, H, dv), dtype=_torch_dtype(out_code), device=dev)
    if want_states:
        if s_final is None:
            s_final = torch.empty((N, H, dv, dk), dtype=torch.float32, device=dev)
        if s_bnd_final is None:
            s_bnd_final = torch.empty((N, H, dv, dk), dtype=torch.float32, device=dev)
    need = forward_workspace_bytes(N, T, H, dk, dv, C, q.dtype)
    if workspace is None:
        workspace = torch.zeros(max(need, 256), dtype=torch.uint8, device=dev)
    ev = None
    if kernel_events is not None:
        if len(kernel_events) != 5 or any(e.cuda_event == 0 for e in kernel_events):
            raise ValueError("kernel_events: 5 torch.cuda.Event objects, each recorded once")
        ev = (ctypes.c_void_p * 5)(*[e.cuda_event for e in kernel_events])
    st = lib.gdn_native_forward(_ptr(q), _ptr(k), _ptr(v), in_code, _ptr(beta), _ptr(g),
                                _ptr(cu_seqlens), N, T, H, dk, dv, C, float(scale), _ptr(h0),
                                _ptr(o), out_code, _ptr(s_final), _ptr(s_bnd_final),
                                _ptr(workspace), workspace.numel(), ev, _stream(stream))
    _check(st, "gdn_native_forward")
    return o, s_final, s_bnd_final, workspace


def recurrent_forward(q, k, v, beta, g, cu_seqlens, *, n_seqs: Optional[int] = None, h0=None,
                      scale: float = 1.0, out_dtype=None, o=None, s_final=None,
                      s_final_scale=None, want_state: bool = True, error=None, stream=None):
    """gdn_recurrent_forward (the recurrent-everywhere forward).  Returns
    (o, s_final, s_final_scale, error word).  s_final is the state itself
    unless an ``s_final_scale`` tensor [N, H] fp32 is passed: then s_final
    holds the mantissa and s_final_scale the scale."""
    T, H, dk = q.shape
    dv = v.shape[2]
    N = (cu_seqlens.numel() - 1) if n_seqs is None else int(n_seqs)
    in_code = _dtype_code(q)
    out_code = _out_code(in_code, out_dtype, o)
    dev = q.device
    if o is None:
        o = torch.empty((T, H, dv), dtype=_torch_dtype(out_code), device=dev)
    if want_state and s_final is None:
        s_final = torch.empty((N, H, dv, dk), dtype=torch.float32, device=dev)
    if error is None:
        error = torch.zeros(1, dtype=torch.int32, device=dev)
    st = lib.gdn_recurrent_forward(_ptr(q), _ptr(k), _ptr(v), in_code, _ptr(beta), _ptr(g),
                                   _ptr(cu_seqlens), N, T, H, dk, dv, float(scale), _ptr(h0),
                                   _ptr(o), out_code, _ptr(s_final), _ptr(s_final_scale),
                                   _ptr(error), _stream(stream))
    _check(st, "gdn_recurrent_forward")
    return o, s_final, s_final_scale, error


def recurrent_decode_step(q, k, v, beta, g, s, s_scale, *, scale: float = 1.0, out_dtype=None,
                          o=None, stream=None):
    """gdn_recurrent_decode_step: one token per row b; (s, s_scale) updated in
    place.  q, k, v [B, H, d]; beta, g [B, H].  Returns o [B, H, dv]."""
    B, H, dk = q.shape
    dv = v.shape[2]
    in_code = _dtype_code(q)
    out_code = _out_code(in_code, out_dtype, o)
    if o is None:
        o = torch.empty((B, H, dv), dtype=_torch_dtype(out_code), device=q.device)
    st = lib.gdn_recurrent_decode_step(_ptr(q), _ptr(k), _ptr(v), in_code, _ptr(beta), _ptr(g),
                                       B, H, dk, dv, float(scale), _ptr(s), _ptr(s_scale),
                                       _ptr(o), out_code, _stream(stream))
    _check(st, "gdn_recurrent_decode_step")
    return o


def backward_workspace_bytes(n_seqs: int, total_tokens: int, H: int, dk: int, dv: int,
                             C: int = CHUNK, dtype=torch.bfloat16) -> int:
    code = _dtype_code(torch.empty(0, dtype=dtype))
    return int(lib.gdn_cpr_backward_workspace_bytes(n_seqs, total_tokens, H, dk, dv, C, code))


def backward(q, k, v, beta, g, cu_seqlens, d_o, *, n_seqs: Optional[int] = None, h0=None,
             ds_final=None, C: int = CHUNK, scale: float = 1.0, want_dh0: bool = True,
             grads=None, workspace=None, reuse_forward: bool = False, stream=None,
             kernel_events=None):
    """gdn_cpr_backward.  Returns (grads, workspace); grads is a dict of fp32
    tensors dq, dk, dv [T, H, d], dbeta, dg [T, H] and dh0 [N, H, dv, dk]
    (None unless want_dh0).  Pass ``grads`` (the same dict) to reuse buffers.
    reuse_forward=True (GDN_BWD_REUSE_FORWARD): ``workspace`` was last used by
    forward() on this same batch, whose first pass is then reused.
    kernel_events: 5 recorded torch.cuda.Event objects (gdn_cpr_backward_ex)."""
    T, H, dk = q.shape
    dv = v.shape[2]
    N = (cu_seqlens.numel() - 1) if n_seqs is None else int(n_seqs)
    in_code = _dtype_code(q)
    if d_o.dtype != q.dtype:
        raise ValueError("gdn_cpr: d_o must have the dtype of q, k and v")
    dev = q.device
    if grads is None:
        f32 = dict(dtype=torch.float32, device=dev)
        grads = {"dq": torch.empty((T, H, dk), **f32), "dk": torch.empty((T, H, dk), **f32),
                 "dv": torch.empty((T, H, dv), **f32), "dbeta": torch.empty((T, H), **f32),
                 "dg": torch.empty((T, H), **f32),
                 "dh0": torch.empty((N, H, dv, dk), **f32) if want_dh0 else None}
    need = backward_workspace_bytes(N, T, H, dk, dv, C, q.dtype)
    if workspace is None:
        workspace = torch.zeros(max(need, 256), dtype=torch.uint8, device=dev)
    ev = None
    if kernel_events is not None:
        if len(kernel_events) != 5 or any(e.cuda_event == 0 for e in kernel_events):
            raise ValueError("kernel_events: 5 torch.cuda.Event objects, each recorded once")
        ev = (ctypes.c_void_p * 5)(*[e.cuda_event for e in kernel_events])
    st = lib.gdn_cpr_backward_ex(_ptr(q), _ptr(k), _ptr(v), in_code, _ptr(beta), _ptr(g),
                                 _ptr(cu_seqlens), N, T, H, dk, dv, C, float(scale), _ptr(h0),
                                 _ptr(d_o), _ptr(ds_final), _ptr(grads["dq"]),
                                 _ptr(grads["dk"]), _ptr(grads["dv"]), _ptr(grads["dbeta"]),
                                 _ptr(grads["dg"]), _ptr(grads.get("dh0")), _ptr(workspace),
                                 workspace.numel(), GDN_BWD_REUSE_FORWARD if reuse_forward else 0,
                                 ev, _stream(stream))
    _check(st, "gdn_cpr_backward")
    return grads, workspace


def pik_workspace_bytes(M: int, N: int, K: int, n_leaves: int, n_ranks: int = 1) -> int:
    return int(lib.gdn_pik_workspace_bytes(M, N, K, n_leaves, n_ranks))


def pik_gemm(A, B, n_leaves: int, n_ranks: int = 1, *, C=None, workspace=None, error=None,
             stream=None):
    """gdn_pik_gemm: C = A B^T (A [M, K], B [N, K] bf16; C [M, N] fp32) with K in
    n_leaves contiguous leaves combined by the fixed binary tree, computed in the
    layout of n_ranks emulated ranks.  Returns (C, error word tensor)."""
    if A.dtype != torch.bfloat16 or B.dtype != torch.bfloat16:
        raise ValueError("gdn_pik_gemm: A and B must be bf16")
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K:
        raise ValueError("gdn_pik_gemm: A and B must have the same K")
    dev = A.device
    if C is None:
        C = torch.empty((M, N), dtype=torch.float32, device=dev)
    need = pik_workspace_bytes(M, N, K, n_leaves, n_ranks)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if error is None:
        error = torch.zeros(1, dtype=torch.int32, device=dev)
    st = lib.gdn_pik_gemm(_ptr(A) if K else None, _ptr(B) if K else None, _ptr(C), M, N, K,
                          int(n_leaves), int(n_ranks),
                          _ptr(workspace), 0 if workspace is None else workspace.numel(),
                          _ptr(error), _stream(stream))
    _check(st, "gdn_pik_gemm")
    return C, error


def check_error(error_word: torch.Tensor, stream=None) -> int:
    """gdn_check_error: synchronises, returns the device error bits (and clears them)."""
    bits = ctypes.c_int32(0)
    st = lib.gdn_check_error(_ptr(error_word), ctypes.byref(bits), _stream(stream))
    if st not in (GDN_OK, GDN_ERR_DEVICE_DATA):
        _check(st, "gdn_check_error")
    return int(bits.value)


class DecodeState:
    """Caller-owned decode state (device tensors) for n_slots sequences."""

    def __init__(self, n_slots: int, H: int, dk: int, dv: int, in_dtype=torch.bfloat16,
                 C: int = CHUNK, device="cuda"):
        self.n_slots, self.H, self.dk, self.dv, self.C = n_slots, H, dk, dv, C
        self.in_dtype = in_dtype
        f32 = torch.float32
        self.s_run = torch.zeros((n_slots, H, dv, dk), dtype=f32, device=device)
        self.s_scale = torch.ones((n_slots, H), dtype=f32, device=device)
        self.s_bnd = torch.zeros((n_slots, H, dv, dk), dtype=f32, device=device)
        self.buf_k = torch.zeros((n_slots, H, C, dk), dtype=in_dtype, device=device)
        self.buf_v = torch.zeros((n_slots, H, C, dv), dtype=in_dtype, device=device)
        self.buf_beta = torch.zeros((n_slots, H, C), dtype=f32, device=device)
        self.buf_g = torch.zeros((n_slots, H, C), dtype=f32, device=device)
        self.pos = torch.zeros((n_slots, H), dtype=torch.int32, device=device)
        self.error = torch.zeros((1,), dtype=torch.int32, device=device)
        # work list of the resync inside decode_step (scratch, zero between steps)
        self.resync = torch.zeros((4 + n_slots * H,), dtype=torch.int32, device=device)

    def struct(self) -> DecodeStateStruct:
        return DecodeStateStruct(self.s_run.data_ptr(), self.s_scale.data_ptr(),
                                 self.s_bnd.data_ptr(),
                                 self.buf_k.data_ptr(), self.buf_v.data_ptr(),
                                 self.buf_beta.data_ptr(), self.buf_g.data_ptr(),
                                 self.pos.data_ptr(), self.error.data_ptr(),
                                 self.resync.data_ptr(), self.n_slots)

    def tensors(self):
        return (self.s_run, self.s_scale, self.s_bnd, self.buf_k, self.buf_v, self.buf_beta,
                self.buf_g, self.pos)

    def clone(self) -> "DecodeState":
        c = DecodeState.__new__(DecodeState)
        c.__dict__.update({k: (v.clone() if isinstance(v, torch.Tensor) else v)
                           for k, v in self.__dict__.items()})
        return c


def decode_state_from_prefill(state: DecodeState, k, v, beta, g, cu_seqlens, s_run_final,
                              s_bnd_final, *, s_run_scale=None, slot_idx=None, stream=None):
    N = cu_seqlens.numel() - 1
    T, H, dk = k.shape
    st = lib.gdn_cpr_decode_state_from_prefill(
        _ptr(k), _ptr(v), _dtype_code(k), _ptr(beta), _ptr(g), _ptr(cu_seqlens), N, T, H, dk,
        v.shape[2], state.C, _ptr(s_run_final), _ptr(s_run_scale), _ptr(s_bnd_final),
        _ptr(slot_idx), state.struct(), _stream(stream))
    _check(st, "gdn_cpr_decode_state_from_prefill")


def decode_step(state: DecodeState, q, k, v, beta, g, *, slot_idx=None, scale: float = 1.0,
                out_dtype=None, o=None, stream=None):
    """gdn_cpr_decode_step for B rows: q,k [B,H,dk], v [B,H,dv], beta,g [B,H]."""
    B, H, dk = q.shape
    dv = v.shape[2]
    in_code = _dtype_code(q)
    out_code = _out_code(in_code, out_dtype, o)
    if o is None:
        o = torch.empty((B, H, dv), dtype=_torch_dtype(out_code), device=q.device)
    st = lib.gdn_cpr_decode_step(_ptr(q), _ptr(k), _ptr(v), in_code, _ptr(beta), _ptr(g),
                                 _ptr(slot_idx), B, H, dk, dv, state.C, float(scale),
                                 state.struct(), _ptr(o), out_code, _stream(stream))
    _check(st, "gdn_cpr_decode_step")
    return o


def chunk_boundary(s_start, k, v, beta, g, *, s_end=None, stream=None):
    """gdn_chunk_boundary: k [B,H,C,dk], v [B,H,C,dv], beta,g [B,H,C]; s [B,H,dv,dk]."""
    B, H, C, dk = k.shape
    dv = v.shape[3]
    if s_end is None:
        s_end = torch.empty_like(s_start)
    st = lib.gdn_chunk_boundary(_ptr(s_start), _ptr(k), _ptr(v), _dtype_code(k), _ptr(beta),
                                _ptr(g), B, H, dk, dv, C, _ptr(s_end), _stream(stream))
    _check(st, "gdn_chunk_boundary")
    return s_end


# ---------------------------------------------------------------------------
# q/k norm and gated linear recurrence (gdn_qk_norm.h, gdn_glr.h)
# ---------------------------------------------------------------------------
# These calls take strided rows, run on the device of their tensors (current
# or not) and check every tensor's shape, dtype and device here, since the C
# entry points see bare pointers.

class _Call:
    """Device, stream and checks of one call.  (These run in front of kernels of a few
    microseconds: messages are put together only when a check has failed.)"""

    __slots__ = ("what", "index", "dev", "user_stream", "raw")

    def __init__(self, what: str, t: torch.Tensor, stream):
        if not t.is_cuda:
            raise ValueError("gdn_cpr: tensors must be on a CUDA device (there is no CPU path)")
        self.what = what
        self.dev = t.device
        self.index = t.get_device()
        self.user_stream = stream
        if stream is None:
            self.raw = torch._C._cuda_getCurrentRawStream(self.index)
        else:
            self.raw = stream.cuda_stream
            self.need(stream.device_index == self.index,
                      "stream and tensors are on different devices")

    def need(self, ok: bool, why: str):
        if not ok:
            raise ValueError(f"{self.what}: {why}")

    def empty(self, shape, dtype):
        """New memory for an output or scratch, used on the call's stream."""
        t = torch.empty(*shape, dtype=dtype, device=self.dev)  # (a tuple takes twice as long)
        if self.user_stream is not None:
            # the memory may have been freed on the current stream, whose work on it
            # is waited for; and it is kept from reuse until the call's stream is done
            self.user_stream.wait_stream(torch.cuda.current_stream(self.dev))
            t.record_stream(self.user_stream)
        return t

    def full(self, t, name: str, shape, dtype):
        """Address of a contiguous tensor (None stays NULL)."""
        if t is None:
            return None
        if (t.get_device() != self.index or t.dtype != dtype or t.shape != shape
                or not t.is_contiguous()):
            self.need(t.device == self.dev, f"{name} is on {t.device}, not {self.dev}")
            self.need(t.dtype == dtype, f"{name} must be {dtype}")
            self.need(t.shape == shape, f"{name} must have shape {tuple(shape)}")
            self.need(False, f"{name} must be contiguous")
        return t.data_ptr()

    def rows(self, t, name: str, shape, dtype=None):
        """Address and row stride of [T, ...] whose rows are contiguous."""
        if t.get_device() != self.index or t.shape != shape or (dtype is not None
                                                                and t.dtype != dtype):
            self.need(t.device == self.dev, f"{name} is on {t.device}, not {self.dev}")
            self.need(t.shape == shape, f"{name} must have shape {tuple(shape)}")
            self.need(False, f"{name} must be {dtype}")
        step, width = t.stride(), shape[-1]
        ok = step[-1] == 1 or width <= 1
        if len(shape) == 3:
            ok = ok and (step[1] == width or shape[1] <= 1)
            width *= shape[1]
        if not ok:
            self.need(False, f"the rows of {name} must be contiguous")
        return t.data_ptr(), (step[0] if shape[0] > 1 else width)

    def out_full(self, t, want: bool, name: str, shape, dtype):
        """An output: the caller's (checked), a new one if wanted, or None."""
        if t is not None:
            return t, self.full(t, name, shape, dtype)
        if not want:
            return None, None
        t = self.empty(shape, dtype)
        return t, t.data_ptr()

    def out_rows(self, t, name: str, shape, dtype):
        """The same for strided rows, which are always wanted."""
        if t is not None:
            return t, *self.rows(t, name, shape, dtype)
        t = self.empty(shape, dtype)
        return t, t.data_ptr(), (shape[1] if len(shape) == 2 else shape[1] * shape[2])

    def run(self, fn, *args):
        if self.index == torch._C._cuda_getDevice():
            st = fn(*args, self.raw)
        else:
            with torch.cuda.device(self.index):
                st = fn(*args, self.raw)
        if st != GDN_OK:
            raise GdnError(st, self.what)


def _dtype_of(code_or_dtype, default):
    if code_or_dtype is None:
        return default
    if code_or_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"gdn_cpr: unsupported dtype {code_or_dtype}")
    return code_or_dtype


def _norm_kind(norm: str) -> int:
    if norm not in ("l2", "rms"):
        raise ValueError("norm must be 'l2' or 'rms'")
    return GDN_QK_NORM_RMS if norm == "rms" else GDN_QK_NORM_L2


def _qk_call(what, q, k, norm, wq, wk, positions, inv_freq, stream):
    some = q if q is not None else k
    if (some is None or some.dim() != 3) or (k is not None and k.dim() != 3):
        raise ValueError(f"{what}: q, k must be [tokens, heads, d] (one of them may be None)")
    c = _Call(what, some, stream)
    T, _, d = some.shape
    Hq = 0 if q is None else q.shape[1]
    Hk = 0 if k is None else k.shape[1]
    qp, ldq = (None, 0) if q is None else c.rows(q, "q", (T, Hq, d))
    kp, ldk = (None, 0) if k is None else c.rows(k, "k", (T, Hk, d), some.dtype)
    c.need((positions is None) == (inv_freq is None), "positions and inv_freq go together")
    F = 0
    if inv_freq is not None:
        F = inv_freq.numel()
        c.full(inv_freq, "inv_freq", (F,), torch.float32)
        c.full(positions, "positions", (T,), torch.int32)
    head = (qp, ldq, kp, ldk, _dtype_code(some), T, Hq, Hk, d, _norm_kind(norm))
    tail = (c.full(wq, "wq", (d,), torch.float32), c.full(wk, "wk", (d,), torch.float32),
            None if F == 0 else positions.data_ptr(), None if F == 0 else inv_freq.data_ptr(),
            2 * F)
    return c, some.dtype, (T, Hq, Hk, d), head, tail


def qk_norm_forward(q, k, *, norm: str = "l2", eps: float = 1e-6, wq=None, wk=None,
                    positions=None, inv_freq=None, interleaved: bool = False, out_dtype=None,
                    oq=None, ok=None, stream=None):
    """gdn_qk_norm_forward: every head of q [T, Hq, d] and k [T, Hk, d] normalised
    (norm "l2" or "rms", fp32 weights wq, wk [d] or None) and, with positions [T]
    int32 and inv_freq [rot_dim / 2] fp32, rotated.  Tokens may be strided; q or
    k may be None.  oq=q, ok=k works in place.  Returns (oq, ok)."""
    c, dt, (T, Hq, Hk, d), head, tail = _qk_call("gdn_qk_norm_forward", q, k, norm, wq, wk,
                                                 positions, inv_freq, stream)
    given = oq if oq is not None else ok
    odt = _dtype_of(out_dtype, given.dtype if given is not None else dt)
    out = []
    for x, o, H, name in ((q, oq, Hq, "oq"), (k, ok, Hk, "ok")):
        if x is None:
            out += [None, None, 0]
            continue
        out += c.out_rows(o, name, (T, H, d), odt)
    c.run(lib.gdn_qk_norm_forward, *head, float(eps), *tail, int(bool(interleaved)), out[1],
          out[2], out[4], out[5], _dtype_code_of(odt))
    return out[0], out[3]


def qk_norm_backward_workspace_bytes(T: int, Hq: int, Hk: int, d: int) -> int:
    return int(lib.gdn_qk_norm_backward_workspace_bytes(T, Hq, Hk, d))


def qk_norm_backward(q, k, d_oq, d_ok, *, norm: str = "l2", eps: float = 1e-6, wq=None, wk=None,
                     positions=None, inv_freq=None, interleaved: bool = False,
                     want_dw: bool = True, grads=None, workspace=None, stream=None):
    """gdn_qk_norm_backward: q, k and the options of the forward; d_oq, d_ok of
    one dtype (bf16 or fp32, the fp32 of backward()'s dq and dk for one).  Returns
    a dict of dq, dk (the dtype of q and k) and dwq, dwk [d] fp32 (None without
    the weight or want_dw).  Pass ``grads`` (such a dict) to reuse its buffers; what
    it lacks is allocated as without it."""
    c, dt, (T, Hq, Hk, d), head, tail = _qk_call("gdn_qk_norm_backward", q, k, norm, wq, wk,
                                                 positions, inv_freq, stream)
    c.need((q is None) == (d_oq is None) and (k is None) == (d_ok is None),
           "d_oq and d_ok go with q and k")
    gdt = (d_oq if q is not None else d_ok).dtype
    gin, gout, res = [], [], {}
    for s, x, g, H in (("q", q, d_oq, Hq), ("k", k, d_ok, Hk)):
        if x is None:
            gin += [None, 0]
            gout += [None, 0]
            res["d" + s] = None
            continue
        gin += [*c.rows(g, "d_o" + s, (T, H, d), gdt)]
        given = grads.get("d" + s) if grads is not None else None
        res["d" + s], *at = c.out_rows(given, "d" + s, (T, H, d), dt)
        gout += at
    for s, w in (("q", wq), ("k", wk)):
        given = grads.get("dw" + s) if grads is not None and w is not None and want_dw else None
        res["dw" + s], at = c.out_full(given, w is not None and want_dw, "dw" + s, (d,),
                                       torch.float32)
        gout.append(at)
    need = 0
    if res["dwq"] is not None or res["dwk"] is not None:
        need = qk_norm_backward_workspace_bytes(T, Hq, Hk, d)
        if workspace is None:
            workspace = c.empty((max(need, 16),), torch.uint8)
    size = 0
    if workspace is not None:
        size = workspace.numel() * workspace.element_size()
        c.need(workspace.device == c.dev and workspace.is_contiguous(),
               "workspace must be contiguous and on the device of q and k")
    c.run(lib.gdn_qk_norm_backward, *head, float(eps), *tail, int(bool(interleaved)), *gin,
          _dtype_code_of(gdt), *gout, None if workspace is None else workspace.data_ptr(), size)
    return res


_CODES = {torch.bfloat16: GDN_BF16, torch.float32: GDN_F32}


def _dtype_code_of(dtype) -> int:
    code = _CODES.get(dtype)
    if code is None:
        raise ValueError(f"gdn_cpr: unsupported dtype {dtype}")
    return code


class GlrDecodeState:
    """Caller-owned decode state (device tensors) of the gated linear recurrence
    for n_slots sequences; a new one starts every slot from a zero state."""

    def __init__(self, n_slots: int, D: int, device="cuda"):
        self.n_slots, self.D = n_slots, D
        f32 = torch.float32
        self.h = torch.zeros((n_slots, D), dtype=f32, device=device)
        self.a = torch.ones((n_slots, D), dtype=f32, device=device)
        self.b = torch.zeros((n_slots, D), dtype=f32, device=device)
        self.pos = torch.zeros((n_slots,), dtype=torch.int32, device=device)
        self.error = torch.zeros((1,), dtype=torch.int32, device=device)

    def tensors(self):
        return (self.h, self.a, self.b, self.pos)

    def clone(self) -> "GlrDecodeState":
        c = GlrDecodeState.__new__(GlrDecodeState)
        c.__dict__.update({k: (v.clone() if isinstance(v, torch.Tensor) else v)
                           for k, v in self.__dict__.items()})
        return c


def _glr_state(c: _Call, state: GlrDecodeState, D: int) -> GlrStateStruct:
    n = state.n_slots
    shape = (n, D)
    return GlrStateStruct(c.full(state.h, "state.h", shape, torch.float32),
                          c.full(state.a, "state.a", shape, torch.float32),
                          c.full(state.b, "state.b", shape, torch.float32),
                          c.full(state.pos, "state.pos", (n,), torch.int32),
                          c.full(state.error, "state.error", (1,), torch.int32), n)


def _glr_inputs(c: _Call, x, g):
    T, D = x.shape
    xp, ldx = c.rows(x, "x", (T, D))
    gp, ldg = c.rows(g, "g", (T, D))
    return xp, ldx, _dtype_code(x), gp, ldg, _dtype_code(g)


def _glr_mode(complement: bool) -> int:
    return GDN_GLR_INPUT_COMPLEMENT if complement else GDN_GLR_INPUT_PLAIN


def _glr_batch(c: _Call, cu_seqlens, n_seqs):
    N = cu_seqlens.numel() - 1 if n_seqs is None else int(n_seqs)
    c.need(0 <= N < max(cu_seqlens.numel(), 1), "cu_seqlens has n_seqs + 1 entries")
    return N, c.full(cu_seqlens, "cu_seqlens", (cu_seqlens.numel(),), torch.int32)


def glr_carry_rows(n_seqs: int, total_tokens: int) -> int:
    return int(lib.gdn_glr_carry_rows(n_seqs, total_tokens))


def glr_forward(x, g, cu_seqlens, *, n_seqs: Optional[int] = None, h0=None,
                complement: bool = False, out_dtype=None, h=None, s_final=None,
                want_state: bool = True, state: Optional[GlrDecodeState] = None, slot_idx=None,
                carry=None, want_carry: bool = False, error=None, stream=None):
    """gdn_glr_forward: h_t = exp(g_t) h_{t-1} + x_t for every channel of packed
    sequences (complement: + (1 - exp(g_t)) x_t).  x, g [T, D], rows may be
    strided; h0, s_final [N, D] fp32.  Gates that grow must not sum to 88 or more
    within a chunk of 16 tokens.  ``state`` (and slot_idx) receives the
    decode state of every sequence; want_carry=True returns the fp32 rows that
    glr_backward needs.  Returns (h, s_final, carry, error word)."""
    c = _Call("gdn_glr_forward", x, stream)
    c.need(x.dim() == 2 and g.dim() == 2, "x, g must be [tokens, channels]")
    T, D = x.shape
    ins = _glr_inputs(c, x, g)
    N, cu = _glr_batch(c, cu_seqlens, n_seqs)
    odt = _dtype_of(out_dtype, h.dtype if h is not None else x.dtype)
    f32 = torch.float32
    rows = glr_carry_rows(N, T)
    h, hp, ldh = c.out_rows(h, "h", (T, D), odt)
    s_final, fin = c.out_full(s_final, want_state, "s_final", (N, D), f32)
    carry, car = c.out_full(carry, want_carry, "carry", (rows, D), f32)
    error, err = c.out_full(error, True, "error", (1,), torch.int32)
    st = None if state is None else ctypes.byref(_glr_state(c, state, D))
    c.run(lib.gdn_glr_forward, *ins, cu, N, T, D, _glr_mode(complement),
          c.full(h0, "h0", (N, D), f32), hp, ldh, _dtype_code_of(odt), fin, st,
          c.full(slot_idx, "slot_idx", (N,), torch.int32), car, err)
    return h, s_final, carry, error


def glr_backward(x, g, cu_seqlens, carry, d_h, *, n_seqs: Optional[int] = None, ds_final=None,
                 complement: bool = False, want_dh0: bool = True, grads=None, error=None,
                 stream=None):
    """gdn_glr_backward: x, g, cu_seqlens and options of the forward that wrote
    ``carry``; d_h [T, D] (bf16 or fp32).  Returns (grads, error word); grads is
    a dict of dx, dg [T, D] (the dtypes of x and g) and dh0 [N, D] fp32 (None
    unless want_dh0).  Pass ``grads`` (such a dict) to reuse its buffers; what it
    lacks is allocated and put into it."""
    c = _Call("gdn_glr_backward", x, stream)
    c.need(x.dim() == 2 and g.dim() == 2, "x, g must be [tokens, channels]")
    T, D = x.shape
    ins = _glr_inputs(c, x, g)
    N, cu = _glr_batch(c, cu_seqlens, n_seqs)
    dhp, lddh = c.rows(d_h, "d_h", (T, D))
    c.need(carry is not None, "carry is the forward's (want_carry=True)")
    car = c.full(carry, "carry", (glr_carry_rows(N, T), D), torch.float32)
    if grads is None:
        grads = {}
    dx, dxp, lddx = c.out_rows(grads.get("dx"), "dx", (T, D), x.dtype)
    dg, dgp, lddg = c.out_rows(grads.get("dg"), "dg", (T, D), g.dtype)
    dh0, dhp0 = c.out_full(grads.get("dh0"), want_dh0, "dh0", (N, D), torch.float32)
    grads.update(dx=dx, dg=dg, dh0=dh0)
    error, err = c.out_full(error, True, "error", (1,), torch.int32)
    c.run(lib.gdn_glr_backward, *ins, cu, N, T, D, _glr_mode(complement), car, dhp, lddh,
          _dtype_code(d_h), c.full(ds_final, "ds_final", (N, D), torch.float32), dxp, lddx, dgp,
          lddg, dhp0, err)
    return grads, error


def glr_decode_step(state: GlrDecodeState, x, g, *, slot_idx=None, complement: bool = False,
                    out_dtype=None, h=None, stream=None):
    """gdn_glr_decode_step for B rows: x, g [B, D]; row b advances slot slot_idx[b]
    (int32; slot b without it).  Returns h [B, D]; bad rows set state.error."""
    c = _Call("gdn_glr_decode_step", x, stream)
    c.need(x.dim() == 2 and g.dim() == 2, "x, g must be [rows, channels]")
    B, D = x.shape
    ins = _glr_inputs(c, x, g)
    odt = _dtype_of(out_dtype, h.dtype if h is not None else x.dtype)
    h, hp, ldh = c.out_rows(h, "h", (B, D), odt)
    c.run(lib.gdn_glr_decode_step, *ins, c.full(slot_idx, "slot_idx", (B,), torch.int32), B, D,
          _glr_mode(complement), _glr_state(c, state, D), hp, ldh, _dtype_code_of(odt))
    return h


def _dt(dtype) -> int:
    return GDN_BF16 if dtype == torch.bfloat16 else GDN_F32 if dtype == torch.float32 else -1


def contract_descriptor(kind: int, in_dtype=torch.bfloat16, out_dtype=torch.bfloat16, dk: int = 128,
                        dv: int = 128, C: int = CHUNK) -> str:
    """gdn_cpr_contract_descriptor: the canonical text a digest hashes."""
    n = ctypes.c_size_t(0)
    args = (kind, _dt(in_dtype), _dt(out_dtype), dk, dv, C)
    _check(lib.gdn_cpr_contract_descriptor(*args, None, 0, ctypes.byref(n)),
           "gdn_cpr_contract_descriptor")
    buf = ctypes.create_string_buffer(n.value + 1)
    _check(lib.gdn_cpr_contract_descriptor(*args, buf, n.value + 1, ctypes.byref(n)),
           "gdn_cpr_contract_descriptor")
    return buf.value.decode()


def contract_digest(kind: int, in_dtype=torch.bfloat16, out_dtype=torch.bfloat16, dk: int = 128,
                    dv: int = 128, C: int = CHUNK) -> bytes:
    """gdn_cpr_contract_digest: 32-byte SHA-256 identity digest."""
    out = ctypes.create_string_buffer(32)
    _check(lib.gdn_cpr_contract_digest(kind, _dt(in_dtype), _dt(out_dtype), dk, dv, C, out),
           "gdn_cpr_contract_digest")
    return out.raw


def contract_check(peer_policy: bytes, in_dtype=torch.bfloat16, out_dtype=torch.bfloat16,
                   dk: int = 128, dv: int = 128, C: int = CHUNK) -> int:
    """gdn_cpr_contract_check: GDN_OK, or GDN_ERR_CONTRACT when the policies differ."""
    if len(peer_policy) != 32:
        raise ValueError("a digest is 32 bytes")
    return lib.gdn_cpr_contract_check(peer_policy, _dt(in_dtype), _dt(out_dtype), dk, dv, C)


def sha256(data: bytes) -> bytes:
    """gdn_sha256 of a byte string."""
    out = ctypes.create_string_buffer(32)
    _check(lib.gdn_sha256(data, len(data), out), "gdn_sha256")
    return out.raw
