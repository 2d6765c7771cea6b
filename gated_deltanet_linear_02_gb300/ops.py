"""Thin ctypes binding of libgdn.so (include/gdn.h), with the same names.

This layer only marshals arguments. It checks the tensors' shapes, dtypes,
devices and contiguity, passes their device pointers and the current CUDA
stream, and turns a non-OK status into ``GdnError``. Every step of the mixer
runs in the library's CUDA kernels. If the library is missing, loading fails
loudly: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import inputs as _inp

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgdn.so")

GDN_OK, GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED, GDN_ERR_WORKSPACE, GDN_ERR_CUDA, GDN_ERR_TIMEOUT = range(6)
GDN_F32, GDN_BF16 = 0, 1
_DT = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16}

HV, HK, DK, DV, KC, CC, DI = _inp.HV, _inp.HK, _inp.DK, _inp.DV, _inp.KCONV, _inp.C_CONV, _inp.D_INNER
N_EMBD = _inp.N_EMBD


class GdnError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}" + (f" ({detail})" if detail else ""))


class gdn_params(ctypes.Structure):
    _fields_ = [("conv_w", ctypes.c_void_p), ("A_log", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p),
                ("norm_w", ctypes.c_void_p), ("norm_eps", ctypes.c_float), ("l2_eps", ctypes.c_float)]


class gdn_attn_params(ctypes.Structure):
    _fields_ = [("q_norm_w", ctypes.c_void_p), ("k_norm_w", ctypes.c_void_p), ("rope", ctypes.c_void_p),
                ("n_pos", ctypes.c_int), ("norm_eps", ctypes.c_float)]


class gdn_norm_params(ctypes.Structure):
    _fields_ = [("norm_w", ctypes.c_void_p), ("post_w", ctypes.c_void_p), ("res_scale", ctypes.c_float),
                ("norm_eps", ctypes.c_float)]


class gdn_moe_params(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("router", "gate", "up", "down", "sh_gate", "sh_up", "sh_down", "sh_router")] + \
        [(n, ctypes.c_int) for n in ("num_experts", "top_k", "ffn_dim", "norm_topk")]


class gdn_kv_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("num_pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("format", ctypes.c_int)]


class gdn_paged_batch(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("ctx_len", ctypes.c_void_p), ("cu_q", ctypes.c_void_p),
                ("B", ctypes.c_int), ("M", ctypes.c_int), ("max_q", ctypes.c_int), ("max_pages", ctypes.c_int)]


_lib = None
_vp, _int, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t


def lib() -> ctypes.CDLL:
    """The loaded libgdn.so. Raises if it has not been built: the mixer has
    no CPU or library fallback."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'` (nvcc, sm_103a)")
        L = ctypes.CDLL(LIB_PATH)
        L.gdn_conv_step.restype = _int
        L.gdn_conv_step.argtypes = [_vp, _vp, _vp, _vp, _int, _int, _vp]
        L.gdn_decode_step.restype = _int
        L.gdn_decode_step.argtypes = [ctypes.POINTER(gdn_params)] + [_vp] * 7 + [_int, _int, _int, _vp]
        L.gdn_decode_multi.restype = _int
        L.gdn_decode_multi.argtypes = [ctypes.POINTER(gdn_params)] + [_vp] * 7 + [_int, _int, _int, _int, _vp]
        L.gdn_in_proj.restype = _int
        L.gdn_in_proj.argtypes = [_vp] * 6 + [_int, _int, _vp]
        L.gdn_out_proj.restype = _int
        L.gdn_out_proj.argtypes = [_vp, _vp, _vp, _int, _int, _vp]
        L.gdn_in_proj_conv.restype = _int
        L.gdn_in_proj_conv.argtypes = [ctypes.POINTER(gdn_params), _vp, _vp, _vp, _int, _int] + [_vp] * 6 + [_vp]
        L.gdn_prefill_xhat.restype = _int
        L.gdn_prefill_xhat.argtypes = [ctypes.POINTER(gdn_params)] + [_vp] * 5 + [_int, _int] + [_vp] * 3 + \
            [_int, _vp, _sz, _vp]
        L.gdn_gated_out_proj.restype = _int
        L.gdn_gated_out_proj.argtypes = [_vp, ctypes.c_float, _vp, _vp, _vp, _vp, _int, _int, _int, _vp]
        L.gdn_prefill.restype = _int
        L.gdn_prefill.argtypes = [ctypes.POINTER(gdn_params)] + [_vp] * 5 + [_int, _int] + [_vp] * 5 + \
            [_int, _int, _int, _vp, _sz, _vp]
        L.gdn_prefill_static.restype = _int
        L.gdn_prefill_static.argtypes = [ctypes.POINTER(gdn_params)] + [_vp] * 5 + [_int, _int] + [_vp] * 5 + \
            [_int, _int, _int, _vp]
        L.gdn_attn_decode.restype = _int
        L.gdn_attn_decode.argtypes = [_vp] * 6 + [_int, _int, _vp, _sz, _int, _vp]
        L.gdn_attn_decode_workspace_size.restype = _sz
        L.gdn_attn_decode_workspace_size.argtypes = [_int, _int]
        _ll = ctypes.c_longlong
        L.gdn_attn_qk_norm_rope.restype = _int
        L.gdn_attn_qk_norm_rope.argtypes = [_vp, _vp, _ll, _ll, _vp, _ll, _ll, _vp, _int, _vp, _vp, _int, _int, _vp]
        L.gdn_kv_append.restype = _int
        L.gdn_kv_append.argtypes = [_vp, _vp, _vp] + [_vp, _ll, _ll] * 3 + [_vp, _vp, _int, _vp]
        L.gdn_kv_gather.restype = _int
        L.gdn_kv_gather.argtypes = [_vp, _vp, _vp, _vp, _int, _vp]
        L.gdn_attn_paged.restype = _int
        L.gdn_attn_paged.argtypes = [_vp, _vp, _vp, _vp, _ll, _ll, _vp, _vp, _sz, _int, _vp]
        L.gdn_attn_paged_workspace_size.restype = _sz
        L.gdn_attn_paged_workspace_size.argtypes = [_vp, _vp]
        L.gdn_add_norm.restype = _int
        L.gdn_add_norm.argtypes = [_vp] + [_vp, _ll] * 5 + [_int, _int, _int, _vp]
        L.gdn_linear.restype = _int
        L.gdn_linear.argtypes = [_vp, _ll, _vp, _vp, _vp, _ll, _vp, _ll] + [_int] * 5 + [_vp]
        L.gdn_moe_route.restype = _int
        L.gdn_moe_route.argtypes = [_vp, _vp, _ll, _int, _vp, _vp, _vp]
        L.gdn_moe.restype = _int
        L.gdn_moe.argtypes = [_vp, _vp, _ll, _vp, _vp, _int, _vp, _vp, _vp, _sz, _int, _vp]
        L.gdn_moe_workspace_size.restype = _sz
        L.gdn_moe_workspace_size.argtypes = [_vp, _int]
        L.gdn_prefill_workspace_size.restype = _sz
        L.gdn_prefill_workspace_size.argtypes = [_int, _int, _int, _int]
        L.gdn_selftest_wait_timeout.restype = _int
        L.gdn_selftest_wait_timeout.argtypes = [_vp]
        L.gdn_selftest_moe_lost_route.restype = _int
        L.gdn_selftest_moe_lost_route.argtypes = [_vp, _vp, _ll, _vp, _vp, _int, _vp, _sz, _int, _vp]
        L.gdn_device_error.restype = _int
        L.gdn_device_error.argtypes = [_vp]
        L.gdn_get_device_error.restype = _int
        L.gdn_get_device_error.argtypes = [_vp, _vp]
        L.gdn_status_string.restype = ctypes.c_char_p
        L.gdn_status_string.argtypes = [_int]
        L.gdn_last_error.restype = ctypes.c_char_p
        L.gdn_last_error.argtypes = []
        L.gdn_abi_version.restype = _int
        L.gdn_abi_version.argtypes = []
        _lib = L
    return _lib


def status_string(s: int) -> str:
    return lib().gdn_status_string(int(s)).decode()


def last_error() -> str:
    return lib().gdn_last_error().decode()


def abi_version() -> int:
    return lib().gdn_abi_version()


def _check(status: int, where: str):
    if status != GDN_OK:
        raise GdnError(status, where, last_error())


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if isinstance(stream, torch.cuda.Stream) else int(stream)


def _ptr(t: torch.Tensor | None, name: str, shape=None, dtype=None, device=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def make_params(p) -> gdn_params:
    """gdn_params from anything with conv_w, A_log, dt_bias, norm_w fp32 CUDA
    tensors and norm_eps, l2_eps floats (e.g. inputs.LayerParams).

    The struct holds raw device pointers, so it also keeps references to the
    four tensors: they stay alive as long as the struct does, even when the
    caller passed a temporary such as ``make_params(lp.to("cuda"))``."""
    cp = gdn_params(_ptr(p.conv_w, "conv_w", (CC, KC), torch.float32),
                    _ptr(p.A_log, "A_log", (HV,), torch.float32),
                    _ptr(p.dt_bias, "dt_bias", (HV,), torch.float32),
                    _ptr(p.norm_w, "norm_w", (DV,), torch.float32),
                    float(p.norm_eps), float(p.l2_eps))
    cp._keep_alive = (p.conv_w, p.A_log, p.dt_bias, p.norm_w)
    return cp


def _act_dtype(t: torch.Tensor) -> int:
    if t.dtype not in _DT:
        raise ValueError(f"activation dtype {t.dtype} unsupported (float32 or bfloat16)")
    return _DT[t.dtype]


def conv_step(conv_w, qkv_in, qkv_out, conv_state, stream=None):
    """gdn_conv_step: qkv_out = SiLU(causal conv(conv_state, qkv_in)); conv_state shifts."""
    B = qkv_in.shape[0]
    act = _act_dtype(qkv_in)
    st = lib().gdn_conv_step(_ptr(conv_w, "conv_w", (CC, KC), torch.float32),
                             _ptr(qkv_in, "qkv_in", (B, CC)), _ptr(qkv_out, "qkv_out", (B, CC), qkv_in.dtype),
                             _ptr(conv_state, "conv_state", (B, KC - 1, CC), qkv_in.dtype), B, act,
                             _stream(stream))
    _check(st, "gdn_conv_step")


def decode_step(params, qkv, z, alpha, beta, conv_state, ssm_state, out, stream=None,
                cparams: gdn_params | None = None):
    """gdn_decode_step: one token for B sequences, states updated in place."""
    B = qkv.shape[0]
    dt = qkv.dtype
    act = _act_dtype(qkv)
    od = _act_dtype(out)
    cp = cparams if cparams is not None else make_params(params)
    st = lib().gdn_decode_step(ctypes.byref(cp), _ptr(qkv, "qkv", (B, CC)), _ptr(z, "z", (B, DI), dt),
                               _ptr(alpha, "alpha", (B, HV), dt), _ptr(beta, "beta", (B, HV), dt),
                               _ptr(conv_state, "conv_state", (B, KC - 1, CC), dt),
                               _ptr(ssm_state, "ssm_state", (B, HV, DV, DK), torch.float32),
                               _ptr(out, "out", (B, DI)), B, act, od, _stream(stream))
    _check(st, "gdn_decode_step")


def decode_multi(params, qkv, z, alpha, beta, conv_state, ssm_state, out, stream=None,
                 cparams: gdn_params | None = None):
    """gdn_decode_multi: T consecutive tokens for each of B sequences (qkv
    [B][T][8192]), states updated in place."""
    B, T = qkv.shape[0], qkv.shape[1]
    dt = qkv.dtype
    act = _act_dtype(qkv)
    od = _act_dtype(out)
    cp = cparams if cparams is not None else make_params(params)
    st = lib().gdn_decode_multi(ctypes.byref(cp), _ptr(qkv, "qkv", (B, T, CC)), _ptr(z, "z", (B, T, DI), dt),
                                _ptr(alpha, "alpha", (B, T, HV), dt), _ptr(beta, "beta", (B, T, HV), dt),
                                _ptr(conv_state, "conv_state", (B, KC - 1, CC), dt),
                                _ptr(ssm_state, "ssm_state", (B, HV, DV, DK), torch.float32),
                                _ptr(out, "out", (B, T, DI)), B, T, act, od, _stream(stream))
    _check(st, "gdn_decode_multi")


IN_PROJ_ROWS = CC + DI + 2 * HV   # GDN_IN_PROJ_ROWS


def in_proj(h, w_in, qkv, z, alpha, beta, stream=None):
    """gdn_in_proj: the four input projections of the normed hidden states h
    [M][2048] (bf16) through the stacked weight w_in [12352][2048] (bf16), into
    qkv [M][8192], z [M][4096], alpha [M][32], beta [M][32] (fp32 or bf16)."""
    M = h.shape[0]
    act = _act_dtype(qkv)
    dt = qkv.dtype
    st = lib().gdn_in_proj(_ptr(h, "h", (M, N_EMBD), torch.bfloat16),
                           _ptr(w_in, "w_in", (IN_PROJ_ROWS, N_EMBD), torch.bfloat16),
                           _ptr(qkv, "qkv", (M, CC)), _ptr(z, "z", (M, DI), dt), _ptr(alpha, "alpha", (M, HV), dt),
                           _ptr(beta, "beta", (M, HV), dt), M, act, _stream(stream))
    _check(st, "gdn_in_proj")


def out_proj(x, w, y, stream=None):
    """gdn_out_proj: y = x w^T on the tensor cores (x [M][4096] bf16, w
    [2048][4096] bf16, y [M][2048] fp32 or bf16)."""
    M = x.shape[0]
    od = _act_dtype(y)
    st = lib().gdn_out_proj(_ptr(x, "x", (M, DI), torch.bfloat16), _ptr(w, "w", (N_EMBD, DI), torch.bfloat16),
                            _ptr(y, "y", (M, N_EMBD)), M, od, _stream(stream))
    _check(st, "gdn_out_proj")


def in_proj_conv(params, h, w_in, cu_seqlens, xhat, z, alpha, beta, conv_state_in=None, conv_state_out=None,
                 stream=None, cparams: gdn_params | None = None):
    """gdn_in_proj_conv: the input projections with the conv, SiLU and q/k L2
    norms in the GEMM's epilogue (h [M][2048] bf16, w_in [12352][2048] bf16)
    into xhat [M][8192] fp16, z [M][4096], alpha/beta [M][32] bf16, and
    conv_state_out [N][3][8192] bf16."""
    M = h.shape[0]
    N = cu_seqlens.shape[0] - 1
    cp = cparams if cparams is not None else make_params(params)
    st = lib().gdn_in_proj_conv(ctypes.byref(cp), _ptr(h, "h", (M, N_EMBD), torch.bfloat16),
                                _ptr(w_in, "w_in", (IN_PROJ_ROWS, N_EMBD), torch.bfloat16),
                                _ptr(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32), N, M,
                                _ptr(conv_state_in, "conv_state_in", (N, KC - 1, CC), torch.bfloat16),
                                _ptr(conv_state_out, "conv_state_out", (N, KC - 1, CC), torch.bfloat16),
                                _ptr(xhat, "xhat", (M, CC), torch.float16), _ptr(z, "z", (M, DI), torch.bfloat16),
                                _ptr(alpha, "alpha", (M, HV), torch.bfloat16), _ptr(beta, "beta", (M, HV), torch.bfloat16),
                                _stream(stream))
    _check(st, "gdn_in_proj_conv")


def prefill_xhat(params, xhat, z, alpha, beta, cu_seqlens, out, ssm_state_in=None, ssm_state_out=None,
                 workspace=None, stream=None, cparams: gdn_params | None = None):
    """gdn_prefill_xhat: the chunked prefill from gdn_in_proj_conv's activations.
    Allocates the workspace through torch when none is given."""
    T = xhat.shape[0]
    N = cu_seqlens.shape[0] - 1
    if workspace is None:
        workspace = torch.empty(max(prefill_workspace_size(N, T, torch.bfloat16, 64), 256), dtype=torch.uint8,
                                device=xhat.device)
    cp = cparams if cparams is not None else make_params(params)
    st = lib().gdn_prefill_xhat(ctypes.byref(cp), _ptr(xhat, "xhat", (T, CC), torch.float16),
                                _ptr(z, "z", (T, DI), torch.bfloat16), _ptr(alpha, "alpha", (T, HV), torch.bfloat16),
                                _ptr(beta, "beta", (T, HV), torch.bfloat16),
                                _ptr(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32), N, T,
                                _ptr(ssm_state_in, "ssm_state_in", (N, HV, DV, DK), torch.float32),
                                _ptr(ssm_state_out, "ssm_state_out", (N, HV, DV, DK), torch.float32),
                                _ptr(out, "out", (T, DI)), _act_dtype(out), _ptr(workspace, "workspace"),
                                workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "gdn_prefill_xhat")
    return workspace


def gated_out_proj(norm_w, norm_eps, y, z, w, out, stream=None):
    """gdn_gated_out_proj: out = (gated RMSNorm(y) . silu(z)) w^T in one
    tensor-core GEMM. y and z [M][4096] in the same dtype (fp32 or bf16; y is
    the mixer's output with the norm left out), norm_w [128] fp32, w
    [2048][4096] bf16, out [M][2048] fp32 or bf16."""
    M = y.shape[0]
    act = _act_dtype(y)
    st = lib().gdn_gated_out_proj(_ptr(norm_w, "norm_w", (DV,), torch.float32), float(norm_eps),
                                  _ptr(y, "y", (M, DI)), _ptr(z, "z", (M, DI), y.dtype),
                                  _ptr(w, "w", (N_EMBD, DI), torch.bfloat16), _ptr(out, "out", (M, N_EMBD)),
                                  M, act, _act_dtype(out), _stream(stream))
    _check(st, "gdn_gated_out_proj")


ATTN_HQ, ATTN_HKV, ATTN_D = 16, 2, 256   # GDN_ATTN_Q_HEADS, GDN_ATTN_KV_HEADS, GDN_ATTN_HEAD_DIM


def attn_decode_workspace_size(B: int, Lmax: int) -> int:
    return int(lib().gdn_attn_decode_workspace_size(int(B), int(Lmax)))


def attn_decode(q, k_cache, v_cache, ctx_len, z, out, workspace=None, stream=None):
    """gdn_attn_decode: one decode step of GQA attention (16 query / 2 KV heads,
    head_dim 256) with the sigmoid output gate. q, z [B][16][256] bf16; caches
    [B][2][Lmax][256] bf16; ctx_len [B] int32; out [B][16][256] fp32 or bf16.
    Allocates the workspace through torch when none is given."""
    B = q.shape[0]
    Lmax = k_cache.shape[2] if k_cache.dim() == 4 else 0
    od = _act_dtype(out)
    need = attn_decode_workspace_size(B, Lmax) if B > 0 else 0
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    st = lib().gdn_attn_decode(_ptr(q, "q", (B, ATTN_HQ, ATTN_D), torch.bfloat16),
                               _ptr(k_cache, "k_cache", (B, ATTN_HKV, Lmax, ATTN_D), torch.bfloat16),
                               _ptr(v_cache, "v_cache", (B, ATTN_HKV, Lmax, ATTN_D), torch.bfloat16),
                               _ptr(ctx_len, "ctx_len", (B,), torch.int32),
                               _ptr(z, "z", (B, ATTN_HQ, ATTN_D), torch.bfloat16),
                               _ptr(out, "out", (B, ATTN_HQ, ATTN_D)), B, Lmax, _ptr(workspace, "workspace"),
                               workspace.numel() * workspace.element_size(), od, _stream(stream))
    _check(st, "gdn_attn_decode")
    return workspace


# ---- the full-attention layers' input side and paged cache

GDN_KV_BF16, GDN_KV_Q4 = 0, 1
ATTN_ROT = 64                    # GDN_ATTN_ROT_DIM
KV_RECORD_ROWS, KV_RECORD_BYTES = 16, 4608


def make_attn_params(q_norm_w=None, k_norm_w=None, rope=None, norm_eps: float = 1e-6) -> gdn_attn_params:
    """gdn_attn_params from fp32 CUDA tensors: the RMSNorm weights [256] of
    queries and keys (None: no norm) and the rotation table [n_pos][64], 32
    cosines then 32 sines per position (None: no rotation). The struct keeps the
    tensors alive."""
    n_pos = rope.shape[0] if rope is not None else 0
    p = gdn_attn_params(_ptr(q_norm_w, "q_norm_w", (ATTN_D,), torch.float32),
                        _ptr(k_norm_w, "k_norm_w", (ATTN_D,), torch.float32),
                        _ptr(rope, "rope", (n_pos, ATTN_ROT), torch.float32), n_pos, float(norm_eps))
    p._keep_alive = (q_norm_w, k_norm_w, rope)
    p._device = _one_device(q_norm_w, k_norm_w, rope)
    p._ref = ctypes.addressof(p)
    return p


def make_kv_cache(k, v=None) -> gdn_kv_cache:
    """gdn_kv_cache over caller-owned tensors: bf16 k and v
    [num_pages][2][page_size][256], or for the 4-bit format one uint8 tensor
    [num_pages][2][page_size / 16][4608] (zeroed: rows of zeros). The struct
    keeps the tensors alive."""
    if v is None:
        pages, recs = k.shape[0], k.shape[2] if k.dim() == 4 else 0
        c = gdn_kv_cache(_ptr(k, "k", (pages, ATTN_HKV, recs, KV_RECORD_BYTES), torch.uint8), None, pages,
                         recs * KV_RECORD_ROWS, GDN_KV_Q4)
    else:
        pages, page = k.shape[0], k.shape[2] if k.dim() == 4 else 0
        shape = (pages, ATTN_HKV, page, ATTN_D)
        c = gdn_kv_cache(_ptr(k, "k", shape, torch.bfloat16), _ptr(v, "v", shape, torch.bfloat16, k.device), pages,
                         page, GDN_KV_BF16)
    c._keep_alive = (k, v)
    c._device = k.device
    c._ref = ctypes.addressof(c)
    return c


def make_paged_batch(page_table, ctx_len, M: int, cu_q=None, max_q: int = 1) -> gdn_paged_batch:
    """gdn_paged_batch from int32 CUDA tensors: page_table [B][max_pages],
    ctx_len [B] (the new tokens included), cu_q [B+1] packed row offsets (None:
    one token per sequence). M packed rows, at most max_q of one sequence. The
    struct reads the tensors at every call (update them in place from step to
    step) and keeps them alive."""
    B, mp = page_table.shape
    b = gdn_paged_batch(_ptr(page_table, "page_table", (B, mp), torch.int32),
                        _ptr(ctx_len, "ctx_len", (B,), torch.int32, page_table.device),
                        _ptr(cu_q, "cu_q", (B + 1,), torch.int32, page_table.device), B, int(M), int(max_q), mp)
    b._keep_alive = (page_table, ctx_len, cu_q)
    b._device = page_table.device
    b._ref = ctypes.addressof(b)
    return b


def _one_device(*tensors):
    devs = {t.device for t in tensors if t is not None}
    if len(devs) > 1:
        raise ValueError(f"tensors on different devices: {sorted(map(str, devs))}")
    return devs.pop() if devs else None


_one_gpu = None          # cuda:0 where it is the only device, so that it is the current one


def _on_current(device, where: str) -> torch.device:
    """The library launches on the current device: tensors of another one are refused."""
    global _one_gpu
    if device == _one_gpu:
        return device
    if device.type != "cuda":
        raise ValueError(f"{where}: tensors must be on a CUDA device, not {device}")
    if device.index != torch.cuda.current_device():
        raise ValueError(f"{where}: tensors are on {device}, the current device is cuda:{torch.cuda.current_device()}")
    if torch.cuda.device_count() == 1:
        _one_gpu = device
    return device


def _heads(t, name: str, M: int, heads: int, device, dtype=None):
    """(pointer, row stride, head stride) of a [M][heads][256] tensor whose last
    dim is dense; other strides are free (multiples of 16 bytes, checked by the
    library)."""
    if t is None:
        return None, 0, 0
    if t.shape == (M, heads, ATTN_D) and t.device == device and (dtype is None or t.dtype is dtype):
        row, head, last = t.stride()
        if last == 1:
            return t.data_ptr(), row, head
    _refuse(t, name, (M, heads, ATTN_D), device, dtype)
    raise ValueError(f"{name} must be dense in its last dimension")


def _dense(t, name: str, shape, device, dtype=None):
    """The pointer of a contiguous tensor of this shape (None for None)."""
    if t is None:
        return None
    if t.shape == shape and t.device == device and (dtype is None or t.dtype is dtype) and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, name, shape, device, dtype)
    raise ValueError(f"{name} must be contiguous")


def _refuse(t, name: str, shape, device, dtype):
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")


# The current stream's handle without a Stream object around it: 0.1 instead of 2 us a call.
_raw_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(stream, device) -> int:
    if stream is not None:
        return _stream(stream)
    if _raw_current_stream is not None:
        return _raw_current_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def attn_qk_norm_rope(params: gdn_attn_params, q, positions, q_out, k=None, k_out=None, stream=None):
    """gdn_attn_qk_norm_rope: per-head RMSNorm and rotation of q [M][16][256] and
    optionally k [M][2][256] (fp32 or bf16, strided views allowed, e.g. the query
    half of a joint query+gate projection) into dense q_out and k_out (fp32 or
    bf16). positions [M] int32: rows of the rotation table (None without one)."""
    M, dev = q.shape[0], _on_current(q.device, "attn_qk_norm_rope")
    if params._device is not None and params._device != dev:
        raise ValueError(f"the parameters are on {params._device}, expected {dev}")
    qp, qr, qh = _heads(q, "q", M, ATTN_HQ, dev)
    kp, kr, kh = _heads(k, "k", M, ATTN_HKV, dev, q.dtype)
    st = (_lib or lib()).gdn_attn_qk_norm_rope(params._ref, qp, qr, qh, kp, kr, kh,
                                     _dense(positions, "positions", (M,), dev, torch.int32), M,
                                     _dense(q_out, "q_out", (M, ATTN_HQ, ATTN_D), dev),
                                     _dense(k_out, "k_out", (M, ATTN_HKV, ATTN_D), dev, q_out.dtype), _act_dtype(q),
                                     _act_dtype(q_out), _raw_stream(stream, dev))
    if st:
        _check(st, "gdn_attn_qk_norm_rope")


def _on_batch(batch, cache, where: str, params=None):
    dev = _on_current(batch._device, where)
    if cache._device != dev or (params is not None and params._device is not None and params._device != dev):
        raise ValueError(f"{where}: batch, cache and parameters are on different devices")
    return dev


def kv_append(params: gdn_attn_params, batch: gdn_paged_batch, cache: gdn_kv_cache, k, v, q=None, q_out=None,
              positions=None, stream=None):
    """gdn_kv_append: the batch's new keys (normed and rotated on the way) and
    values [M][2][256] (fp32 or bf16, strided views allowed) into the paged
    cache. With q [M][16][256] and q_out (dense bf16) the queries are normed and
    rotated in the same launch. positions [M] int32 overrides the rows of the
    rotation table (default: the token's position in its context)."""
    M, dev = batch.M, _on_batch(batch, cache, "kv_append", params)
    kp, kr, kh = _heads(k, "k", M, ATTN_HKV, dev)
    vp, vr, vh = _heads(v, "v", M, ATTN_HKV, dev, k.dtype)
    qp, qr, qh = _heads(q, "q", M, ATTN_HQ, dev, k.dtype)
    st = (_lib or lib()).gdn_kv_append(params._ref, batch._ref, cache._ref, kp, kr, kh, vp, vr, vh, qp, qr, qh,
                             _dense(q_out, "q_out", (M, ATTN_HQ, ATTN_D), dev, torch.bfloat16),
                             _dense(positions, "positions", (M,), dev, torch.int32), _act_dtype(k),
                             _raw_stream(stream, dev))
    if st:
        _check(st, "gdn_kv_append")


def kv_gather(batch: gdn_paged_batch, cache: gdn_kv_cache, k_out, v_out, stream=None):
    """gdn_kv_gather: the cached rows of the batch's new tokens as values, into
    dense k_out and v_out [M][2][256] (fp32 or bf16; either may be None)."""
    M, dev = batch.M, _on_batch(batch, cache, "kv_gather")
    some = k_out if k_out is not None else v_out
    if some is None:
        return
    st = (_lib or lib()).gdn_kv_gather(batch._ref, cache._ref, _dense(k_out, "k_out", (M, ATTN_HKV, ATTN_D), dev, some.dtype),
                             _dense(v_out, "v_out", (M, ATTN_HKV, ATTN_D), dev, some.dtype), _act_dtype(some),
                             _raw_stream(stream, dev))
    if st:
        _check(st, "gdn_kv_gather")


def attn_paged_workspace_size(batch: gdn_paged_batch, cache: gdn_kv_cache) -> int:
    return int(lib().gdn_attn_paged_workspace_size(batch._ref, cache._ref))


def attn_paged(batch: gdn_paged_batch, cache: gdn_kv_cache, q, out, gate=None, workspace=None, stream=None):
    """gdn_attn_paged: causal attention of the batch's new tokens over the paged
    cache. q [M][16][256] dense bf16 (normed and rotated), out dense fp32 or
    bf16, gate [M][16][256] bf16 (strided views allowed; None: no output gate).
    Allocates the workspace through torch, for the stream the call runs on, when
    none is given, and returns it."""
    M, dev = batch.M, _on_batch(batch, cache, "attn_paged")
    gp, gr, gh = _heads(gate, "gate", M, ATTN_HQ, dev, torch.bfloat16)
    if workspace is None:
        need = max(attn_paged_workspace_size(batch, cache), 256)
        if stream is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        else:                                      # from that stream's memory: the current one may still use its own
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream), device=dev)
            with torch.cuda.stream(stream):
                workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    st = (_lib or lib()).gdn_attn_paged(batch._ref, cache._ref, _dense(q, "q", (M, ATTN_HQ, ATTN_D), dev, torch.bfloat16), gp, gr, gh,
                              _dense(out, "out", (M, ATTN_HQ, ATTN_D), dev), _dense(workspace, "workspace", workspace.shape, dev),
                              workspace.nbytes, _act_dtype(out), _raw_stream(stream, dev))
    if st:
        _check(st, "gdn_attn_paged")
    return workspace


# ---- around the mixers: residual and norms, dense products, mixture of experts

ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2, "sigmoid": 3}      # gdn_activation
MOE_MAX_EXPERTS, MOE_MAX_TOPK = 256, 16


def _rows(t, name: str, M: int, width: int, device, dtype=None):
    """(pointer, row stride) of a [M][width] tensor whose rows are dense."""
    if t is None:
        return None, 0
    if t.shape == (M, width) and t.device == device and (dtype is None or t.dtype is dtype):
        row, last = t.stride()
        if last == 1:
            return t.data_ptr(), row if M > 1 else width   # a single row has no next one
    _refuse(t, name, (M, width), device, dtype)
    raise ValueError(f"{name} must be dense in its last dimension")


def make_norm_params(norm_w=None, post_w=None, res_scale: float = 1.0, norm_eps: float = 1e-6) -> gdn_norm_params:
    """gdn_norm_params from fp32 CUDA tensors [2048]: the weight of the sum's norm
    (None: no normed output) and of the norm of the block's output (None: none).
    The struct keeps the tensors alive."""
    p = gdn_norm_params(_ptr(norm_w, "norm_w", (N_EMBD,), torch.float32), _ptr(post_w, "post_w", (N_EMBD,), torch.float32),
                        float(res_scale), float(norm_eps))
    p._keep_alive = (norm_w, post_w)
    p._device = _one_device(norm_w, post_w)
    p._ref = ctypes.addressof(p)
    return p


def add_norm(params: gdn_norm_params, x, delta, x_out, h, gate=None, stream=None):
    """gdn_add_norm: x_out = x + res_scale * gate * norm(delta) and its norm h, rows
    of 2048. x and x_out share one dtype (fp32 or bf16), delta, gate and h another;
    rows may be strided. delta, gate, x_out and h may be None; x_out may be x, and
    h may be delta. A gate of one row for all tokens: gate.expand(M, 2048)."""
    M, dev = x.shape[0], _on_current(x.device, "add_norm")
    if params._device is not None and params._device != dev:
        raise ValueError(f"the parameters are on {params._device}, expected {dev}")
    act = h if h is not None else delta if delta is not None else x
    xp, xr = _rows(x, "x", M, N_EMBD, dev)
    dp, dr = _rows(delta, "delta", M, N_EMBD, dev, act.dtype)
    gp, gr = _rows(gate, "gate", M, N_EMBD, dev, act.dtype)
    op, orow = _rows(x_out, "x_out", M, N_EMBD, dev, x.dtype)
    hp, hr = _rows(h, "h", M, N_EMBD, dev)
    st = (_lib or lib()).gdn_add_norm(params._ref, xp, xr, dp, dr, gp, gr, op, orow, hp, hr, M, _act_dtype(x),
                                      _act_dtype(act), _raw_stream(stream, dev))
    if st:
        _check(st, "gdn_add_norm")


def linear(x, w, y, bias=None, residual=None, activation: str = "none", stream=None):
    """gdn_linear: y = residual + activation(x w^T + bias). x [M][K] and w [N][K]
    bf16, y [M][N] and residual fp32 or bf16, bias [N] fp32; rows of x, residual
    and y may be strided, residual may be y. activation: one of ACTIVATIONS."""
    (M, K), N, dev = x.shape, w.shape[0], _on_current(x.device, "linear")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation {activation!r}: expected one of {sorted(ACTIVATIONS)}")
    xp, xr = _rows(x, "x", M, K, dev, torch.bfloat16)
    yp, yr = _rows(y, "y", M, N, dev)
    rp, rr = _rows(residual, "residual", M, N, dev, y.dtype)
    st = (_lib or lib()).gdn_linear(xp, xr, _dense(w, "w", (N, K), dev, torch.bfloat16),
                                    _dense(bias, "bias", (N,), dev, torch.float32), rp, rr, yp, yr, M, N, K,
                                    ACTIVATIONS[activation], _act_dtype(y), _raw_stream(stream, dev))
    if st:
        _check(st, "gdn_linear")


def make_moe_params(router, gate=None, up=None, down=None, sh_gate=None, sh_up=None, sh_down=None, sh_router=None,
                    top_k: int = 8, norm_topk: bool = True) -> gdn_moe_params:
    """gdn_moe_params from bf16 CUDA tensors: router [E][2048] (None: the routing is
    always given), gate and up [E][F][2048], down [E][2048][F] (None: for
    moe_route alone), the shared expert's gate and up [F][2048], down [2048][F]
    and sigmoid gate [2048] (None: none). The struct keeps the tensors alive."""
    bf = torch.bfloat16
    E = router.shape[0] if router is not None else gate.shape[0]
    F = gate.shape[1] if gate is not None and gate.dim() == 3 else 0
    ts = (router, gate, up, down, sh_gate, sh_up, sh_down, sh_router)
    shapes = ((E, N_EMBD), (E, F, N_EMBD), (E, F, N_EMBD), (E, N_EMBD, F), (F, N_EMBD), (F, N_EMBD), (N_EMBD, F), (N_EMBD,))
    names = [n for n, _ in gdn_moe_params._fields_]
    p = gdn_moe_params(*(_ptr(t, n, s, bf) for t, n, s in zip(ts, names, shapes)), E, int(top_k), F, int(bool(norm_topk)))
    p._keep_alive = ts
    p._device = _one_device(*ts)
    p._ref = ctypes.addressof(p)
    return p


def moe_route(params: gdn_moe_params, x, ids, weights, stream=None):
    """gdn_moe_route: the top_k experts of each row of x [M][2048] bf16 (rows may be
    strided), best first, into ids [M][top_k] int32 and weights [M][top_k] fp32."""
    M, dev = x.shape[0], _on_current(x.device, "moe_route")
    if params._device != dev:
        raise ValueError(f"the parameters are on {params._device}, expected {dev}")
    xp, xr = _rows(x, "x", M, N_EMBD, dev, torch.bfloat16)
    st = (_lib or lib()).gdn_moe_route(params._ref, xp, xr, M, _dense(ids, "ids", (M, params.top_k), dev, torch.int32),
                                       _dense(weights, "weights", (M, params.top_k), dev, torch.float32),
                                       _raw_stream(stream, dev))
    if st:
        _check(st, "gdn_moe_route")


def moe_workspace_size(params: gdn_moe_params, M: int) -> int:
    return int(lib().gdn_moe_workspace_size(params._ref, int(M)))


def _workspace(need: int, device, stream):
    """Scratch through torch, from the memory of the stream that the call runs on."""
    if stream is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(need, dtype=torch.uint8, device=device)


def moe(params: gdn_moe_params, x, out, residual=None, ids=None, weights=None, workspace=None, stream=None):
    """gdn_moe: the whole mixture-of-experts feed-forward of x [M][2048] bf16 (rows
    may be strided) into out [M][2048] (fp32 or bf16), plus residual (same dtype;
    may be out). ids and weights [M][top_k]: the routing, if it is given.
    Allocates the workspace through torch, for the stream the call runs on, when
    none is given, and returns it."""
    M, dev = x.shape[0], _on_current(x.device, "moe")
    if params._device != dev:
        raise ValueError(f"the parameters are on {params._device}, expected {dev}")
    if workspace is None:
        workspace = _workspace(max(moe_workspace_size(params, M), 256), dev, stream)
    xp, xr = _rows(x, "x", M, N_EMBD, dev, torch.bfloat16)
    st = (_lib or lib()).gdn_moe(params._ref, xp, xr, _dense(residual, "residual", (M, N_EMBD), dev, out.dtype),
                                 _dense(out, "out", (M, N_EMBD), dev), M,
                                 _dense(ids, "ids", (M, params.top_k), dev, torch.int32),
                                 _dense(weights, "weights", (M, params.top_k), dev, torch.float32),
                                 _dense(workspace, "workspace", workspace.shape, dev), workspace.nbytes, _act_dtype(out),
                                 _raw_stream(stream, dev))
    if st:
        _check(st, "gdn_moe")
    return workspace


def prefill_workspace_size(N: int, T_total: int, act=torch.bfloat16, chunk_size: int = 0) -> int:
    return int(lib().gdn_prefill_workspace_size(int(N), int(T_total), _DT[act], int(chunk_size)))


def prefill(params, qkv, z, alpha, beta, cu_seqlens, out, conv_state_in=None, conv_state_out=None,
            ssm_state_in=None, ssm_state_out=None, chunk_size: int = 0, workspace=None, stream=None,
            cparams: gdn_params | None = None):
    """gdn_prefill over N packed sequences (cu_seqlens: int32 CUDA [N+1]).
    Allocates the workspace through torch when none is given."""
    T = qkv.shape[0]
    N = cu_seqlens.shape[0] - 1
    dt = qkv.dtype
    act = _act_dtype(qkv)
    od = _act_dtype(out)
    need = prefill_workspace_size(N, T, dt, chunk_size)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=qkv.device)
    cp = cparams if cparams is not None else make_params(params)
    st = lib().gdn_prefill(ctypes.byref(cp), _ptr(qkv, "qkv", (T, CC)), _ptr(z, "z", (T, DI), dt),
                           _ptr(alpha, "alpha", (T, HV), dt), _ptr(beta, "beta", (T, HV), dt),
                           _ptr(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32), N, T,
                           _ptr(conv_state_in, "conv_state_in", (N, KC - 1, CC), dt),
                           _ptr(conv_state_out, "conv_state_out", (N, KC - 1, CC), dt),
                           _ptr(ssm_state_in, "ssm_state_in", (N, HV, DV, DK), torch.float32),
                           _ptr(ssm_state_out, "ssm_state_out", (N, HV, DV, DK), torch.float32),
                           _ptr(out, "out", (T, DI)), act, od, int(chunk_size),
                           _ptr(workspace, "workspace"), workspace.numel() * workspace.element_size(),
                           _stream(stream))
    _check(st, "gdn_prefill")
    return workspace


def device_error(stream=None) -> int:
    """Synchronises the stream, then reads and clears the library's device error
    word: GDN_OK, or GDN_ERR_TIMEOUT if a bounded device-side wait gave up."""
    return lib().gdn_device_error(_stream(stream))


def selftest_wait_timeout(stream=None) -> None:
    """gdn_selftest_wait_timeout: enqueue the kernel whose bounded wait runs
    out (about 2 s); the next device_error() then reports GDN_ERR_TIMEOUT."""
    _check(lib().gdn_selftest_wait_timeout(_stream(stream)), "gdn_selftest_wait_timeout")


def selftest_moe_lost_route(params: gdn_moe_params, x, out, residual=None, stream=None) -> None:
    """gdn_selftest_moe_lost_route: moe() of more than 4 tokens whose router's wait runs out (about
    2 s): out = residual + the shared expert, and the next device_error() reports GDN_ERR_TIMEOUT."""
    M, dev = x.shape[0], _on_current(x.device, "selftest_moe_lost_route")
    ws = _workspace(max(moe_workspace_size(params, M), 256), dev, stream)
    xp, xr = _rows(x, "x", M, N_EMBD, dev, torch.bfloat16)
    _check(lib().gdn_selftest_moe_lost_route(params._ref, xp, xr, _dense(residual, "residual", (M, N_EMBD), dev, out.dtype),
                                             _dense(out, "out", (M, N_EMBD), dev), M, ws.data_ptr(), ws.nbytes, _act_dtype(out),
                                             _raw_stream(stream, dev)), "gdn_selftest_moe_lost_route")


def static_scratch_bytes() -> int:
    """Bytes of the fixed scratch gdn_prefill_static uses, from the library."""
    L = lib()
    L.gdn_static_scratch_bytes.restype = _sz
    L.gdn_static_scratch_bytes.argtypes = []
    return int(L.gdn_static_scratch_bytes())


DECODE_MAX_T = 8   # GDN_DECODE_MAX_T: tokens per sequence of gdn_decode_multi, at most


def prefill_static(params, qkv, z, alpha, beta, cu_seqlens, out, conv_state_in=None, conv_state_out=None,
                   ssm_state_in=None, ssm_state_out=None, chunk_size: int = 0, stream=None,
                   cparams: gdn_params | None = None):
    """gdn_prefill_static: gdn_prefill without a workspace argument, for callers
    that cannot allocate device memory. The library's fixed 64 MiB device
    scratch is used instead, shared by every call on the device."""
    T = qkv.shape[0]
    N = cu_seqlens.shape[0] - 1
    dt = qkv.dtype
    cp = cparams if cparams is not None else make_params(params)
    st = lib().gdn_prefill_static(ctypes.byref(cp), _ptr(qkv, "qkv", (T, CC)), _ptr(z, "z", (T, DI), dt),
                                  _ptr(alpha, "alpha", (T, HV), dt), _ptr(beta, "beta", (T, HV), dt),
                                  _ptr(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32), N, T,
                                  _ptr(conv_state_in, "conv_state_in", (N, KC - 1, CC), dt),
                                  _ptr(conv_state_out, "conv_state_out", (N, KC - 1, CC), dt),
                                  _ptr(ssm_state_in, "ssm_state_in", (N, HV, DV, DK), torch.float32),
                                  _ptr(ssm_state_out, "ssm_state_out", (N, HV, DV, DK), torch.float32),
                                  _ptr(out, "out", (T, DI)), _act_dtype(qkv), _act_dtype(out), int(chunk_size),
                                  _stream(stream))
    _check(st, "gdn_prefill_static")
