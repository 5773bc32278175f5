"""Gated DeltaNet (GDN) decode / MTP-verify / commit on one GB300 -- Python binding of ``libgdn.so``.

Argument marshalling only: every step of the computation runs in the library's CUDA kernels
(``csrc/``); PyTorch supplies device memory and the current stream.  There is no CPU fallback: if the
library has not been built, every call raises.

    gdn_decode(q, k, v, a, b, A_log, dt_bias, state_pool, state_indices, o, err_word=None, scale=1.0, l2_eps=1e-6)
    gdn_decode_gated(q, k, v, a, b, A_log, dt_bias, state_pool, state_indices, o, norm, err_word=None, ...)
    gdn_mtp_verify(q, k, v, a, b, A_log, dt_bias, state_pool, state_indices, o, intermediate_states=None, ...)
    gdn_commit(state_pool, state_indices, intermediate_states, accept_len, err_word=None)
    gdn_commit_replay(q, k, v, a, b, A_log, dt_bias, state_pool, state_indices, accept_len, err_word=None, ...)
    gdn_mtp_verify_commit(prev, q, k, v, a, b, A_log, dt_bias, state_pool, state_indices, o, err_word=None,
                          norm=None, ...)
    gdn_mtp_verify_gated(q, k, v, a, b, A_log, dt_bias, state_pool, state_indices, o, norm,
                         intermediate_states=None, err_word=None, ...)
    gdn_prefill(q, k, v, a, b, A_log, dt_bias, state_pool, state_indices, cu_seqlens, o,
                has_initial_state=None, err_word=None, ...)
    gdn_gated_rmsnorm(o, z, norm_weight, y=None, eps=1e-6)
    gdn_in_proj_conv(x, W, conv_w, conv_b, conv_state, state_indices, out, write_state, records=None,
                     err_word=None, silu=True)
    gdn_conv_commit(conv_state, state_indices, records, accept_len, err_word=None)

and, for the softmax-attention layers between the recurrent ones, over a paged 4-bit K/V cache (``Kv4Cache``):

    gdn_page_plan(kv_lens, new_lens, page_size, block_tables, held, free_pages, taken, plan, ticket, err_word=None)
    gdn_qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, q_out, k_out=None, *, v=None, cache=None,
                     slot_map=None, err_word=None, eps=1e-6, interleaved=False)
    gdn_kv4_read(cache, slot_map, k_out, v_out, err_word=None)
    gdn_kv4_attention(q, cache, block_tables, kv_lens, o, workspace, *, cu_seqlens=None, max_q=None, lse=None,
                      scale=None, err_word=None)
    kv4_attention_workspace(B, max_q, HQ, HK, D, device=None)

Shapes and semantics are those of ``include/gdn.h``: q, k ``[B,T,HK,DK]``; v, o ``[B,T,HV,DV]``; a, b
``[B,T,HV]``; A_log, dt_bias ``[HV]`` fp32; state_pool ``[num_slots,HV,DV,DK]``; state_indices, accept_len
``[B]`` int32; intermediate_states ``[B,T,HV,DV,DK]``; err_word a 1-element int32 device tensor.  Prefill takes
packed tokens: q, k ``[N,HK,DK]``; v, o ``[N,HV,DV]``; a, b ``[N,HV]``; cu_seqlens ``[B+1]`` and
has_initial_state ``[B]`` int32.  The in_proj projection takes x ``[B,T,H]`` bf16, W ``[C,H]`` bf16, conv_w
``[Cc,K]`` / conv_b ``[Cc]`` fp32, conv_state ``[num_slots,K-1,Cc]`` and records ``[B,T,Cc]``, and writes the q, k,
v, z, b, a of an ``InProjOut`` (their shapes give HK, DK, HV, DV).
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

from .build import LIB_PATH

__all__ = ["gdn_decode", "gdn_decode_gated", "gdn_mtp_verify", "gdn_commit", "gdn_commit_replay", "gdn_mtp_verify_commit", "ReplayTokens",
           "gdn_mtp_verify_gated", "GatedNorm",
           "gdn_prefill", "gdn_gated_rmsnorm", "gdn_in_proj_conv", "gdn_conv_commit", "InProjOut", "GdnError", "GdnDims", "lib", "STATUS", "ERRBIT_INDEX", "ERRBIT_ACCEPT_LEN", "ERRBIT_TIMEOUT",
           "ERRBIT_SEQLEN", "ERRBIT_PAGES", "ERRBIT_NONFINITE", "MAX_T", "EXPORTS",
           "gdn_page_plan", "gdn_qk_norm_rope", "gdn_kv4_read", "gdn_kv4_attention", "kv4_attention_workspace", "Kv4Cache",
           "PagePlan"]

STATUS = {0: "GDN_OK", 1: "GDN_ERR_NULL", 2: "GDN_ERR_SHAPE", 3: "GDN_ERR_DTYPE", 4: "GDN_ERR_ALIGN",
          5: "GDN_ERR_UNSUPPORTED", 6: "GDN_ERR_CUDA", 7: "GDN_ERR_VALUE"}
ERRBIT_INDEX = 1
ERRBIT_ACCEPT_LEN = 2
ERRBIT_TIMEOUT = 4
ERRBIT_SEQLEN = 8
ERRBIT_PAGES = 16
ERRBIT_NONFINITE = 32
MAX_T = 16
F32, BF16 = 0, 1
EXPORTS = ("gdn_decode", "gdn_decode_gated", "gdn_mtp_verify", "gdn_commit", "gdn_commit_replay",
           "gdn_mtp_verify_commit", "gdn_mtp_verify_gated", "gdn_prefill",
           "gdn_gated_rmsnorm", "gdn_in_proj_conv", "gdn_conv_commit", "gdn_page_plan", "gdn_qk_norm_rope",
           "gdn_kv4_read", "gdn_kv4_attention", "gdn_kv4_attention_workspace", "gdn_status_string",
           "gdn_last_cuda_error", "gdn_abi_version")


class GdnDims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("HK", ctypes.c_int32), ("HV", ctypes.c_int32),
                ("DK", ctypes.c_int32), ("DV", ctypes.c_int32), ("num_slots", ctypes.c_int32),
                ("qkv_dtype", ctypes.c_int32), ("state_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("scale", ctypes.c_float), ("l2_eps", ctypes.c_float)]


class _ReplayTokensC(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("a", ctypes.c_void_p),
                ("b", ctypes.c_void_p), ("accept_len", ctypes.c_void_p)]


class ReplayTokens:
    """The k, v, a, b of an earlier ``gdn_mtp_verify`` on the same lanes (``[B, T', ...]``, T' its token count)
    and ``accept_len`` ``[B]`` int32: the tokens ``gdn_mtp_verify_commit`` commits before it verifies."""

    def __init__(self, k, v, a, b, accept_len):
        self.k, self.v, self.a, self.b, self.accept_len = k, v, a, b, accept_len


class _GatedNormC(ctypes.Structure):
    _fields_ = [("z", ctypes.c_void_p), ("z_dtype", ctypes.c_int32), ("norm_weight", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("y", ctypes.c_void_p)]


class GatedNorm:
    """The gated RMSNorm of a verify's outputs into ``y``: ``z`` (the gate, o's shape, fp32 or bf16),
    ``norm_weight`` ``[DV]`` fp32, ``y`` (o's shape and dtype; may be o itself)."""

    def __init__(self, z, norm_weight, y, eps=1e-6):
        self.z, self.norm_weight, self.y, self.eps = z, norm_weight, y, eps


class _ConvDimsC(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32), ("HK", ctypes.c_int32),
                ("HV", ctypes.c_int32), ("DK", ctypes.c_int32), ("DV", ctypes.c_int32), ("K", ctypes.c_int32),
                ("num_slots", ctypes.c_int32), ("conv_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("silu", ctypes.c_int32)]


class _InProjOutC(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("z", ctypes.c_void_p),
                ("b", ctypes.c_void_p), ("a", ctypes.c_void_p)]


class InProjOut:
    """The outputs of ``gdn_in_proj_conv``: q, k ``[B,T,HK,DK]``, v, z ``[B,T,HV,DV]``, b, a ``[B,T,HV]``, one dtype."""

    def __init__(self, q, k, v, z, b, a):
        self.q, self.k, self.v, self.z, self.b, self.a = q, k, v, z, b, a


class _Kv4CacheC(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("HK", ctypes.c_int32), ("D", ctypes.c_int32),
                ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


class Kv4Cache:
    """The paged 4-bit K/V cache of one attention layer: ``codes`` ``[num_pages, 2, HK, page_size, D / 2]`` and ``scales``
    ``[num_pages, 2, HK, page_size, D / 16]``, uint8 on one GPU (keys 0, values 1; two e2m1 codes a byte, an e4m3 scale for
    each 16 dimensions); ``k_scale`` and ``v_scale`` (powers of two) multiply every number."""

    def __init__(self, codes, scales, k_scale=1.0, v_scale=1.0):
        import torch

        if codes.dim() != 5 or scales.dim() != 5:
            raise ValueError("codes is [num_pages,2,HK,page_size,D/2], scales [num_pages,2,HK,page_size,D/16]")
        num_pages, two, HK, page_size, half = codes.shape
        _shape(codes, (num_pages, 2, HK, page_size, half), "codes")
        _shape(scales, (num_pages, 2, HK, page_size, half // 8), "scales")
        self.device = _common_device([("codes", codes), ("scales", scales)])
        self.codes, self.scales = codes, scales
        self.num_pages, self.page_size, self.HK, self.D = num_pages, page_size, HK, 2 * half
        self.c = _Kv4CacheC(_dev(codes, "codes", torch.uint8), _dev(scales, "scales", torch.uint8), num_pages, page_size,
                            HK, 2 * half, float(k_scale), float(v_scale))
        self.ref = ctypes.byref(self.c)


class _PagePlanC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("cu_seqlens", "positions", "slot_map", "total_lens", "held", "taken")]


class PagePlan:
    """What ``gdn_page_plan`` writes, int32 on one GPU: ``cu_seqlens`` ``[B+1]``, ``positions`` and ``slot_map`` ``[N]``,
    ``total_lens`` and ``held`` ``[B]``, ``taken`` ``[1]`` (``held`` and ``taken`` may be the call's inputs)."""

    def __init__(self, cu_seqlens, positions, slot_map, total_lens, held, taken):
        import torch

        B, N = cu_seqlens.numel() - 1, positions.numel()
        named = (("cu_seqlens", cu_seqlens, B + 1), ("positions", positions, N), ("slot_map", slot_map, N),
                 ("total_lens", total_lens, B), ("held", held, B), ("taken", taken, 1))
        for name, t, n in named:
            _shape(t, (n,), name)
        self.device = _common_device([(name, t) for name, t, _ in named])
        self.B, self.N = B, N
        self.cu_seqlens, self.positions, self.slot_map = cu_seqlens, positions, slot_map
        self.total_lens, self.held, self.taken = total_lens, held, taken
        self.c = _PagePlanC(*(_dev(t, name, torch.int32) for name, t, _ in named))
        self.ref = ctypes.byref(self.c)


class _QkDimsC(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("HQ", ctypes.c_int32), ("HK", ctypes.c_int32), ("D", ctypes.c_int32),
                ("R", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("eps", ctypes.c_float)]


class _Kv4AttentionDimsC(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("N", ctypes.c_int32), ("max_q", ctypes.c_int32), ("HQ", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("scale", ctypes.c_float)]


class GdnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = _lib_handle.gdn_status_string(status).decode() if _lib_handle is not None else STATUS.get(status)
        if status == 6 and _lib_handle is not None:
            msg += f" (cudaError {_lib_handle.gdn_last_cuda_error()})"
        super().__init__(f"{what}: {msg}")


_lib_handle: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """The loaded ``libgdn.so``; raises if it has not been built (no fallback exists)."""
    global _lib_handle
    if _lib_handle is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m gated_deltanet_linear_mtp_gb300.build` (there is no CPU fallback)")
        L = ctypes.CDLL(LIB_PATH)
        vp, dp, ip = ctypes.c_void_p, ctypes.POINTER(GdnDims), ctypes.c_void_p
        L.gdn_decode.argtypes = [dp] + [vp] * 5 + [vp, vp, vp, ip, vp, ip, vp]
        L.gdn_decode_gated.argtypes = [dp] + [vp] * 5 + [vp, vp, vp, ip, vp, ctypes.POINTER(_GatedNormC), ip, vp]
        L.gdn_mtp_verify.argtypes = [dp] + [vp] * 5 + [vp, vp, vp, ip, vp, vp, ip, vp]
        L.gdn_commit.argtypes = [dp, vp, ip, vp, ip, ip, vp]
        L.gdn_commit_replay.argtypes = [dp] + [vp] * 5 + [vp, vp, vp, ip, ip, ip, vp]
        L.gdn_mtp_verify_commit.argtypes = ([dp, ctypes.POINTER(_ReplayTokensC)] + [vp] * 5 +
                                            [vp, vp, vp, ip, vp, ctypes.POINTER(_GatedNormC), ip, vp])
        L.gdn_mtp_verify_gated.argtypes = [dp] + [vp] * 5 + [vp, vp, vp, ip, vp, vp, ctypes.POINTER(_GatedNormC), ip, vp]
        L.gdn_prefill.argtypes = [dp, ip] + [vp] * 5 + [vp, vp, vp, ip, ip, vp, ip, vp]
        L.gdn_gated_rmsnorm.argtypes = [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, vp, vp, vp,
                                        ctypes.c_float, vp, vp]
        cdp = ctypes.POINTER(_ConvDimsC)
        L.gdn_in_proj_conv.argtypes = [cdp, vp, vp, vp, vp, vp, ip, ctypes.c_int32, ctypes.POINTER(_InProjOutC), vp,
                                       ip, vp]
        L.gdn_conv_commit.argtypes = [cdp, vp, ip, vp, ip, ip, vp]
        i32 = ctypes.c_int32
        L.gdn_page_plan.argtypes = [i32] * 5 + [vp] * 10
        L.gdn_qk_norm_rope.argtypes = [vp] * 14
        L.gdn_kv4_read.argtypes = [vp, i32] + [vp] * 5
        L.gdn_kv4_attention.argtypes = [vp] * 9 + [ctypes.c_int64, vp, vp]
        L.gdn_kv4_attention_workspace.argtypes = [i32] * 5
        L.gdn_kv4_attention_workspace.restype = ctypes.c_int64
        for f in (L.gdn_in_proj_conv, L.gdn_conv_commit, L.gdn_page_plan, L.gdn_qk_norm_rope, L.gdn_kv4_read,
                  L.gdn_kv4_attention):
            f.restype = ctypes.c_int
        for f in (L.gdn_decode, L.gdn_decode_gated, L.gdn_mtp_verify, L.gdn_commit, L.gdn_commit_replay, L.gdn_mtp_verify_commit,
                  L.gdn_mtp_verify_gated, L.gdn_prefill, L.gdn_gated_rmsnorm):
            f.restype = ctypes.c_int
        L.gdn_status_string.argtypes = [ctypes.c_int]
        L.gdn_status_string.restype = ctypes.c_char_p
        L.gdn_last_cuda_error.restype = ctypes.c_int32
        L.gdn_abi_version.restype = ctypes.c_int32
        _lib_handle = L
    return _lib_handle


# ---- marshalling -------------------------------------------------------------------------------------
def _code(t, name: str) -> int:
    import torch

    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"{name}: dtype {t.dtype} (fp32 or bf16 expected)")


def _dev(t, name: str, dtype=None):
    """Pointer of a contiguous CUDA tensor (None -> NULL)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    return ctypes.c_void_p(t.data_ptr())


def _shape(t, want, name: str):
    if tuple(t.shape) != tuple(want):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(want)}")


def _common_device(named):
    """The one CUDA device that every given tensor (``(name, tensor)`` pairs, None skipped) lives on.

    A call launches its kernels on one GPU with raw pointers: a tensor on another GPU would be read through
    peer access or fault, so mixed devices are rejected before anything is launched."""
    dev, first = None, None
    for name, t in named:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if dev is None:
            dev, first = t.device, name
        elif t.device != dev:
            raise ValueError(f"{name} is on {t.device} but {first} is on {dev}: every tensor of one call must be "
                             "on the same GPU")
    if dev is None:
        raise ValueError("no CUDA tensor given")
    return dev


def _stream(stream, device):
    """The launch stream: the given one (which must belong to `device`) or `device`'s current stream."""
    import torch

    s = torch.cuda.current_stream(device) if stream is None else stream
    if s.device != device:
        raise ValueError(f"stream is on {s.device}, the tensors on {device}")
    return ctypes.c_void_p(s.cuda_stream)


def _io_dims(q, k, v, a, b, A_log, dt_bias, state_pool, state_indices, o, scale, l2_eps) -> GdnDims:
    import torch

    if q.dim() != 4 or v.dim() != 4 or state_pool.dim() != 4:
        raise ValueError("q/k and v/o are 4-D, state_pool is 4-D")
    B, T, HK, DK = q.shape
    HV, DV = v.shape[2], v.shape[3]
    _shape(k, q.shape, "k")
    _shape(v, (B, T, HV, DV), "v")
    if o is not None:
        _shape(o, (B, T, HV, DV), "o")
    _shape(a, (B, T, HV), "a")
    _shape(b, (B, T, HV), "b")
    _shape(A_log, (HV,), "A_log")
    _shape(dt_bias, (HV,), "dt_bias")
    if state_indices is not None:  # None: the caller checks the indices (prefill: one per prompt)
        _shape(state_indices, (B,), "state_indices")
    num_slots = state_pool.shape[0]
    _shape(state_pool, (num_slots, HV, DV, DK), "state_pool")
    qkv = _code(q, "q")
    for t, n in ((k, "k"), (v, "v"), (a, "a"), (b, "b")):
        if _code(t, n) != qkv:
            raise TypeError(f"{n} must have q's dtype")
    for t, n in ((A_log, "A_log"), (dt_bias, "dt_bias")):
        if t.dtype != torch.float32:
            raise TypeError(f"{n} must be fp32")
    if state_indices is not None and state_indices.dtype != torch.int32:
        raise TypeError("state_indices must be int32")
    out = _code(o, "o") if o is not None else _code(state_pool, "state_pool")
    return GdnDims(B, T, HK, HV, DK, DV, num_slots, qkv, _code(state_pool, "state_pool"), out, float(scale),
                   float(l2_eps))


def _call(status: int, what: str) -> None:
    if status != 0:
        raise GdnError(status, what)


def _launch(device, stream, fn, args, what: str) -> None:
    """One library call with `device` current, on `stream` (default: `device`'s current stream)."""
    import torch

    s = _stream(stream, device)
    with torch.cuda.device(device):
        _call(fn(*args, s), what)


def _io_named(q, k, v, a, b, A_log, dt_bias, state_pool, state_indices):
    return [("q", q), ("k", k), ("v", v), ("a", a), ("b", b), ("A_log", A_log), ("dt_bias", dt_bias),
            ("state_pool", state_pool), ("state_indices", state_indices)]


# ---- the calls -------------------------------------------------------------------------------------------
def gdn_decode(q, k, v, a, b, A_log, dt_bias, state_pool, state_indices, o, err_word=None, *, scale=1.0,
               l2_eps=1e-6, stream=None) -> None:
    """T tokens (normally 1) from ``state_pool[state_indices[b]]``; the final state is written back in place."""
    L = lib()
    d = _io_dims(q, k, v, a, b, A_log, dt_bias, state_pool, state_indices, o, scale, l2_eps)
    device = _common_device(_io_named(q, k, v, a, b, A_log, dt_bias, state_pool, state_indices)
                            + [("o", o), ("err_word", err_word)])
    _launch(device, stream, L.gdn_decode,
            (ctypes.byref(d), _dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(a, "a"), _dev(b, "b"),
             _dev(A_log, "A_log"), _dev(dt_bias, "dt_bias"), _dev(state_pool, "state_pool"),
             _dev(state_indices, "state_indices"), _dev(o, "o"), _dev(err_word, "err_word")), "gdn_decode")


def gdn_decode_gated(q, k, v, a, b, A_log, dt_bias, state_pool, state_indices, o, norm, err_word=None, *,
                     scale=1.0, l2_eps=1e-6, stream=None) -> None:
    """``gdn_decode`` (o and the write-back) and the gated RMSNorm of o into ``norm.y`` (``norm``: a GatedNorm), in
    the same launch where the CTAs of a head fit one thread-block cluster."""
    L = lib()
    d = _io_dims(q, k, v, a, b, A_log, dt_bias, state_pool, state_indices, o, scale, l2_eps)
    nc = _norm_c(norm, o)
    device = _common_device(_io_named(q, k, v, a, b, A_log, dt_bias, state_pool, state_indices)
                            + [("o", o), ("err_word", err_word)] + _norm_named(norm))
    _launch(device, stream, L.gdn_decode_gated,
            (ctypes.byref(d), _dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(a, "a"), _dev(b, "b"),
             _dev(A_log, "A_log"), _dev(dt_bias, "dt_bias"), _dev(state_pool, "state_pool"),
             _dev(state_indices, "state_indices"), _dev(o, "o"), ctypes.byref(nc), _dev(err_word, "err_word")),
            "gdn_decode_gated")


def gdn_mtp_verify(q, k, v, a, b, A_log, dt_bias, state_pool, state_indices, o, intermediate_states=None,
                   err_word=None, *, scale=1.0, l2_eps=1e-6, stream=None) -> None:
    """T draft tokens from ``state_pool[state_indices[b]]`` (read only); optional per-token state cache."""
    L = lib()
    d = _io_dims(q, k, v, a, b, A_log, dt_bias, state_pool, state_indices, o, scale, l2_eps)
    if intermediate_states is not None:
        _shape(intermediate_states, (d.B, d.T, d.HV, d.DV, d.DK), "intermediate_states")
        if intermediate_states.dtype != state_pool.dtype:
            raise TypeError("intermediate_states must have state_pool's dtype")
    device = _common_device(_io_named(q, k, v, a, b, A_log, dt_bias, state_pool, state_indices)
                            + [("o", o), ("intermediate_states", intermediate_states), ("err_word", err_word)])
    _launch(device, stream, L.gdn_mtp_verify,
            (ctypes.byref(d), _dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(a, "a"), _dev(b, "b"),
             _dev(A_log, "A_log"), _dev(dt_bias, "dt_bias"), _dev(state_pool, "state_pool"),
             _dev(state_indices, "state_indices"), _dev(o, "o"), _dev(intermediate_states, "intermediate_states"),
             _dev(err_word, "err_word")), "gdn_mtp_verify")


def gdn_commit(state_pool, state_indices, intermediate_states, accept_len, err_word=None, *, stream=None) -> None:
    """``state_pool[state_indices[b]] = intermediate_states[b, accept_len[b] - 1]`` for active lanes."""
    import torch

    L = lib()
    if intermediate_states.dim() != 5 or state_pool.dim() != 4:
        raise ValueError("intermediate_states is [B,T,HV,DV,DK], state_pool is [num_slots,HV,DV,DK]")
    B, T, HV, DV, DK = intermediate_states.shape
    num_slots = state_pool.shape[0]
    _shape(state_pool, (num_slots, HV, DV, DK), "state_pool")
    _shape(state_indices, (B,), "state_indices")
    _shape(accept_len, (B,), "accept_len")
    if state_indices.dtype != torch.int32 or accept_len.dtype != torch.int32:
        raise TypeError("state_indices and accept_len must be int32")
    if intermediate_states.dtype != state_pool.dtype:
        raise TypeError("intermediate_states must have state_pool's dtype")
    sd = _code(state_pool, "state_pool")
    d = GdnDims(B, T, 1, HV, DK, DV, num_slots, sd, sd, sd, 1.0, 0.0)
    device = _common_device([("state_pool", state_pool), ("state_indices", state_indices),
                             ("intermediate_states", intermediate_states), ("accept_len", accept_len),
                             ("err_word", err_word)])
    _launch(device, stream, L.gdn_commit,
            (ctypes.byref(d), _dev(state_pool, "state_pool"), _dev(state_indices, "state_indices"),
             _dev(intermediate_states, "intermediate_states"), _dev(accept_len, "accept_len"),
             _dev(err_word, "err_word")), "gdn_commit")


def gdn_commit_replay(q, k, v, a, b, A_log, dt_bias, state_pool, state_indices, accept_len, err_word=None, *,
                      scale=1.0, l2_eps=1e-6, stream=None) -> None:
    """The first ``accept_len[b]`` tokens again from ``state_pool[state_indices[b]]``, final state written back
    (the verify call's inputs; no outputs).  The pool state ``gdn_commit`` leaves after a caching verify: the
    same bits for an fp32 pool or T > 8, within one bf16 ulp (the chunked tensor-core form) for a bf16 pool
    with T <= 8."""
    import torch

    L = lib()
    d = _io_dims(q, k, v, a, b, A_log, dt_bias, state_pool, state_indices, None, scale, l2_eps)
    _shape(accept_len, (d.B,), "accept_len")
    if accept_len.dtype != torch.int32:
        raise TypeError("accept_len must be int32")
    device = _common_device(_io_named(q, k, v, a, b, A_log, dt_bias, state_pool, state_indices)
                            + [("accept_len", accept_len), ("err_word", err_word)])
    _launch(device, stream, L.gdn_commit_replay,
            (ctypes.byref(d), _dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(a, "a"), _dev(b, "b"),
             _dev(A_log, "A_log"), _dev(dt_bias, "dt_bias"), _dev(state_pool, "state_pool"),
             _dev(state_indices, "state_indices"), _dev(accept_len, "accept_len"), _dev(err_word, "err_word")),
            "gdn_commit_replay")


def _norm_c(norm, o):
    """The C record of a GatedNorm for outputs o (checked: shapes, dtypes)."""
    import torch

    if norm is None:
        return None
    _shape(norm.z, o.shape, "norm.z")
    _shape(norm.y, o.shape, "norm.y")
    _shape(norm.norm_weight, (o.shape[-1],), "norm.norm_weight")
    if norm.y.dtype != o.dtype:
        raise TypeError("norm.y must have o's dtype")
    if norm.norm_weight.dtype != torch.float32:
        raise TypeError("norm.norm_weight must be fp32")
    return _GatedNormC(_dev(norm.z, "norm.z"), _code(norm.z, "norm.z"), _dev(norm.norm_weight, "norm.norm_weight"),
                       float(norm.eps), _dev(norm.y, "norm.y"))


def _norm_named(norm):
    return [] if norm is None else [("norm.z", norm.z), ("norm.norm_weight", norm.norm_weight), ("norm.y", norm.y)]


def gdn_mtp_verify_gated(q, k, v, a, b, A_log, dt_bias, state_pool, state_indices, o, norm, intermediate_states=None,
                         err_word=None, *, scale=1.0, l2_eps=1e-6, stream=None) -> None:
    """``gdn_mtp_verify`` (o, optional intermediate states) and the gated RMSNorm of o into ``norm.y``
    (``norm``: a GatedNorm), inside the verify kernel where one item holds a whole head."""
    L = lib()
    d = _io_dims(q, k, v, a, b, A_log, dt_bias, state_pool, state_indices, o, scale, l2_eps)
    if intermediate_states is not None:
        _shape(intermediate_states, (d.B, d.T, d.HV, d.DV, d.DK), "intermediate_states")
        if intermediate_states.dtype != state_pool.dtype:
            raise TypeError("intermediate_states must have state_pool's dtype")
    nc = _norm_c(norm, o)
    device = _common_device(_io_named(q, k, v, a, b, A_log, dt_bias, state_pool, state_indices)
                            + [("o", o), ("intermediate_states", intermediate_states), ("err_word", err_word)]
                            + _norm_named(norm))
    _launch(device, stream, L.gdn_mtp_verify_gated,
            (ctypes.byref(d), _dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(a, "a"), _dev(b, "b"),
             _dev(A_log, "A_log"), _dev(dt_bias, "dt_bias"), _dev(state_pool, "state_pool"),
             _dev(state_indices, "state_indices"), _dev(o, "o"), _dev(intermediate_states, "intermediate_states"),
             ctypes.byref(nc), _dev(err_word, "err_word")), "gdn_mtp_verify_gated")


def gdn_mtp_verify_commit(prev, q, k, v, a, b, A_log, dt_bias, state_pool, state_indices, o, err_word=None, *,
                          norm=None, scale=1.0, l2_eps=1e-6, stream=None) -> None:
    """One speculative step in one pass: commit ``prev``'s accepted prefix (``prev``: a ``ReplayTokens``, exactly
    ``gdn_commit_replay`` of those tokens) into the slots, then verify these T tokens from the committed states
    (exactly ``gdn_mtp_verify`` without intermediate states).  ``prev`` may have another token count."""
    import torch

    L = lib()
    d = _io_dims(q, k, v, a, b, A_log, dt_bias, state_pool, state_indices, o, scale, l2_eps)
    if prev.k.dim() != 4:
        raise ValueError("prev.k is [B, T', HK, DK]")
    Tp = prev.k.shape[1]
    _shape(prev.k, (d.B, Tp, d.HK, d.DK), "prev.k")
    _shape(prev.v, (d.B, Tp, d.HV, d.DV), "prev.v")
    _shape(prev.a, (d.B, Tp, d.HV), "prev.a")
    _shape(prev.b, (d.B, Tp, d.HV), "prev.b")
    _shape(prev.accept_len, (d.B,), "prev.accept_len")
    for t, n in ((prev.k, "prev.k"), (prev.v, "prev.v"), (prev.a, "prev.a"), (prev.b, "prev.b")):
        if t.dtype != q.dtype:
            raise TypeError(f"{n} must have q's dtype")
    if prev.accept_len.dtype != torch.int32:
        raise TypeError("prev.accept_len must be int32")
    nc = _norm_c(norm, o)
    device = _common_device(_io_named(q, k, v, a, b, A_log, dt_bias, state_pool, state_indices)
                            + [("o", o), ("err_word", err_word), ("prev.k", prev.k), ("prev.v", prev.v),
                               ("prev.a", prev.a), ("prev.b", prev.b), ("prev.accept_len", prev.accept_len)]
                            + _norm_named(norm))
    rt = _ReplayTokensC(Tp, _dev(prev.k, "prev.k"), _dev(prev.v, "prev.v"), _dev(prev.a, "prev.a"),
                        _dev(prev.b, "prev.b"), _dev(prev.accept_len, "prev.accept_len"))
    _launch(device, stream, L.gdn_mtp_verify_commit,
            (ctypes.byref(d), ctypes.byref(rt), _dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(a, "a"),
             _dev(b, "b"), _dev(A_log, "A_log"), _dev(dt_bias, "dt_bias"), _dev(state_pool, "state_pool"),
             _dev(state_indices, "state_indices"), _dev(o, "o"), ctypes.byref(nc) if nc is not None else None,
             _dev(err_word, "err_word")),
            "gdn_mtp_verify_commit")


def gdn_prefill(q, k, v, a, b, A_log, dt_bias, state_pool, state_indices, cu_seqlens, o, has_initial_state=None,
                err_word=None, *, scale=1.0, l2_eps=1e-6, stream=None) -> None:
    """Prefill of ``len(cu_seqlens) - 1`` packed sequences: sequence b (tokens ``cu_seqlens[b]`` ..
    ``cu_seqlens[b+1]-1``) starts from ``state_pool[state_indices[b]]`` (or zero where
    ``has_initial_state[b] == 0``), writes o at its tokens and its final state into that slot."""
    import torch

    L = lib()
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("prefill takes packed tokens: q, k [N,HK,DK], v, o [N,HV,DV], a, b [N,HV]")
    N = q.shape[0]
    B = cu_seqlens.shape[0] - 1
    if cu_seqlens.dim() != 1 or B < 0:
        raise ValueError("cu_seqlens is [B+1]")
    if cu_seqlens.dtype != torch.int32:
        raise TypeError("cu_seqlens must be int32")
    # the [B, T] checks of the other calls, with the token axis as T of one "lane"; the indices are per prompt
    d = _io_dims(q.unsqueeze(0), k.unsqueeze(0), v.unsqueeze(0), a.unsqueeze(0), b.unsqueeze(0), A_log, dt_bias,
                 state_pool, None, o.unsqueeze(0), scale, l2_eps)
    _shape(state_indices, (B,), "state_indices")
    if state_indices.dtype != torch.int32:
        raise TypeError("state_indices must be int32")
    if has_initial_state is not None:
        _shape(has_initial_state, (B,), "has_initial_state")
        if has_initial_state.dtype != torch.int32:
            raise TypeError("has_initial_state must be int32")
    d.B, d.T = B, N
    device = _common_device(_io_named(q, k, v, a, b, A_log, dt_bias, state_pool, state_indices)
                            + [("cu_seqlens", cu_seqlens), ("o", o), ("has_initial_state", has_initial_state),
                               ("err_word", err_word)])
    _launch(device, stream, L.gdn_prefill,
            (ctypes.byref(d), _dev(cu_seqlens, "cu_seqlens"), _dev(q, "q"), _dev(k, "k"), _dev(v, "v"),
             _dev(a, "a"), _dev(b, "b"), _dev(A_log, "A_log"), _dev(dt_bias, "dt_bias"),
             _dev(state_pool, "state_pool"), _dev(state_indices, "state_indices"),
             _dev(has_initial_state, "has_initial_state"), _dev(o, "o"), _dev(err_word, "err_word")), "gdn_prefill")


def gdn_gated_rmsnorm(o, z, norm_weight, y=None, *, eps=1e-6, stream=None):
    """``y = o / sqrt(mean(o^2) + eps) * norm_weight * silu(z)`` over the last axis (DV) of o; returns y
    (a new tensor of o's shape and dtype unless given; ``y`` may be ``o`` itself)."""
    import torch

    L = lib()
    if o.dim() < 1 or tuple(z.shape) != tuple(o.shape):
        raise ValueError("z must have o's shape")
    DV = o.shape[-1]
    _shape(norm_weight, (DV,), "norm_weight")
    if norm_weight.dtype != torch.float32:
        raise TypeError("norm_weight must be fp32")
    if y is None:
        y = torch.empty_like(o)
    _shape(y, o.shape, "y")
    if y.dtype != o.dtype:
        raise TypeError("y must have o's dtype")
    rows = o.numel() // DV if DV > 0 else 0
    device = _common_device([("o", o), ("z", z), ("norm_weight", norm_weight), ("y", y)])
    _launch(device, stream, L.gdn_gated_rmsnorm,
            (rows, DV, _code(o, "o"), _code(z, "z"), _dev(o, "o"), _dev(z, "z"), _dev(norm_weight, "norm_weight"),
             float(eps), _dev(y, "y")), "gdn_gated_rmsnorm")
    return y


def _conv_dims(x, W, conv_w, conv_state, out, silu):
    """gdn_conv_dims from the tensors: x [B,T,H], W [C,H], conv_w [Cc,K], conv_state [num_slots,K-1,Cc] and the
    outputs' shapes (HK, DK from q; HV, DV from v)."""
    import torch

    if x.dim() != 3 or W.dim() != 2 or conv_w.dim() != 2 or conv_state.dim() != 3:
        raise ValueError("x is [B,T,H], W [C,H], conv_w [Cc,K], conv_state [num_slots,K-1,Cc]")
    B, T, H = x.shape
    if out.q.dim() != 4 or out.v.dim() != 4:
        raise ValueError("q and v are 4-D")
    HK, DK = out.q.shape[2], out.q.shape[3]
    HV, DV = out.v.shape[2], out.v.shape[3]
    Cc = 2 * HK * DK + HV * DV
    C = Cc + HV * DV + 2 * HV
    K = conv_w.shape[1]
    _shape(W, (C, H), "W")
    _shape(conv_w, (Cc, K), "conv_w")
    _shape(conv_state, (conv_state.shape[0], K - 1, Cc), "conv_state")
    for t, n, want in ((out.q, "q", (B, T, HK, DK)), (out.k, "k", (B, T, HK, DK)), (out.v, "v", (B, T, HV, DV)),
                       (out.z, "z", (B, T, HV, DV)), (out.b, "b", (B, T, HV)), (out.a, "a", (B, T, HV))):
        _shape(t, want, n)
    for t, n in ((x, "x"), (W, "W")):
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{n} must be bf16")
    if conv_w.dtype != torch.float32:
        raise TypeError("conv_w must be fp32")
    od = _code(out.q, "q")
    for t, n in ((out.k, "k"), (out.v, "v"), (out.z, "z"), (out.b, "b"), (out.a, "a")):
        if _code(t, n) != od:
            raise TypeError(f"{n} must have q's dtype")
    return _ConvDimsC(B, T, H, HK, HV, DK, DV, K, conv_state.shape[0], _code(conv_state, "conv_state"), od,
                      1 if silu else 0)


def gdn_in_proj_conv(x, W, conv_w, conv_b, conv_state, state_indices, out, write_state, records=None,
                     err_word=None, *, silu=True, stream=None) -> None:
    """The in_proj projection of x's rows with its causal conv1d epilogue into ``out`` (an ``InProjOut``);
    ``write_state`` (decode) moves each lane's convolution state on by its T rows, otherwise ``records``
    (``[B,T,Cc]``, conv_state's dtype) receives the pre-convolution values for ``gdn_conv_commit``."""
    import torch

    L = lib()
    d = _conv_dims(x, W, conv_w, conv_state, out, silu)
    _shape(state_indices, (d.B,), "state_indices")
    if state_indices.dtype != torch.int32:
        raise TypeError("state_indices must be int32")
    Cc = 2 * d.HK * d.DK + d.HV * d.DV
    if conv_b is not None:
        _shape(conv_b, (Cc,), "conv_b")
        if conv_b.dtype != torch.float32:
            raise TypeError("conv_b must be fp32")
    if records is not None:
        _shape(records, (d.B, d.T, Cc), "records")
        if _code(records, "records") != d.conv_dtype:
            raise TypeError("records must have conv_state's dtype")
    device = _common_device([("x", x), ("W", W), ("conv_w", conv_w), ("conv_b", conv_b), ("conv_state", conv_state),
                             ("state_indices", state_indices), ("q", out.q), ("k", out.k), ("v", out.v),
                             ("z", out.z), ("b", out.b), ("a", out.a), ("records", records), ("err_word", err_word)])
    oc = _InProjOutC(*(_dev(t, n) for t, n in ((out.q, "q"), (out.k, "k"), (out.v, "v"), (out.z, "z"),
                                                (out.b, "b"), (out.a, "a"))))
    _launch(device, stream, L.gdn_in_proj_conv,
            (ctypes.byref(d), _dev(x, "x"), _dev(W, "W"), _dev(conv_w, "conv_w"), _dev(conv_b, "conv_b"),
             _dev(conv_state, "conv_state"), _dev(state_indices, "state_indices"), 1 if write_state else 0,
             ctypes.byref(oc), _dev(records, "records"), _dev(err_word, "err_word", torch.int32)),
            "gdn_in_proj_conv")


def gdn_conv_commit(conv_state, state_indices, records, accept_len, err_word=None, *, stream=None) -> None:
    """The convolution state after each lane's first ``accept_len[b]`` verify rows, from their records."""
    import torch

    L = lib()
    if conv_state.dim() != 3 or records.dim() != 3:
        raise ValueError("conv_state is [num_slots,K-1,Cc], records [B,T,Cc]")
    B, T, Cc = records.shape
    K = conv_state.shape[1] + 1
    _shape(conv_state, (conv_state.shape[0], K - 1, Cc), "conv_state")
    _shape(state_indices, (B,), "state_indices")
    _shape(accept_len, (B,), "accept_len")
    for t, n in ((state_indices, "state_indices"), (accept_len, "accept_len")):
        if t.dtype != torch.int32:
            raise TypeError(f"{n} must be int32")
    if _code(records, "records") != _code(conv_state, "conv_state"):
        raise TypeError("records must have conv_state's dtype")
    # the commit needs only the channel count Cc = 2*HK*DK + HV*DV (at least 3): any head layout with that count
    if Cc < 3:
        raise ValueError("records: fewer than 3 channels")
    d = _ConvDimsC(B, T, 8, 1, 1, 1, Cc - 2, K, conv_state.shape[0], _code(conv_state, "conv_state"), BF16, 1)
    device = _common_device([("conv_state", conv_state), ("state_indices", state_indices), ("records", records),
                             ("accept_len", accept_len), ("err_word", err_word)])
    _launch(device, stream, L.gdn_conv_commit,
            (ctypes.byref(d), _dev(conv_state, "conv_state"), _dev(state_indices, "state_indices"),
             _dev(records, "records"), _dev(accept_len, "accept_len"), _dev(err_word, "err_word", torch.int32)),
            "gdn_conv_commit")


# ---- attention over the paged 4-bit cache ------------------------------------------------------------
# These calls take a few microseconds on the GPU, so their marshalling is kept as short as its checks allow.
def _ptr(t, name: str, dtype, shape, dev: int):
    """Address of a contiguous CUDA tensor of this dtype and shape on GPU `dev` (None -> NULL)."""
    if t is None:
        return None
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on GPU {dev}, as the other tensors of the call are: it is on {t.device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _run(dev: int, stream, fn, args, what: str) -> None:
    """One library call on GPU `dev`'s given or current stream, with that GPU current."""
    import torch

    if stream is not None:
        s = _stream(stream, torch.device("cuda", dev))
    else:
        s = torch._C._cuda_getCurrentRawStream(dev)
    if torch.cuda.current_device() == dev:
        status = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, s)
    if status != 0:
        raise GdnError(status, what)


def _gpu(t, name: str) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def gdn_page_plan(kv_lens, new_lens, page_size, block_tables, held, free_pages, taken, plan, ticket, err_word=None, *,
                  stream=None) -> None:
    """Block tables, slot map, positions and offsets of a step: lane b has ``kv_lens[b]`` cached tokens in ``held[b]``
    pages and brings ``new_lens[b]`` more.  New pages come from ``free_pages[taken:]`` into ``block_tables``
    ``[B, max_pages]``; the rest goes into ``plan`` (a ``PagePlan``).  ``ticket`` is one int32, 0 before the first call.  Of no
    lanes at all (B = 0), the plan is that of a step without tokens."""
    import torch

    L = lib()
    dev = _gpu(kv_lens, "kv_lens")
    if block_tables.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("block_tables is [B,max_pages], free_pages [num_pages]")
    i32, B = torch.int32, plan.B
    if plan.device.index != dev:
        raise ValueError(f"plan is on {plan.device}, kv_lens on GPU {dev}")
    max_pages, num_pages = block_tables.shape[1], free_pages.shape[0]
    args = (B, plan.N, page_size, max_pages, num_pages, _ptr(kv_lens, "kv_lens", i32, (B,), dev),
            _ptr(new_lens, "new_lens", i32, (B,), dev), _ptr(block_tables, "block_tables", i32, (B, max_pages), dev),
            _ptr(held, "held", i32, (B,), dev), _ptr(free_pages, "free_pages", i32, (num_pages,), dev),
            _ptr(taken, "taken", i32, (1,), dev), plan.ref, _ptr(ticket, "ticket", i32, (1,), dev),
            _ptr(err_word, "err_word", i32, (1,), dev))
    _run(dev, stream, L.gdn_page_plan, args, "gdn_page_plan")
    if B == 0:  # the library writes nothing then, and an earlier step's slots must not stay
        with torch.cuda.stream(stream):
            plan.cu_seqlens.zero_()
            plan.positions.zero_()
            plan.slot_map.fill_(-1)
            plan.taken.copy_(taken)


def _rows(t, name: str, dtype, shape, dev: int):
    """Address and token stride of a tensor ``[N, heads, D]`` whose tokens are without gaps in themselves."""
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on GPU {dev}, as the other tensors of the call are: it is on {t.device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    step, head, one = t.stride()
    if (one != 1 and shape[2] > 1) or (head != shape[2] and shape[1] > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous (strides {t.stride()})")
    return t.data_ptr(), step if shape[0] > 1 else shape[1] * shape[2]


def gdn_qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, q_out, k_out=None, *, v=None, cache=None,
                     slot_map=None, err_word=None, eps=1e-6, interleaved=False, stream=None) -> None:
    """RMS norm of every head of q ``[N,HQ,D]`` and k ``[N,HK,D]`` (any token stride) and the rotation of its first
    ``2 * len(inv_freq)`` dimensions by ``positions[n] * inv_freq`` into ``q_out`` and ``k_out``.  With ``cache`` (a
    ``Kv4Cache``), v ``[N,HK,D]`` and ``slot_map`` ``[N]``, the keys and values are stored there; k_out may be None."""
    import torch

    L = lib()
    dev = _gpu(q, "q")
    if q.dim() != 3 or k.dim() != 3 or inv_freq.dim() != 1:
        raise ValueError("q is [N,HQ,D], k [N,HK,D], inv_freq [R/2]")
    N, HQ, D = q.shape
    HK, half = k.shape[1], inv_freq.shape[0]
    dt, f32, i32 = q.dtype, torch.float32, torch.int32
    code = _code(q, "q")
    qp, qs = _rows(q, "q", dt, (N, HQ, D), dev)
    kp, ks = _rows(k, "k", dt, (N, HK, D), dev)
    vp, vs = (None, 0) if v is None else _rows(v, "v", dt, (N, HK, D), dev)
    if cache is not None and cache.device.index != dev:
        raise ValueError(f"cache is on {cache.device}, q on GPU {dev}")
    d = _QkDimsC(N, HQ, HK, D, 2 * half, 1 if interleaved else 0, code, qs, ks, vs, eps)
    _run(dev, stream, L.gdn_qk_norm_rope,
         (ctypes.byref(d), qp, kp, _ptr(q_weight, "q_weight", f32, (D,), dev), _ptr(k_weight, "k_weight", f32, (D,), dev),
          _ptr(positions, "positions", i32, (N,), dev), _ptr(inv_freq, "inv_freq", f32, (half,), dev),
          _ptr(q_out, "q_out", dt, (N, HQ, D), dev), _ptr(k_out, "k_out", dt, (N, HK, D), dev), vp,
          None if cache is None else cache.ref, _ptr(slot_map, "slot_map", i32, (N,), dev),
          _ptr(err_word, "err_word", i32, (1,), dev)), "gdn_qk_norm_rope")


def gdn_kv4_read(cache, slot_map, k_out, v_out, err_word=None, *, stream=None) -> None:
    """The cached rows of ``slot_map`` ``[N]`` as numbers: ``k_out``, ``v_out`` ``[N,HK,D]`` bf16."""
    import torch

    L = lib()
    dev, N, bf16 = _gpu(slot_map, "slot_map"), slot_map.shape[0], torch.bfloat16
    if cache.device.index != dev:
        raise ValueError(f"cache is on {cache.device}, slot_map on GPU {dev}")
    shape = (N, cache.HK, cache.D)
    _run(dev, stream, L.gdn_kv4_read,
         (cache.ref, N, _ptr(slot_map, "slot_map", torch.int32, (N,), dev), _ptr(k_out, "k_out", bf16, shape, dev),
          _ptr(v_out, "v_out", bf16, shape, dev), _ptr(err_word, "err_word", torch.int32, (1,), dev)), "gdn_kv4_read")


def kv4_attention_workspace(B, max_q, HQ, HK, D, device=None):
    """A workspace for ``gdn_kv4_attention`` calls of up to B lanes and max_q tokens a lane (one call at a time)."""
    import torch

    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(device):
        n = lib().gdn_kv4_attention_workspace(B, max_q, HQ, HK, D)
    if n < 0:
        raise ValueError(f"kv4_attention_workspace: sizes out of range (B {B}, max_q {max_q}, HQ {HQ}, HK {HK}, D {D})")
    return torch.empty(n, dtype=torch.uint8, device=device)


def gdn_kv4_attention(q, cache, block_tables, kv_lens, o, workspace, *, cu_seqlens=None, max_q=None, lse=None, scale=None,
                      err_word=None, stream=None) -> None:
    """Causal attention of q ``[N,HQ,D]`` bf16 over each lane's cached tokens (``kv_lens`` ``[B]``, the step's own
    included) into ``o`` and, if given, ``lse`` ``[N,HQ]`` fp32.  Lane b's rows are ``cu_seqlens[b] .. cu_seqlens[b+1]-1``
    (then ``max_q``, the most of any lane, has to be given), or N / B rows each.  ``scale`` is 1 / sqrt(D) by default."""
    import torch

    L = lib()
    dev = _gpu(q, "q")
    if q.dim() != 3 or block_tables.dim() != 2:
        raise ValueError("q is [N,HQ,D], block_tables [B,max_pages]")
    N, HQ, D = q.shape
    B, max_pages = block_tables.shape
    bf16, i32 = torch.bfloat16, torch.int32
    if cu_seqlens is None:
        if B > 0 and N % B != 0:
            raise ValueError(f"q: {N} rows are not the same number for each of {B} lanes: give cu_seqlens")
        max_q = max(1, N // B) if B > 0 else 1
    elif max_q is None:
        raise ValueError("max_q, the most tokens of a lane, goes with cu_seqlens")
    if cache.device.index != dev:
        raise ValueError(f"cache is on {cache.device}, q on GPU {dev}")
    if D != cache.D:
        raise ValueError(f"q: head dimension {D}, the cache's is {cache.D}")
    d = _Kv4AttentionDimsC(B, N, max_q, HQ, max_pages, D ** -0.5 if scale is None else scale)
    _run(dev, stream, L.gdn_kv4_attention,
         (ctypes.byref(d), cache.ref, _ptr(q, "q", bf16, (N, HQ, D), dev),
          _ptr(cu_seqlens, "cu_seqlens", i32, (B + 1,), dev), _ptr(block_tables, "block_tables", i32, (B, max_pages), dev),
          _ptr(kv_lens, "kv_lens", i32, (B,), dev), _ptr(o, "o", bf16, (N, HQ, D), dev),
          _ptr(lse, "lse", torch.float32, (N, HQ), dev),
          _ptr(workspace, "workspace", torch.uint8, (workspace.numel(),), dev), workspace.numel(),
          _ptr(err_word, "err_word", i32, (1,), dev)), "gdn_kv4_attention")
