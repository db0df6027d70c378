"""GB300-native K-draft verify step for MTP speculative decoding.

Thin ctypes binding over ``libspecverify.so`` (see ``include/specverify.h``).
Every compute function has the same name and argument order as its C entry
point; this module only marshals torch tensors (device memory) and the
current CUDA stream into pointers and sizes.  All arithmetic happens in the
library's CUDA kernels; there is no Python or CPU fallback, and a missing
library raises immediately.

    import speculative_decoding_verify_08_gb300 as sv
    packed = sv.prepack(codes, scales, biases)          # once per matrix
    ws = sv.workspace(sv.qmm_workspace_bytes(M, N, K))  # zeroed scratch
    sv.qmm_small_m(x, packed, y, M, N, K, ws)           # y = x @ W^T

The calls over a paged cache take their sizes from the tensors' shapes and their
strides as they are (a slice of a fused projection's rows will do); all operands
live on the current device:

    phases = sv.rope_phases(inv_freq)                   # once per model
    cache = sv.PagedKV(k_pages, v_pages, layout="HND")  # bf16 or e4m3 pages
    sv.qk_norm_rope(q, k, q_rot, k_rot, positions, phases)           # a prompt
    sv.window_attn(q_rot, k_rot, v, o, cu_rows, cu_rows, scale, window=1024)
    sv.paged_kv_append(k, v, cache, slots, q=q, q_out=q_rot,         # new tokens
                       positions=positions, phases=phases)
    sv.paged_attn(q_rot, cache, block_table, lens, o, M, scale, workspace=ws)
    sv.paged_chunk_attn(q, cache, block_table, lens, o, cu_rows, scale,     # prompts in chunks
                        workspace=ws)
    sv.gdn_chunk(states, places, q, k, v, g, beta, o, cu_rows, workspace=ws)   # recurrent layers
    sv.gdn_step(states, places, q, k, v, g, beta, o, M, tape=last_round, n_replay=accepted)
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

import torch

__all__ = [
    "load", "SvError", "SV_OK", "SV_ERR_INVALID_ARG", "SV_ERR_UNSUPPORTED", "SV_ERR_CUDA",
    "SV_ERR_TIMEOUT", "SV_ERR_WORKSPACE", "SV_ERR_OVERFLOW", "SV_BF16", "SV_F32", "SV_LAUNCH_PDL",
    "SV_LAUNCH_QMM_CUDA_CORES", "SV_LAUNCH_ATTN_MMA_SYNC", "SV_LAUNCH_ATTN_TCGEN05",
    "SV_LAUNCH_TEST_STALL_COPY",
    "qmm_packed_bytes", "qmm_prepack", "qmm_workspace_bytes", "qmm_small_m",
    "qmm8_packed_bytes", "qmm8_prepack", "qmm8_workspace_bytes", "qmm8_small_m",
    "verify_attn_workspace_bytes", "verify_attn", "verify_attn_masked", "verify_attn_noalloc", "spec_accept_workspace_bytes", "spec_accept",
    "qmm_topk_lists_bytes", "qmm_small_m_topk", "spec_accept_draft_select", "spec_accept_lists",
    "sv_status_string", "sv_last_device_error", "sv_set_launch_flags", "sv_get_launch_flags",
    "sv_kernel_launch_count", "prepack", "workspace", "library_path", "spec_pick_depth",
    "gdn_verify",
    "SV_E4M3", "rope_phases", "qk_norm_rope", "PagedKV", "paged_kv_append",
    "paged_attn_workspace_bytes", "paged_attn", "window_attn_workspace_bytes", "window_attn",
    "paged_chunk_attn_workspace_bytes", "paged_chunk_attn", "gdn_step", "gdn_chunk_workspace_bytes", "gdn_chunk",
]

SV_OK, SV_ERR_INVALID_ARG, SV_ERR_UNSUPPORTED, SV_ERR_CUDA = 0, 1, 2, 3
SV_ERR_TIMEOUT, SV_ERR_WORKSPACE, SV_ERR_OVERFLOW = 4, 5, 6
SV_BF16, SV_F32, SV_E4M3 = 0, 1, 2
SV_LAUNCH_PDL = 1
SV_LAUNCH_QMM_CUDA_CORES = 2  # measurement aid: qmm on CUDA-core FFMA at M = 1 and 4
SV_LAUNCH_ATTN_MMA_SYNC = 4  # verify_attn on the mma.sync kernel
SV_LAUNCH_ATTN_TCGEN05 = 8   # verify_attn on the tcgen05 kernel
SV_LAUNCH_TEST_STALL_COPY = 0x10000  # test aid: waits of attention (not tcgen05 verify_attn) and matmul run out

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "lib", "libspecverify.so")
_lock = threading.Lock()
_lib = None


class SvError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {sv_status_string(status)} (status {status})")


class _Sampling(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_float), ("top_k", ctypes.c_int32),
                ("top_p", ctypes.c_float)]


def library_path() -> str:
    return _LIB_PATH


def load():
    """Load libspecverify.so (built by ``__graft_entry__.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"{_LIB_PATH} is missing: build the CUDA library first "
                "(python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(_LIB_PATH)
        P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L = ctypes.c_int64
        sig = {
            "qmm_packed_bytes": (Z, [I, I, I]),
            "qmm_prepack": (I, [P, P, P, I, I, I, P, Z, P]),
            "qmm_workspace_bytes": (Z, [I, I, I]),
            "qmm_small_m": (I, [P, P, P, I, I, I, I, I, P, Z, P]),
            "qmm8_packed_bytes": (Z, [I, I, I]),
            "qmm8_prepack": (I, [P, P, P, I, I, I, P, Z, P]),
            "qmm8_workspace_bytes": (Z, [I, I, I]),
            "qmm8_small_m": (I, [P, P, P, I, I, I, I, I, P, Z, P]),
            "verify_attn_workspace_bytes": (Z, [I, I, I, I, L]),
            "verify_attn": (I, [P, P, P, P, I, I, I, I, L, L, ctypes.c_float, P, Z, P]),
            "verify_attn_noalloc": (I, [P, P, P, P, I, I, I, I, L, L, ctypes.c_float, P]),
            "verify_attn_masked": (I, [P, P, P, P, I, I, I, I, L, L, ctypes.c_float, P, P, Z, P]),
            "spec_accept_workspace_bytes": (Z, [I, I, I]),
            "spec_accept": (I, [P, P, I, P, P, _Sampling, I, I, I, P, P, P, Z, P]),
            "qmm_topk_lists_bytes": (Z, [I, I, I]),
            "qmm_small_m_topk": (I, [P, P, P, I, I, I, I, _Sampling, P, Z, P, Z, P]),
            "spec_accept_draft_select": (I, [P, I, _Sampling, I, I, I, P, Z, P]),
            "spec_accept_lists": (I, [P, P, P, P, _Sampling, I, I, I, P, P, P, Z, P]),
            "sv_status_string": (ctypes.c_char_p, [I]),
            "sv_last_device_error": (I, [P]),
            "sv_set_launch_flags": (None, [ctypes.c_uint]),
            "sv_get_launch_flags": (ctypes.c_uint, []),
            "sv_kernel_launch_count": (ctypes.c_uint64, []),
            "spec_pick_depth": (I, [P, P, P, I, P]),
            "gdn_verify": (I, [P, P, P, P, P, I, P, P, P, P, P, P, I, I, I, I, I, I, P]),
            "rope_phases": (I, [P, I, P]),
            "qk_norm_rope": (I, [P, P, P, P, P, P, I, I, I, I, P]),
            "paged_kv_append": (I, [P, P, P, P, P, P, P, P, I, I, I, I, P]),
            "paged_kv_maps": (I, [P, I, I, P, Z]),
            "paged_attn_workspace_bytes": (Z, [I, I, I, I, I]),
            "paged_attn": (I, [P, P, P, L, I, P, P, I, I, I, I, I, ctypes.c_float, I, I, P, Z, P]),
            "window_attn_workspace_bytes": (Z, [I, I, I, I]),
            "paged_chunk_attn_workspace_bytes": (Z, [I, I, I, I, I]),
            "paged_chunk_attn": (I, [P, P, P, L, I, P, P, P, I, I, I, I, I, ctypes.c_float, I, I, P, Z, P]),
            "gdn_step": (I, [P, P, P, P, P, P, P, I, P, P, P, P, P, P, I, I, I, I, I, I, I, I, P]),
            "gdn_chunk_workspace_bytes": (Z, [I, I, I, I, I, I]),
            "gdn_chunk": (I, [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, P, Z, P]),
            "window_attn": (I, [P, P, P, P, P, P, I, I, I, I, I, I, ctypes.c_float, I, I, P, Z, P]),
        }
        for name, (res, args) in sig.items():
            f = getattr(lib, name)
            f.restype = res
            f.argtypes = args
        _lib = lib
        return lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str):
    if status != SV_OK:
        raise SvError(status, where)


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


# ------------------------------------------------------------- queries ----
def sv_status_string(status: int) -> str:
    return load().sv_status_string(int(status)).decode()


def qmm_packed_bytes(N: int, K: int, group: int = 64) -> int:
    return load().qmm_packed_bytes(N, K, group)


def qmm_workspace_bytes(M: int, N: int, K: int) -> int:
    return load().qmm_workspace_bytes(M, N, K)


def qmm8_packed_bytes(N: int, K: int, group: int = 64) -> int:
    return load().qmm8_packed_bytes(N, K, group)


def qmm8_workspace_bytes(M: int, N: int, K: int) -> int:
    return load().qmm8_workspace_bytes(M, N, K)


def verify_attn_workspace_bytes(M: int, Hq: int, Hkv: int, D: int, kv_len: int) -> int:
    return load().verify_attn_workspace_bytes(M, Hq, Hkv, D, kv_len)


def spec_accept_workspace_bytes(R: int, K: int, V: int) -> int:
    return load().spec_accept_workspace_bytes(R, K, V)


def sv_set_launch_flags(flags: int) -> None:
    load().sv_set_launch_flags(int(flags))


def sv_get_launch_flags() -> int:
    return load().sv_get_launch_flags()


def sv_kernel_launch_count() -> int:
    return load().sv_kernel_launch_count()


def sv_last_device_error(stream=None) -> int:
    return load().sv_last_device_error(_stream(stream))


# ------------------------------------------------------------- compute ----
def qmm_prepack(codes, scales, biases, N: int, K: int, group: int, packed_out, stream=None):
    _check(load().qmm_prepack(_ptr(codes), _ptr(scales), _ptr(biases), N, K, group,
                              _ptr(packed_out), _nbytes(packed_out), _stream(stream)),
           "qmm_prepack")


def qmm_small_m(x, packed_w, y, M: int, N: int, K: int, workspace=None, group: int = 64,
                stream=None):
    ydt = SV_F32 if y.dtype == torch.float32 else SV_BF16
    _check(load().qmm_small_m(_ptr(x), _ptr(packed_w), _ptr(y), ydt, M, N, K, group,
                              _ptr(workspace), _nbytes(workspace), _stream(stream)),
           "qmm_small_m")


def qmm8_prepack(codes, scales, biases, N: int, K: int, group: int, packed_out, stream=None):
    _check(load().qmm8_prepack(_ptr(codes), _ptr(scales), _ptr(biases), N, K, group,
                               _ptr(packed_out), _nbytes(packed_out), _stream(stream)),
           "qmm8_prepack")


def qmm8_small_m(x, packed_w, y, M: int, N: int, K: int, workspace=None, group: int = 64,
                 stream=None):
    ydt = SV_F32 if y.dtype == torch.float32 else SV_BF16
    _check(load().qmm8_small_m(_ptr(x), _ptr(packed_w), _ptr(y), ydt, M, N, K, group,
                               _ptr(workspace), _nbytes(workspace), _stream(stream)),
           "qmm8_small_m")


def verify_attn(q, k_cache, v_cache, o, M: int, Hq: int, Hkv: int, D: int, kv_len: int,
                kv_stride_tokens: int, scale: float, workspace=None, stream=None):
    _check(load().verify_attn(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(o), M, Hq, Hkv, D,
                              kv_len, kv_stride_tokens, float(scale), _ptr(workspace),
                              _nbytes(workspace), _stream(stream)),
           "verify_attn")


def verify_attn_masked(q, k_cache, v_cache, o, M: int, Hq: int, Hkv: int, D: int, kv_len: int,
                       kv_stride_tokens: int, scale: float, draft_mask, workspace=None, stream=None):
    """verify_attn over a draft tree: draft_mask is a device int32/uint32
    tensor [M]; bit j of draft_mask[i] lets row i see draft slot kv_len-M+j."""
    _check(load().verify_attn_masked(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(o), M, Hq, Hkv,
                                     D, kv_len, kv_stride_tokens, float(scale), _ptr(draft_mask),
                                     _ptr(workspace), _nbytes(workspace), _stream(stream)),
           "verify_attn_masked")


def verify_attn_noalloc(q, k_cache, v_cache, o, M: int, Hq: int, Hkv: int, D: int,
                        kv_len: int, kv_stride_tokens: int, scale: float, stream=None):
    """verify_attn without a workspace argument, for callers that cannot
    allocate device memory; its scratch is a fixed 16 MiB array inside the
    library (see include/specverify.h for the rules of use)."""
    _check(load().verify_attn_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(o), M, Hq,
                                      Hkv, D, kv_len, kv_stride_tokens, float(scale),
                                      _stream(stream)),
           "verify_attn_noalloc")


def spec_accept(target_logits, draft_logits, draft_tokens, uniforms, temperature: float,
                top_k: int, top_p: float, R: int, K: int, V: int, out_tokens,
                out_num_accepted, workspace=None, stream=None):
    dt = SV_BF16 if target_logits.dtype == torch.bfloat16 else SV_F32
    sp = _Sampling(float(temperature), int(top_k), float(top_p))
    _check(load().spec_accept(_ptr(target_logits), _ptr(draft_logits), dt, _ptr(draft_tokens),
                              _ptr(uniforms), sp, R, K, V, _ptr(out_tokens),
                              _ptr(out_num_accepted), _ptr(workspace), _nbytes(workspace),
                              _stream(stream)),
           "spec_accept")


def qmm_topk_lists_bytes(M: int, N: int, K: int) -> int:
    return load().qmm_topk_lists_bytes(M, N, K)


def qmm_small_m_topk(x, packed_w, y, M: int, N: int, K: int, temperature: float, top_k: int,
                     top_p: float, lists, workspace=None, group: int = 64, stream=None):
    sp = _Sampling(float(temperature), int(top_k), float(top_p))
    _check(load().qmm_small_m_topk(_ptr(x), _ptr(packed_w), _ptr(y), M, N, K, group, sp, _ptr(lists),
                                   _nbytes(lists), _ptr(workspace), _nbytes(workspace),
                                   _stream(stream)),
           "qmm_small_m_topk")


def spec_accept_draft_select(draft_logits, temperature: float, top_k: int, top_p: float, R: int,
                             K: int, V: int, workspace, stream=None):
    dt = SV_BF16 if draft_logits.dtype == torch.bfloat16 else SV_F32
    sp = _Sampling(float(temperature), int(top_k), float(top_p))
    _check(load().spec_accept_draft_select(_ptr(draft_logits), dt, sp, R, K, V, _ptr(workspace),
                                           _nbytes(workspace), _stream(stream)),
           "spec_accept_draft_select")


def spec_accept_lists(target_lists, draft_tokens, uniforms, temperature: float, top_k: int,
                      top_p: float, R: int, K: int, V: int, out_tokens, out_num_accepted,
                      workspace, draft_lists=None, stream=None):
    sp = _Sampling(float(temperature), int(top_k), float(top_p))
    _check(load().spec_accept_lists(_ptr(target_lists), _ptr(draft_lists), _ptr(draft_tokens),
                                    _ptr(uniforms), sp, R, K, V, _ptr(out_tokens),
                                    _ptr(out_num_accepted), _ptr(workspace), _nbytes(workspace),
                                    _stream(stream)),
           "spec_accept_lists")


# ------------------------------------------------------------- helpers ----
def workspace(nbytes: int, device=None):
    """Zero-filled device scratch of at least ``nbytes`` bytes (None if 0)."""
    if nbytes <= 0:
        return None
    dev = device if device is not None else torch.device("cuda")
    return torch.zeros(((nbytes + 255) // 256) * 256, dtype=torch.uint8, device=dev)


def prepack(codes, scales, biases, group: int = 64, stream=None, bits: int = 4):
    """Allocate and fill the prepacked weight buffer of an [N, K] matrix
    (4-bit codes [N, K/8], or 8-bit codes [N, K/4] with bits=8)."""
    if bits not in (4, 8):
        raise SvError(SV_ERR_UNSUPPORTED, "prepack")
    N, KW = codes.shape
    K = KW * (32 // bits)
    nb = (qmm_packed_bytes if bits == 4 else qmm8_packed_bytes)(N, K, group)
    if nb == 0:
        raise SvError(SV_ERR_UNSUPPORTED, "qmm_packed_bytes")
    out = torch.empty(nb, dtype=torch.uint8, device=codes.device)
    (qmm_prepack if bits == 4 else qmm8_prepack)(codes, scales, biases, N, K, group, out, stream=stream)
    return out


def spec_pick_depth(verify_us, accept, draft_us=None):
    """Draft depth with the most tokens per microsecond (0 unless it beats
    plain decoding) and every depth's rate.  verify_us[K]: cost of a verify
    pass with K+1 rows; accept[i-1]: P(at least i drafts accepted)."""
    import numpy as np
    v = np.ascontiguousarray(verify_us, dtype=np.float64).ravel()
    a = np.ascontiguousarray(accept, dtype=np.float64).ravel()
    kmax = v.shape[0] - 1
    if a.shape[0] != kmax:
        raise SvError(SV_ERR_INVALID_ARG, "spec_pick_depth")
    d = None if draft_us is None else np.ascontiguousarray(draft_us, dtype=np.float64).ravel()
    rates = np.zeros(kmax + 1, dtype=np.float64)
    k = load().spec_pick_depth(v.ctypes.data, None if d is None else d.ctypes.data,
                               a.ctypes.data if kmax > 0 else None, kmax, rates.ctypes.data)
    if k < 0:
        raise SvError(SV_ERR_INVALID_ARG, "spec_pick_depth")
    return k, rates


def gdn_verify(state, q, k, v, g, beta, o, tape=None, n_replay=0, stream=None):
    """GatedDeltaNet verify step: commits the first n_replay tokens of the
    previous round's tape (k, v, g, beta) into `state` (fp32 [Hv, dv, dk]),
    then runs this round's rows into `o`.  q, k bf16 [M, Hk, dk]; v bf16
    [M, Hv, dv]; g, beta fp32 [M, Hv]."""
    Hv, dv, dk = state.shape
    M, Hk = (k.shape[0], k.shape[1]) if k is not None else (0, tape[0].shape[1])
    tk, tv, tg, tb = tape if tape is not None else (None, None, None, None)
    odt = SV_F32 if (o is not None and o.dtype == torch.float32) else SV_BF16
    _check(load().gdn_verify(_ptr(state), _ptr(tk), _ptr(tv), _ptr(tg), _ptr(tb), int(n_replay),
                             _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(o), odt, M, Hk, Hv,
                             dk, dv, _stream(stream)),
           "gdn_verify")


# --------------------------------------------- rows, rotations, paged cache ----
# C structs passed by address, packed per call: a pack() is a fraction of a
# microsecond, where filling a ctypes.Structure takes several.
_ROWS = struct.Struct("Pqq")            # sv_rows
_NORM = struct.Struct("PPff")           # sv_head_norm
_ROTATION = struct.Struct("PPii")       # sv_rotation
_PAGED_KV = struct.Struct("PPPPqqqqiiP")  # sv_paged_kv
_STATES = struct.Struct("Pqq")          # sv_states
_PAGED_MAPS_BYTES = 256


def _bad(where: str, status: int = SV_ERR_INVALID_ARG):
    raise SvError(status, where)


# What a call checks here is what the library cannot see (types, shapes, that
# memory is the current GPU's); one attribute of a tensor costs about 0.1 us.
_BF16 = torch.bfloat16


# GPUs of this process, once known.  With one, what is a GPU's is on it, and
# asking every tensor for its device (0.2 us each) is left out.
_gpus = 0


def _device(t, where):
    """The device of a call, that of its first operand.  The library launches on
    the current one, so it has to be that, and the other operands' too.  None:
    the only one there is."""
    global _gpus
    d = t.get_device()
    if d < 0 or d != torch._C._cuda_getDevice():
        _bad(where)
    _gpus = _gpus or torch._C._cuda_getDeviceCount()
    return d if _gpus > 1 else None


def _rows(t, tokens, heads, D, dev, where):
    """sv_rows of a bf16 tensor [tokens, heads, D] of the call's device (any strides, D contiguous)."""
    if t.dtype is not _BF16 or t.shape != (tokens, heads, D) or not t.is_cuda or (
            dev is not None and t.get_device() != dev):
        _bad(where)
    ts, hs, ds = t.stride()
    if ds != 1:
        _bad(where)
    # a dimension of one may carry any stride
    return _ROWS.pack(t.data_ptr(), ts if tokens > 1 else 0, hs if heads > 1 else 0)


def _vector(t, dtype, n, dev, where):
    """Address of a contiguous tensor of n values of the call's device."""
    if t.dtype is not dtype or t.numel() != n or not t.is_cuda or not t.is_contiguous() or (
            dev is not None and t.get_device() != dev):
        _bad(where)
    return t.data_ptr()


def _launch_stream(dev, stream):
    """The given stream, or the current one of the call's device."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev or 0)
    return _stream(stream)


def rope_phases(inv_freq, device=None):
    """Device table of a rotation (int64 [rot_dim/2], the bits of fractions of
    a turn in 2^-64) from its inverse frequencies in radians per position."""
    import numpy as np
    if isinstance(inv_freq, torch.Tensor):
        inv_freq = inv_freq.detach().cpu().double().numpy()
    f = np.ascontiguousarray(inv_freq, dtype=np.float64).ravel()
    out = np.empty(f.shape[0], dtype=np.uint64)
    _check(load().rope_phases(f.ctypes.data, f.shape[0], out.ctypes.data), "rope_phases")
    return torch.from_numpy(out.view(np.int64)).to(device if device is not None else torch.device("cuda"))


def _norm_rotation(q_weight, k_weight, eps, weight_offset, positions, phases, interleaved, T, D, dev, where):
    norm = rot = None
    if q_weight is not None or k_weight is not None:
        norm = _NORM.pack(0 if q_weight is None else _vector(q_weight, _BF16, D, dev, where),
                          0 if k_weight is None else _vector(k_weight, _BF16, D, dev, where),
                          eps, weight_offset)
    if phases is not None:
        if positions is None:
            _bad(where)
        half = phases.numel()
        rot = _ROTATION.pack(_vector(phases, torch.int64, half, dev, where),
                             _vector(positions, torch.int32, T, dev, where), 2 * half, 1 if interleaved else 0)
    return norm, rot


def qk_norm_rope(q, k, q_out, k_out, positions=None, phases=None, q_weight=None, k_weight=None,
                 eps: float = 1e-6, weight_offset: float = 0.0, interleaved: bool = False, stream=None):
    """RMS norm (where a weight is given) and position rotation (where phases
    are) of query and key rows [T, heads, D] in one pass; q_out and k_out may
    be q and k themselves.  rot_dim = 2 * phases.numel()."""
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    w = "qk_norm_rope"
    dev = None if _gpus == 1 else _device(q, w)
    norm, rot = _norm_rotation(q_weight, k_weight, eps, weight_offset, positions, phases, interleaved, T, D, dev, w)
    status = load().qk_norm_rope(_rows(q, T, Hq, D, dev, w), _rows(k, T, Hkv, D, dev, w),
                                 _rows(q_out, T, Hq, D, dev, w), _rows(k_out, T, Hkv, D, dev, w), norm, rot, T, Hq,
                                 Hkv, D, _launch_stream(dev, stream))
    if status:
        _check(status, w)


class PagedKV:
    """A paged cache: k and v are CUDA tensors of one shape and one set of
    strides, [pages, slots, heads, D] ("NHD") or [pages, heads, slots, D]
    ("HND"), bf16 or float8_e4m3fn; with the latter, the stored value times
    k_scale[head] (v_scale[head], fp32 [heads], None for 1) counts.  Holds the
    tensors and what the calls need of them, worked out once: its attributes
    are read-only, and a copy (copy, deepcopy, pickle) is made anew from the
    copied tensors."""

    def __init__(self, k, v, layout: str = "NHD", k_scale=None, v_scale=None):
        w = "PagedKV"
        if layout not in ("NHD", "HND") or k.dim() != 4 or k.shape != v.shape:
            _bad(w)
        # a dimension of one may carry any stride: here a row's, which is a valid one
        strides, of_v = ([s if n > 1 else k.shape[3] for n, s in zip(t.shape[:3], t.stride())] for t in (k, v))
        if strides != of_v:
            _bad(w)
        if k.dtype not in (torch.bfloat16, torch.float8_e4m3fn) or v.dtype is not k.dtype:
            _bad(w)
        device = k.get_device()
        if device < 0 or v.get_device() != device or k.stride(3) != 1 or v.stride(3) != 1:
            _bad(w)
        slot, head = (1, 2) if layout == "NHD" else (2, 1)
        page_size, heads, D = k.shape[slot], k.shape[head], k.shape[3]
        fields = (k.data_ptr(), v.data_ptr(),
                  0 if k_scale is None else _vector(k_scale, torch.float32, heads, device, w),
                  0 if v_scale is None else _vector(v_scale, torch.float32, heads, device, w),
                  strides[0], strides[slot], strides[head], k.shape[0], page_size,
                  SV_BF16 if k.dtype is torch.bfloat16 else SV_E4M3)
        packed, maps = _PAGED_KV.pack(*fields, 0), None
        if D in (128, 256):  # what paged_attn reads
            maps = (ctypes.c_uint64 * (_PAGED_MAPS_BYTES // 8))()
            _check(load().paged_kv_maps(packed, heads, D, maps, _PAGED_MAPS_BYTES), w)
            packed = _PAGED_KV.pack(*fields, ctypes.addressof(maps))
        self.__dict__.update(k=k, v=v, k_scale=k_scale, v_scale=v_scale, layout=layout, device=device,
                             page_size=page_size, heads=heads, D=D, packed=packed, _maps=maps)

    def __setattr__(self, name, value):
        raise AttributeError(f"PagedKV.{name} is read-only: make another PagedKV")

    def __delattr__(self, name):
        raise AttributeError(f"PagedKV.{name} is read-only")

    def __reduce__(self):  # `packed` and `_maps` hold addresses
        return type(self), (self.k, self.v, self.layout, self.k_scale, self.v_scale)


def paged_kv_append(k, v, cache: PagedKV, slots, q=None, q_out=None, positions=None, phases=None,
                    q_weight=None, k_weight=None, eps: float = 1e-6, weight_offset: float = 0.0,
                    interleaved: bool = False, stream=None):
    """Write the keys [T, heads, D] (normed and rotated as in qk_norm_rope) and
    values of T tokens to slots int64 [T] of the cache (negative: skipped),
    and in the same launch the queries' rows to q_out when q is given."""
    T, Hkv, D = k.shape
    w = "paged_kv_append"
    dev = None if _gpus == 1 else _device(k, w)
    if Hkv != cache.heads or D != cache.D or (q is None) != (q_out is None) or (
            dev is not None and dev != cache.device):
        _bad(w)
    Hq = 0 if q is None else q.shape[1]
    norm, rot = _norm_rotation(q_weight if q is not None else None, k_weight, eps, weight_offset, positions,
                               phases, interleaved, T, D, dev, w)
    status = load().paged_kv_append(None if q is None else _rows(q, T, Hq, D, dev, w),
                                    None if q is None else _rows(q_out, T, Hq, D, dev, w),
                                    _rows(k, T, Hkv, D, dev, w), _rows(v, T, Hkv, D, dev, w), cache.packed,
                                    _vector(slots, torch.int64, T, dev, w), norm, rot, T, Hq, Hkv, D,
                                    _launch_stream(dev, stream))
    if status:
        _check(status, w)


def paged_attn_workspace_bytes(B: int, M: int, Hq: int, Hkv: int, D: int) -> int:
    return load().paged_attn_workspace_bytes(B, M, Hq, Hkv, D)


def paged_attn(q, cache: PagedKV, block_table, kv_lens, o, M: int, scale: float, window: int = 0,
               sinks: int = 0, workspace=None, stream=None):
    """Attention of the newest M rows of each sequence over the cache: q and o
    [B*M, Hq, D], block_table int32 [B, width], kv_lens int32 [B]; window 0:
    none; sinks: first positions that stay visible under a window."""
    rows, Hq, D = q.shape
    w = "paged_attn"
    B, width = block_table.shape
    dev = None if _gpus == 1 else _device(q, w)
    if (D != cache.D or rows != B * M or block_table.dtype is not torch.int32 or not block_table.is_cuda
            or (workspace is not None and not workspace.is_cuda)):
        _bad(w)
    if dev is not None and (dev != cache.device or block_table.get_device() != dev
                            or (workspace is not None and workspace.get_device() != dev)):
        _bad(w)
    ts, es = block_table.stride()
    if es != 1 and width != 1:
        _bad(w)
    status = load().paged_attn(_rows(q, rows, Hq, D, dev, w), cache.packed, block_table.data_ptr(), ts, width,
                               _vector(kv_lens, torch.int32, B, dev, w), _rows(o, rows, Hq, D, dev, w), B, M, Hq,
                               cache.heads, D, scale, window, sinks, _ptr(workspace), _nbytes(workspace),
                               _launch_stream(dev, stream))
    if status:
        _check(status, w)


def window_attn_workspace_bytes(B: int, Hq: int, Hkv: int, D: int) -> int:
    return load().window_attn_workspace_bytes(B, Hq, Hkv, D)


def window_attn(q, k, v, o, cu_q, cu_k, scale: float, window: int = 0, sinks: int = 0, workspace=None,
                stream=None):
    """Causal attention of packed prompts: q and o [Tq, Hq, D], k and v [Tk,
    Hkv, D]; sequence b is rows cu_q[b]..cu_q[b+1] (int32 [B+1]) against keys
    cu_k[b]..cu_k[b+1], its last row at its last key."""
    Tq, Hq, D = q.shape
    Tk, Hkv, _ = k.shape
    w = "window_attn"
    n = cu_q.shape[0]
    dev = None if _gpus == 1 else _device(q, w)
    status = load().window_attn(_rows(q, Tq, Hq, D, dev, w), _rows(k, Tk, Hkv, D, dev, w),
                                _rows(v, Tk, Hkv, D, dev, w), _rows(o, Tq, Hq, D, dev, w),
                                _vector(cu_q, torch.int32, n, dev, w), _vector(cu_k, torch.int32, n, dev, w), n - 1,
                                Tq, Tk, Hq, Hkv, D, scale, window, sinks, _ptr(workspace), _nbytes(workspace),
                                _launch_stream(dev, stream))
    if status:
        _check(status, w)


def paged_chunk_attn_workspace_bytes(B: int, Tq: int, Hq: int, Hkv: int, D: int) -> int:
    return load().paged_chunk_attn_workspace_bytes(B, Tq, Hq, Hkv, D)


def paged_chunk_attn(q, cache: PagedKV, block_table, kv_lens, o, cu_q, scale: float, window: int = 0,
                     sinks: int = 0, workspace=None, stream=None):
    """Attention of ragged chunks of new tokens over the cache that already
    holds them: q and o [Tq, Hq, D], sequence b rows cu_q[b]..cu_q[b+1] (int32
    [B+1]), its last row at position kv_lens[b] - 1 (int32 [B]); block_table
    int32 [B, width]; window 0: none; sinks: first positions that stay visible
    under a window."""
    Tq, Hq, D = q.shape
    w = "paged_chunk_attn"
    B, width = block_table.shape
    dev = None if _gpus == 1 else _device(q, w)
    if (D != cache.D or block_table.dtype is not torch.int32 or not block_table.is_cuda
            or (workspace is not None and not workspace.is_cuda)):
        _bad(w)
    if dev is not None and (dev != cache.device or block_table.get_device() != dev
                            or (workspace is not None and workspace.get_device() != dev)):
        _bad(w)
    ts, es = block_table.stride()
    if es != 1 and width != 1:
        _bad(w)
    status = load().paged_chunk_attn(_rows(q, Tq, Hq, D, dev, w), cache.packed, block_table.data_ptr(), ts, width,
                                     _vector(kv_lens, torch.int32, B, dev, w), _rows(o, Tq, Hq, D, dev, w),
                                     _vector(cu_q, torch.int32, B + 1, dev, w), B, Tq, Hq, cache.heads, D, scale,
                                     window, sinks, _ptr(workspace), _nbytes(workspace), _launch_stream(dev, stream))
    if status:
        _check(status, w)


# ----------------------------------------------- recurrent layers over a pool ----
def _states(t, dev, where):
    """sv_states of an fp32 tensor [slots, Hv, dv, dk] of the call's device (any
    slot stride, the rest contiguous), and its Hv, dv and dk."""
    if t.dtype is not torch.float32 or t.dim() != 4 or not t.is_cuda or (dev is not None and t.get_device() != dev):
        _bad(where)
    n, Hv, dv, dk = t.shape
    s0, s1, s2, s3 = t.stride()
    # a dimension of one may carry any stride
    if (s3 != 1 and dk > 1) or (s2 != dk and dv > 1) or (s1 != dv * dk and Hv > 1):
        _bad(where)
    return _STATES.pack(t.data_ptr(), s0 if n > 1 else Hv * dv * dk, n), Hv, dv, dk


def _out_rows(t, tokens, heads, D, dev, where):
    """sv_rows of an output of bf16 or fp32, and which."""
    if t.dtype is not torch.float32:
        return _rows(t, tokens, heads, D, dev, where), SV_BF16
    if t.shape != (tokens, heads, D) or not t.is_cuda or (dev is not None and t.get_device() != dev):
        _bad(where)
    ts, hs, ds = t.stride()
    if ds != 1 and D != 1:
        _bad(where)
    return _ROWS.pack(t.data_ptr(), ts if tokens > 1 else 0, hs if heads > 1 else 0), SV_F32


def gdn_step(states, slots, q, k, v, g, beta, o, M: int, tape=None, n_replay=None, commit: bool = False, stream=None):
    """The gated delta rule over M newest rows of each of B sequences: states
    fp32 [slots, Hv, dv, dk], slots int32 [B] (negative: from zeros, not kept),
    q and k bf16 [B*M, Hk, dk], v and o [B*M, Hv, dv] (o bf16 or fp32), g (log
    decay) and beta fp32 [B*M, Hv].  tape: (k, v, g, beta) of the last round,
    the same number of rows for each sequence, of which the first n_replay[b]
    (int32 [B]) go into the state first.  commit: the M rows go into it too.
    M = 0 only commits the tape; q, k, v, g, beta and o may be None then."""
    w = "gdn_step"
    dev = None if _gpus == 1 else _device(states, w)
    B = slots.numel()
    pool, Hv, dv, dk = _states(states, dev, w)
    if (tape is None) != (n_replay is None):
        _bad(w)
    Hk = (tape[0] if M == 0 and tape is not None else k).shape[1] if M or tape is not None else 1
    t = [None] * 4
    tape_M = 0
    if tape is not None:
        tape_M, rest = divmod(tape[0].shape[0], B) if B else (0, 0)
        if rest or len(tape) != 4:
            _bad(w)
        rows = B * tape_M
        t = [_rows(tape[0], rows, Hk, dk, dev, w), _rows(tape[1], rows, Hv, dv, dev, w),
             _gates(tape[2], rows, Hv, dev, w), _gates(tape[3], rows, Hv, dev, w)]
    own, odt = [None] * 6, SV_BF16
    if M:
        rows = B * M
        out, odt = _out_rows(o, rows, Hv, dv, dev, w)
        own = [_rows(q, rows, Hk, dk, dev, w), _rows(k, rows, Hk, dk, dev, w), _rows(v, rows, Hv, dv, dev, w),
               _gates(g, rows, Hv, dev, w), _gates(beta, rows, Hv, dev, w), out]
    status = load().gdn_step(pool, _vector(slots, torch.int32, B, dev, w), *t,
                             None if n_replay is None else _vector(n_replay, torch.int32, B, dev, w), tape_M, *own,
                             odt, B, M, 1 if commit else 0, Hk, Hv, dk, dv, _launch_stream(dev, stream))
    if status:
        _check(status, w)


def _gates(t, rows, Hv, dev, where):
    """Address of gates fp32 [rows, Hv], contiguous."""
    if t.dtype is not torch.float32 or t.shape != (rows, Hv) or not t.is_cuda or not t.is_contiguous() or (
            dev is not None and t.get_device() != dev):
        _bad(where)
    return t.data_ptr()


def gdn_chunk_workspace_bytes(B: int, T: int, Hk: int, Hv: int, dk: int, dv: int) -> int:
    return load().gdn_chunk_workspace_bytes(B, T, Hk, Hv, dk, dv)


def gdn_chunk(states, slots, q, k, v, g, beta, o, cu, workspace=None, stream=None):
    """The gated delta rule over packed chunks of new tokens: sequence b is rows
    cu[b]..cu[b+1] (int32 [B+1]) of q and k bf16 [T, Hk, dk], v and o bf16
    [T, Hv, dv], g (log decay) and beta fp32 [T, Hv]; it starts from, and goes
    back into, place slots[b] (int32 [B]; negative: from zeros, not kept) of
    the states fp32 [slots, Hv, dv, dk]."""
    w = "gdn_chunk"
    T, Hk, dk = q.shape
    dev = None if _gpus == 1 else _device(q, w)
    pool, Hv, dv, dk_ = _states(states, dev, w)
    B = slots.numel()
    if dk_ != dk or (workspace is not None and (not workspace.is_cuda or (
            dev is not None and workspace.get_device() != dev))):
        _bad(w)
    status = load().gdn_chunk(pool, _vector(slots, torch.int32, B, dev, w),
                              _rows(q, T, Hk, dk, dev, w), _rows(k, T, Hk, dk, dev, w), _rows(v, T, Hv, dv, dev, w),
                              _gates(g, T, Hv, dev, w), _gates(beta, T, Hv, dev, w), _rows(o, T, Hv, dv, dev, w),
                              _vector(cu, torch.int32, B + 1, dev, w), B, T, Hk, Hv, dk, dv, _ptr(workspace),
                              _nbytes(workspace), _launch_stream(dev, stream))
    if status:
        _check(status, w)
