"""Python binding of libvlf.so: fused variable-length flash attention for GB300 (sm_103a).

Argument marshalling only.  Every step of the computation runs in the library's CUDA kernels;
PyTorch supplies device memory and the current stream.  There is no CPU fallback: importing
this package raises if the compiled library is missing.

The functions carry the names of the C entry points in ``include/vlf.h``:

* ``vlf_attn_varlen_fwd(q, k, v, cu_seqlens_q, cu_seqlens_kv, max_seqlen_q, ...)`` -> (out, lse)
* ``vlf_attn_varlen_bwd(dout, q, k, v, out, lse, cu_seqlens_q, cu_seqlens_kv, ...)``
  -> (dq, dk, dv)
* ``vlf_attn_varlen_bwd_workspace_size``, ``vlf_check_error``, ``vlf_status_string``,
  ``vlf_sched_kv_band``, ``vlf_sched_q_band``, ``vlf_version``;
* next to them, for decoding on a bounded cache, ``vlf_rope`` (rotary positions with several axes),
  ``vlf_attn_varlen_fwd_prefix`` (attention behind a prefix that the batch shares),
  ``vlf_attn_key_weights`` (the attention weight each key received) and ``vlf_cache_evict`` (the
  cache cut down to a budget by it);
* for serving from a cache of pages in 8 bits, ``vlf_norm_rope`` / ``vlf_norm_rope_bwd`` (the norm of
  each head with its rotary positions, and its gradients), ``vlf_pages_write`` (new tokens into their
  pages), ``vlf_attn_varlen_fwd_pages`` (attention over them), ``vlf_pages_fork`` and
  ``vlf_pages_compact`` (the sequences' page tables: going on, forking, ending, moving together) and
  ``vlf_pages_copy`` (the copies that those ask for).

The operation is the varlen attention of the mtlattn 0.3.0 page (section "Use"): packed
q/k/v [tokens, heads, head_dim] with int32 cu_seqlens, end-aligned causal, sliding window,
GQA/MQA, additive fp32 bias [total_q, H or 1, max_kv] (held constant in the backward; a bias
that requires grad is refused).
"""
from __future__ import annotations

import ctypes
import os
import warnings

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libvlf.so")

VLF_F16, VLF_BF16, VLF_F32 = 0, 1, 2
VLF_OK = 0
VLF_ERR_INVALID, VLF_ERR_UNSUPPORTED, VLF_ERR_ALIGN, VLF_ERR_LAUNCH = -1, -2, -3, -4
VLF_ERR_TIMEOUT, VLF_ERR_BAD_SEQLENS, VLF_ERR_WORKSPACE, VLF_ERR_BAD_PAGES = -5, -6, -7, -8
VLF_FLAG_NO_SKIP = 1
VLF_FLAG_FORCE_SIMT = 2
VLF_FLAG_NO_PACK = 4
VLF_FLAG_TEST_TIMEOUT = 8  # testing: the forward's pipeline waits run out (VLF_ERR_TIMEOUT)

_DTYPE = {torch.float16: VLF_F16, torch.bfloat16: VLF_BF16, torch.float32: VLF_F32}

EXPORTS = ["vlf_attn_varlen_fwd", "vlf_attn_varlen_fwd_ex", "vlf_attn_varlen_bwd",
           "vlf_attn_varlen_bwd_ex", "vlf_attn_varlen_bwd_workspace_size", "vlf_check_error",
           "vlf_status_string", "vlf_sched_kv_band", "vlf_sched_q_band", "vlf_version",
           "vlf_launch_count", "vlf_fwd_path", "vlf_bwd_path", "vlf_attn_varlen_bwd_noalloc",
           "vlf_noalloc_scratch_bytes", "vlf_attn_varlen_fwd_split", "vlf_fwd_num_splits",
           "vlf_attn_varlen_fwd_split_workspace_size", "vlf_attn_varlen_fwd_latent",
           "vlf_attn_varlen_bwd_latent", "vlf_attn_varlen_bwd_latent_workspace_size",
           "vlf_bias_bands", "vlf_bias_bands_size", "vlf_rope", "vlf_attn_varlen_fwd_prefix",
           "vlf_attn_varlen_fwd_prefix_workspace_size", "vlf_attn_key_weights",
           "vlf_attn_key_weights_workspace_size", "vlf_cache_evict", "vlf_norm_rope", "vlf_norm_rope_bwd",
           "vlf_norm_rope_bwd_workspace_size", "vlf_pages_write", "vlf_attn_varlen_fwd_pages",
           "vlf_attn_varlen_fwd_pages_workspace_size", "vlf_pages_copy", "vlf_pages_fork",
           "vlf_pages_fork_workspace_size", "vlf_pages_compact", "vlf_pages_compact_workspace_size"]
VLF_BWD_STAGES = 3
BWD_STAGE_NAMES = ["rowdot", "dkdv", "dq"]


class VlfError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"vlf status {status}: {vlf_status_string(status)}{': ' + what if what else ''}")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python -c 'import __graft_entry__ as g; "
                          "g.build()'` (needs nvcc for sm_103a)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, F, Z, U = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_uint
    fwd = [P, P, P, P, P, I, I, I, I, I, I, I, I, I, I, F, I, I, P, I, P, P, P]
    lib.vlf_attn_varlen_fwd.argtypes = fwd
    lib.vlf_attn_varlen_fwd_ex.argtypes = fwd + [U, P]
    bwd = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, I, F, I, I, P, I, P, P, P, P, Z, P]
    lib.vlf_attn_varlen_bwd.argtypes = bwd
    lib.vlf_attn_varlen_bwd_ex.argtypes = bwd + [U, P, I, P]
    for name in ("vlf_attn_varlen_fwd", "vlf_attn_varlen_fwd_ex", "vlf_attn_varlen_bwd",
                 "vlf_attn_varlen_bwd_ex"):
        getattr(lib, name).restype = I
    lib.vlf_attn_varlen_bwd_workspace_size.argtypes = [I, I, I, I, I, I, I]
    lib.vlf_attn_varlen_bwd_workspace_size.restype = Z
    lib.vlf_check_error.argtypes = [P]
    lib.vlf_check_error.restype = I
    lib.vlf_status_string.argtypes = [I]
    lib.vlf_status_string.restype = ctypes.c_char_p
    IP = ctypes.POINTER(ctypes.c_int)
    lib.vlf_sched_kv_band.argtypes = [I, I, I, I, I, I, IP, IP]
    lib.vlf_sched_kv_band.restype = I
    lib.vlf_sched_q_band.argtypes = [I, I, I, I, I, I, IP, IP]
    lib.vlf_sched_q_band.restype = I
    lib.vlf_version.argtypes = []
    lib.vlf_version.restype = I
    lib.vlf_attn_varlen_bwd_noalloc.argtypes = bwd[:23] + [P, P, P, P]  # ... bias_heads, dq, dk, dv, stream
    lib.vlf_attn_varlen_bwd_noalloc.restype = I
    lib.vlf_attn_varlen_fwd_split.argtypes = fwd[:22] + [I, P, Z, P, U, P]  # ..., out, lse, splits, ws, bytes, stream, flags, bands
    lib.vlf_attn_varlen_fwd_split.restype = I
    lib.vlf_fwd_num_splits.argtypes = [I, I, I, I, I, I, I, I, U, I]
    lib.vlf_fwd_num_splits.restype = I
    lib.vlf_attn_varlen_fwd_split_workspace_size.argtypes = [I, I, I, I]
    lib.vlf_attn_varlen_fwd_split_workspace_size.restype = Z
    lib.vlf_attn_varlen_fwd_latent.argtypes = [P] * 7 + [I] * 12 + [F, I, I, P, I, P, P, P, U]
    lib.vlf_attn_varlen_fwd_latent.restype = I
    lib.vlf_attn_varlen_bwd_latent_workspace_size.argtypes = [I] * 6
    lib.vlf_attn_varlen_bwd_latent_workspace_size.restype = Z
    lib.vlf_attn_varlen_bwd_latent.argtypes = ([P] * 10 + [I] * 12 + [F, I, I, P, I] + [P] * 6 +
                                               [Z, P, U, P, I])
    lib.vlf_attn_varlen_bwd_latent.restype = I
    lib.vlf_bias_bands_size.argtypes = [I, I]
    lib.vlf_bias_bands_size.restype = Z
    lib.vlf_bias_bands.argtypes = [P, I, P, P, I, I, I, P, Z, P]
    lib.vlf_bias_bands.restype = I
    L = ctypes.c_int64
    lib.vlf_rope.argtypes = [P, L, P, L, P, I, P, P, I, I, I, I, I, I, I, I, P, L, P, L, P]
    lib.vlf_rope.restype = I
    lib.vlf_attn_varlen_fwd_prefix.argtypes = ([P, P, P, I, P, P, P, P] + [I] * 10 + [F, I, I] +
                                               [P, P, P, Z, P, U])
    lib.vlf_attn_varlen_fwd_prefix.restype = I
    lib.vlf_attn_varlen_fwd_prefix_workspace_size.argtypes = [I] * 10 + [U, I]
    lib.vlf_attn_varlen_fwd_prefix_workspace_size.restype = Z
    lib.vlf_attn_key_weights.argtypes = ([P] * 5 + [I] * 9 + [F, I, I, P, P, P, Z, P, U])
    lib.vlf_attn_key_weights.restype = I
    lib.vlf_attn_key_weights_workspace_size.argtypes = [I] * 8 + [U, I]
    lib.vlf_attn_key_weights_workspace_size.restype = Z
    lib.vlf_cache_evict.argtypes = [P] * 4 + [I] * 11 + [P] * 6
    lib.vlf_cache_evict.restype = I
    where = [P, I, P, P]  # positions, axes, sections, inv_freq
    lib.vlf_norm_rope.argtypes = [P, L, P, L, P, P, I, F] + where + [I] * 7 + [P, L, P, L, P]
    lib.vlf_norm_rope.restype = I
    lib.vlf_norm_rope_bwd.argtypes = ([P, L] * 4 + [P, P, I, F] + where + [I] * 7 + [P, L, P, L] +
                                      [P, P, P, Z, P])
    lib.vlf_norm_rope_bwd.restype = I
    lib.vlf_norm_rope_bwd_workspace_size.argtypes = [I]
    lib.vlf_norm_rope_bwd_workspace_size.restype = Z
    lib.vlf_pages_write.argtypes = [P, L, P, L] + [P] * 7 + [I] * 9 + [P]
    lib.vlf_pages_write.restype = I
    lib.vlf_attn_varlen_fwd_pages.argtypes = [P] * 8 + [I] * 11 + [F, I, I, P, P, P, Z, P, U]
    lib.vlf_attn_varlen_fwd_pages.restype = I
    lib.vlf_attn_varlen_fwd_pages_workspace_size.argtypes = [I] * 8 + [U, I]
    lib.vlf_attn_varlen_fwd_pages_workspace_size.restype = Z
    lib.vlf_pages_copy.argtypes = [P] * 6 + [I] * 6 + [P]
    lib.vlf_pages_copy.restype = I
    lib.vlf_pages_fork.argtypes = [P] * 5 + [I] * 5 + [P] * 7 + [Z, P]
    lib.vlf_pages_fork.restype = I
    lib.vlf_pages_fork_workspace_size.argtypes = [I, I]
    lib.vlf_pages_fork_workspace_size.restype = Z
    lib.vlf_pages_compact.argtypes = [P, P, I, I, I] + [P] * 7 + [Z, P]
    lib.vlf_pages_compact.restype = I
    lib.vlf_pages_compact_workspace_size.argtypes = [I]
    lib.vlf_pages_compact_workspace_size.restype = Z
    lib.vlf_noalloc_scratch_bytes.argtypes = []
    lib.vlf_noalloc_scratch_bytes.restype = Z
    lib.vlf_launch_count.argtypes = []
    lib.vlf_launch_count.restype = ctypes.c_uint64
    for name in ("vlf_fwd_path", "vlf_bwd_path"):
        getattr(lib, name).argtypes = [I, I, I, I, I, I, U]
        getattr(lib, name).restype = I
    return lib


class _NoCalls:
    """In place of the native calls: every call is left to the Python functions."""

    def __getattr__(self, name):
        return lambda *args: None


def _load_calls(lib):
    """The native side of the decoding entry points' calls (csrc/calls.cpp), bound to the library.  It
    saves host time only: where it is not built, or for another torch, the Python functions do all."""
    try:
        from . import _calls
        if _calls.TORCH != str(torch.__version__):
            raise ImportError(f"it was built for torch {_calls.TORCH}")
    except (ImportError, AttributeError) as e:
        warnings.warn(f"variable_length_flash_gb300: the native calls are not used ({e}); run `python -c "
                      "'import __graft_entry__ as g; g.build()'`", stacklevel=3)
        return _NoCalls()
    _calls.bind(*[ctypes.cast(f, ctypes.c_void_p).value for f in (
        lib.vlf_rope, lib.vlf_attn_varlen_fwd_prefix, lib.vlf_attn_varlen_fwd_prefix_workspace_size,
        lib.vlf_attn_key_weights, lib.vlf_attn_key_weights_workspace_size, lib.vlf_cache_evict,
        lib.vlf_norm_rope, lib.vlf_norm_rope_bwd, lib.vlf_norm_rope_bwd_workspace_size, lib.vlf_pages_write,
        lib.vlf_attn_varlen_fwd_pages, lib.vlf_attn_varlen_fwd_pages_workspace_size, lib.vlf_pages_copy,
        lib.vlf_pages_fork, lib.vlf_pages_fork_workspace_size, lib.vlf_pages_compact,
        lib.vlf_pages_compact_workspace_size)])
    return _calls


_lib = _load()
_calls = _load_calls(_lib)
_fwd_ex = _lib.vlf_attn_varlen_fwd_ex  # (looked up once: the attribute lookup costs per call)


def _ptr(t):
    # (the argtypes are c_void_p: ctypes takes the integer address, None is NULL)
    return None if t is None else t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, like=None):
    """The handle of ``stream``, else of the current stream of ``like``'s device.  Asking torch
    for the raw handle avoids building a Stream object (microseconds per call)."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None and like is not None:
        return _raw_stream(like.get_device())
    return torch.cuda.current_stream().cuda_stream


def _check(status: int, what: str = ""):
    if status != VLF_OK:
        raise VlfError(status, what)


def vlf_status_string(status: int) -> str:
    return _lib.vlf_status_string(int(status)).decode()


def vlf_version() -> int:
    return _lib.vlf_version()


def vlf_launch_count() -> int:
    """Kernels launched by the library so far in this process."""
    return int(_lib.vlf_launch_count())


def vlf_fwd_path(h_q, h_kv, d_qk, d_v, dtype, bias_heads=0, flags=0) -> int:
    """1: tensor-core forward, 0: SIMT fp32-FMA forward, negative: refused."""
    dt = _DTYPE[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return _lib.vlf_fwd_path(h_q, h_kv, d_qk, d_v, dt, bias_heads, flags)


def vlf_bwd_path(h_q, h_kv, d_qk, d_v, dtype, bias_heads=0, flags=0) -> int:
    """1: tensor-core backward, 0: SIMT fp32-FMA backward, negative: refused."""
    dt = _DTYPE[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return _lib.vlf_bwd_path(h_q, h_kv, d_qk, d_v, dt, bias_heads, flags)


def vlf_check_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error word."""
    return _lib.vlf_check_error(_stream(stream))


def vlf_sched_kv_band(r0, r1, q_len, kv_len, causal, window):
    lo, hi = ctypes.c_int(), ctypes.c_int()
    _check(_lib.vlf_sched_kv_band(r0, r1, q_len, kv_len, int(causal), int(window),
                                  ctypes.byref(lo), ctypes.byref(hi)), "kv band")
    return lo.value, hi.value


def vlf_sched_q_band(j0, j1, q_len, kv_len, causal, window):
    lo, hi = ctypes.c_int(), ctypes.c_int()
    _check(_lib.vlf_sched_q_band(j0, j1, q_len, kv_len, int(causal), int(window),
                                 ctypes.byref(lo), ctypes.byref(hi)), "q band")
    return lo.value, hi.value


def vlf_attn_varlen_bwd_workspace_size(total_q, total_kv, h_q, h_kv, d_qk, d_v, dtype) -> int:
    dt = _DTYPE[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(_lib.vlf_attn_varlen_bwd_workspace_size(total_q, total_kv, h_q, h_kv, d_qk, d_v, dt))


def vlf_fwd_num_splits(num_seqs, max_seqlen_q, max_seqlen_kv, h_q, h_kv, d_qk, d_v, dtype,
                       flags=0, num_sms=0) -> int:
    """Parts the split-KV forward cuts each CTA's KV band into when left to choose (1: no
    split); ``num_sms`` <= 0 takes the current device's SM count."""
    dt = _DTYPE[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(_lib.vlf_fwd_num_splits(num_seqs, max_seqlen_q, max_seqlen_kv, h_q, h_kv, d_qk, d_v,
                                       dt, flags, num_sms))


def vlf_attn_varlen_fwd_split_workspace_size(total_q, h_q, d_v, num_splits) -> int:
    return int(_lib.vlf_attn_varlen_fwd_split_workspace_size(total_q, h_q, d_v, num_splits))


def _events(evs):
    if evs is None:
        return None, 0
    handles = [e.cuda_event for e in evs]
    if not all(handles):
        raise VlfError(VLF_ERR_INVALID, "stage events must exist (torch creates them at their "
                       "first record())")
    arr = (ctypes.c_void_p * len(evs))(*[ctypes.c_void_p(h) for h in handles])
    _events.keep = arr  # keep alive for the duration of the call
    return ctypes.cast(arr, ctypes.c_void_p), len(evs)


def _max_len(cu):
    return int((cu[1:] - cu[:-1]).max().item()) if cu.numel() > 1 else 0


def _req(t, name, dtype=None):
    if t is None:
        raise VlfError(VLF_ERR_INVALID, f"{name} is None")
    if not t.is_cuda:
        raise VlfError(VLF_ERR_INVALID, f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise VlfError(VLF_ERR_INVALID, f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise VlfError(VLF_ERR_INVALID, f"{name} must be {dtype}, got {t.dtype}")
    return t


def _bias_args(bias, total_q, h_q):
    if bias is None:
        return None, 0
    if bias.requires_grad:
        raise VlfError(VLF_ERR_UNSUPPORTED, "the bias is treated as a constant; a bias that "
                       "requires grad is refused")
    _req(bias, "bias", torch.float32)
    if bias.dim() != 3 or bias.shape[0] != total_q or bias.shape[1] not in (1, h_q):
        raise VlfError(VLF_ERR_INVALID, "bias must be [total_q, 1 or H_q, max_seqlen_kv]")
    return bias, int(bias.shape[1])


def _fwd_checks(q, k, v, cu_seqlens_q, cu_seqlens_kv):
    """The forward's argument checks with a message for each failure (the slow path)."""
    _req(q, "q"), _req(k, "k", q.dtype), _req(v, "v", q.dtype)
    _req(cu_seqlens_q, "cu_seqlens_q", torch.int32), _req(cu_seqlens_kv, "cu_seqlens_kv", torch.int32)
    if q.dtype not in _DTYPE:
        raise VlfError(VLF_ERR_INVALID, f"unsupported dtype {q.dtype}")
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise VlfError(VLF_ERR_INVALID, "q, k, v must be [tokens, heads, head_dim]")


def vlf_bias_bands_size(total_q, bias_heads) -> int:
    return int(_lib.vlf_bias_bands_size(int(total_q), int(bias_heads)))


def vlf_bias_bands(bias, cu_seqlens_q, cu_seqlens_kv, max_seqlen_kv=None, out=None, stream=None):
    """The bias bands of ``bias`` [total_q, 1 or H_q, max_seqlen_kv] (fp32, CUDA): per bias head
    and query row the keys from the first to the last finite value and whether the bias is 0
    throughout them, plus the same per 64-row block of each sequence (include/vlf.h).  Returns
    the uint8 CUDA buffer (``out`` when given) to pass as ``bias_bands`` to the forward and
    backward; it stays valid while the bias is unchanged."""
    _req(bias, "bias", torch.float32)
    _req(cu_seqlens_q, "cu_seqlens_q", torch.int32), _req(cu_seqlens_kv, "cu_seqlens_kv", torch.int32)
    if bias.dim() != 3:
        raise VlfError(VLF_ERR_INVALID, "bias must be [total_q, 1 or H_q, max_seqlen_kv]")
    tq, bh, mk = bias.shape
    if max_seqlen_kv is not None and int(max_seqlen_kv) != mk:
        raise VlfError(VLF_ERR_INVALID, "bias last dim must be max_seqlen_kv")
    need = vlf_bias_bands_size(tq, bh)
    if out is None:
        out = torch.empty(max(need, 16), dtype=torch.uint8, device=bias.device)
    st = _lib.vlf_bias_bands(bias.data_ptr(), bh, cu_seqlens_q.data_ptr(), cu_seqlens_kv.data_ptr(),
                             cu_seqlens_q.numel() - 1, tq, mk, out.data_ptr(), out.numel(),
                             _stream(stream, bias))
    _check(st, "vlf_bias_bands")
    return out


def _bands_arg(bias_bands, bias, cu_seqlens_q, cu_seqlens_kv, stream):
    """The bands pointer for a call: computed here for a bias when not given (None); False
    (or no bias) passes none."""
    if bias is None or bias_bands is False:
        return None
    if bias_bands is None:
        bias_bands = vlf_bias_bands(bias, cu_seqlens_q, cu_seqlens_kv, stream=stream)
    return bias_bands.data_ptr()


_SPLITS = {}  # (shape, device) -> the library's split-KV part count


def vlf_attn_varlen_fwd(q, k, v, cu_seqlens_q, cu_seqlens_kv, max_seqlen_q, max_seqlen_kv=None,
                        scale=None, causal=False, window=0, bias=None, out=None, lse=None,
                        stream=None, flags=0, num_splits=None, workspace=None, bias_bands=None):
    """Forward.  q [Tq,Hq,Dqk], k [Tkv,Hkv,Dqk], v [Tkv,Hkv,Dv] (fp16/bf16/fp32, CUDA,
    contiguous), cu_seqlens int32 [n+1].  Returns out [Tq,Hq,Dv] and lse fp32 [Hq,Tq].
    ``max_seqlen_kv=None`` reads it from cu_seqlens_kv (a host sync); the bias's last dim
    must equal max_seqlen_kv when a bias is given.  ``num_splits``: None lets the library
    decide whether to split each CTA's KV band (small-batch / decode shapes; the parts' fp32
    results go to ``workspace``, allocated here when not given), 1 never splits, k > 1 splits
    into k parts.  ``bias_bands``: for a bias, vlf_bias_bands's result for it (None: computed
    here, one extra pass; False: none, every tile's bias is read)."""
    # the common case's conditions in one pass (each tensor attribute costs ~0.1 us of host
    # time, which small problems pay per call); any failure takes the detailed checks
    dtype = q.dtype
    if not (dtype in _DTYPE and k.dtype is dtype and v.dtype is dtype and q.is_cuda and k.is_cuda
            and v.is_cuda and q.is_contiguous() and k.is_contiguous() and v.is_contiguous()
            and q.dim() == 3 and k.dim() == 3 and v.dim() == 3
            and cu_seqlens_q.dtype is torch.int32 and cu_seqlens_kv.dtype is torch.int32
            and cu_seqlens_q.is_cuda and cu_seqlens_kv.is_cuda
            and cu_seqlens_q.is_contiguous() and cu_seqlens_kv.is_contiguous()):
        _fwd_checks(q, k, v, cu_seqlens_q, cu_seqlens_kv)
    tq, hq, dqk = q.shape
    tk, hkv, dv = v.shape
    if k.shape != (tk, hkv, dqk):
        raise VlfError(VLF_ERR_INVALID, "k shape")
    if max_seqlen_kv is None:
        max_seqlen_kv = int(bias.shape[2]) if bias is not None else _max_len(cu_seqlens_kv)
    if bias is not None:
        if bias.shape[2] != max_seqlen_kv:
            raise VlfError(VLF_ERR_INVALID, "bias last dim must be max_seqlen_kv")
        bias, bh = _bias_args(bias, tq, hq)
        bias_p = bias.data_ptr()
        bands_p = _bands_arg(bias_bands, bias, cu_seqlens_q, cu_seqlens_kv, stream)
    else:
        bias_p, bh, bands_p = None, 0, None
    if out is None:
        out = torch.empty((tq, hq, dv), dtype=dtype, device=q.device)
    elif not (out.dtype is dtype and out.is_cuda and out.is_contiguous()):
        _req(out, "out", dtype)
    if lse is None:
        lse = torch.empty((hq, tq), dtype=torch.float32, device=q.device)
    elif not (lse.dtype is torch.float32 and lse.is_cuda and lse.is_contiguous()):
        _req(lse, "lse", torch.float32)
    nseq = cu_seqlens_q.numel() - 1
    dt = _DTYPE[dtype]
    dev = q.get_device()
    st_h = (stream.cuda_stream if stream is not None else
            _raw_stream(dev) if _raw_stream is not None else _stream(None, q))
    if num_splits is None:
        # the library's part count depends on the shape and the device alone: remembered per
        # (shape, device) so that a repeated call makes one foreign call, not two
        key = (nseq, int(max_seqlen_q), int(max_seqlen_kv), hq, hkv, dqk, dv, dt, int(flags), dev)
        num_splits = _SPLITS.get(key)
        if num_splits is None:
            num_splits = _lib.vlf_fwd_num_splits(nseq, int(max_seqlen_q), int(max_seqlen_kv), hq, hkv,
                                                 dqk, dv, dt, int(flags), 0)
            if len(_SPLITS) < 4096:
                _SPLITS[key] = num_splits
    if num_splits >= 2:
        need = vlf_attn_varlen_fwd_split_workspace_size(tq, hq, dv, int(num_splits))
        if workspace is None:
            workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
        _req(workspace, "workspace")
        st = _lib.vlf_attn_varlen_fwd_split(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_seqlens_q.data_ptr(),
            cu_seqlens_kv.data_ptr(), nseq, tq, tk, int(max_seqlen_q), int(max_seqlen_kv), hq, hkv,
            dqk, dv, dt, float(scale) if scale else 0.0, int(bool(causal)), int(window or 0), bias_p,
            bh, out.data_ptr(), lse.data_ptr(), int(num_splits), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), st_h, int(flags), bands_p)
        if st != VLF_OK:
            _check(st, "vlf_attn_varlen_fwd_split")
        return out, lse
    st = _fwd_ex(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_seqlens_q.data_ptr(), cu_seqlens_kv.data_ptr(),
        nseq, tq, tk, int(max_seqlen_q), int(max_seqlen_kv), hq, hkv, dqk, dv, dt,
        float(scale) if scale else 0.0, 1 if causal else 0, int(window) if window else 0, bias_p,
        bh, out.data_ptr(), lse.data_ptr(), st_h, int(flags), bands_p)
    if st != VLF_OK:
        _check(st, "vlf_attn_varlen_fwd")
    return out, lse


def vlf_attn_varlen_bwd(dout, q, k, v, out, lse, cu_seqlens_q, cu_seqlens_kv, max_seqlen_q,
                        max_seqlen_kv=None, scale=None, causal=False, window=0, bias=None,
                        dq=None, dk=None, dv=None, workspace=None, stream=None, flags=0,
                        stage_events=None, bias_bands=None):
    """Backward: gradients of sum(out * dout) w.r.t. q, k, v (bias constant).
    Returns dq, dk, dv in the input dtype.  ``workspace`` (uint8 CUDA tensor of at least
    vlf_attn_varlen_bwd_workspace_size bytes) is allocated with torch when not given.
    ``stage_events``: optional list of VLF_BWD_STAGES + 1 ``torch.cuda.Event`` (timing) recorded
    before the first and after each backward kernel on the same stream."""
    for t, n in ((dout, "dout"), (q, "q"), (k, "k"), (v, "v"), (out, "out")):
        _req(t, n, q.dtype)
    _req(lse, "lse", torch.float32)
    _req(cu_seqlens_q, "cu_seqlens_q", torch.int32), _req(cu_seqlens_kv, "cu_seqlens_kv", torch.int32)
    tq, hq, dqk = q.shape
    tk, hkv, dvv = v.shape
    if max_seqlen_kv is None:
        max_seqlen_kv = int(bias.shape[2]) if bias is not None else _max_len(cu_seqlens_kv)
    bias, bh = _bias_args(bias, tq, hq)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    need = vlf_attn_varlen_bwd_workspace_size(tq, tk, hq, hkv, dqk, dvv, q.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    st = _lib.vlf_attn_varlen_bwd_ex(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), _ptr(cu_seqlens_q),
        _ptr(cu_seqlens_kv), cu_seqlens_q.numel() - 1, tq, tk, int(max_seqlen_q),
        int(max_seqlen_kv), hq, hkv, dqk, dvv, _DTYPE[q.dtype], float(scale) if scale else 0.0,
        int(bool(causal)), int(window or 0), _ptr(bias), bh, _ptr(dq), _ptr(dk), _ptr(dv),
        _ptr(workspace), workspace.numel(), _stream(stream, q), int(flags), *_events(stage_events),
        _bands_arg(bias_bands, bias, cu_seqlens_q, cu_seqlens_kv, stream))
    _check(st, "vlf_attn_varlen_bwd")
    return dq, dk, dv


def _latent_args(q_nope, q_rope, k_nope, k_rope, v):
    """Shapes of a split-operand latent call: (tq, hq, tk, hkv, rope_heads)."""
    _req(q_nope, "q_nope")
    for t, n in ((q_rope, "q_rope"), (k_nope, "k_nope"), (k_rope, "k_rope"), (v, "v")):
        _req(t, n, q_nope.dtype)
    if any(t.dim() != 3 for t in (q_nope, q_rope, k_nope, k_rope, v)):
        raise VlfError(VLF_ERR_INVALID, "latent operands must be [tokens, heads, width]")
    tq, hq, _ = q_nope.shape
    tk, hkv, _ = k_nope.shape
    if tuple(q_rope.shape[:2]) != (tq, hq) or k_rope.shape[0] != tk or tuple(v.shape[:2]) != (tk, hkv):
        raise VlfError(VLF_ERR_INVALID, "latent operand shapes disagree")
    return tq, hq, tk, hkv, int(k_rope.shape[1])


def vlf_attn_varlen_fwd_latent(q_nope, q_rope, k_nope, k_rope, v, cu_seqlens_q, cu_seqlens_kv,
                               max_seqlen_q, max_seqlen_kv=None, scale=None, causal=False,
                               window=0, bias=None, out=None, lse=None, stream=None, flags=0):
    """Latent attention forward with split operands (q_nope [Tq,H,128], q_rope [Tq,H,64],
    k_nope [Tkv,Hkv,128], k_rope [Tkv,1 or Hkv,64], v [Tkv,Hkv,128]); equals the forward on the
    concatenated operands.  Returns out [Tq,H,128] and lse fp32 [H,Tq]."""
    tq, hq, tk, hkv, rh = _latent_args(q_nope, q_rope, k_nope, k_rope, v)
    _req(cu_seqlens_q, "cu_seqlens_q", torch.int32), _req(cu_seqlens_kv, "cu_seqlens_kv", torch.int32)
    if max_seqlen_kv is None:
        max_seqlen_kv = int(bias.shape[2]) if bias is not None else _max_len(cu_seqlens_kv)
    bias, bh = _bias_args(bias, tq, hq)
    dv = v.shape[2]
    if out is None:
        out = torch.empty((tq, hq, dv), dtype=q_nope.dtype, device=q_nope.device)
    if lse is None:
        lse = torch.empty((hq, tq), dtype=torch.float32, device=q_nope.device)
    st = _lib.vlf_attn_varlen_fwd_latent(
        _ptr(q_nope), _ptr(q_rope), _ptr(k_nope), _ptr(k_rope), _ptr(v), _ptr(cu_seqlens_q),
        _ptr(cu_seqlens_kv), cu_seqlens_q.numel() - 1, tq, tk, int(max_seqlen_q),
        int(max_seqlen_kv), hq, hkv, rh, q_nope.shape[2], q_rope.shape[2], dv,
        _DTYPE[q_nope.dtype], float(scale) if scale else 0.0, int(bool(causal)), int(window or 0),
        _ptr(bias), bh, _ptr(out), _ptr(lse), _stream(stream, q_nope), int(flags))
    _check(st, "vlf_attn_varlen_fwd_latent")
    return out, lse


def vlf_attn_varlen_bwd_latent_workspace_size(total_q, total_kv, h_q, h_kv, rope_heads, dtype) -> int:
    dt = _DTYPE[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(_lib.vlf_attn_varlen_bwd_latent_workspace_size(total_q, total_kv, h_q, h_kv,
                                                              rope_heads, dt))


def vlf_attn_varlen_bwd_latent(dout, q_nope, q_rope, k_nope, k_rope, v, out, lse, cu_seqlens_q,
                               cu_seqlens_kv, max_seqlen_q, max_seqlen_kv=None, scale=None,
                               causal=False, window=0, bias=None, grads=None, workspace=None,
                               stream=None, flags=0, stage_events=None):
    """Latent attention backward with split operands.  Returns (dq_nope, dq_rope, dk_nope,
    dk_rope, dv); a shared rope key (k_rope with one head) gets the sum of every head's
    gradient.  ``grads``: optional preallocated 5-tuple in that order."""
    tq, hq, tk, hkv, rh = _latent_args(q_nope, q_rope, k_nope, k_rope, v)
    for t, n in ((dout, "dout"), (out, "out")):
        _req(t, n, q_nope.dtype)
    _req(lse, "lse", torch.float32)
    _req(cu_seqlens_q, "cu_seqlens_q", torch.int32), _req(cu_seqlens_kv, "cu_seqlens_kv", torch.int32)
    if max_seqlen_kv is None:
        max_seqlen_kv = int(bias.shape[2]) if bias is not None else _max_len(cu_seqlens_kv)
    bias, bh = _bias_args(bias, tq, hq)
    if grads is None:
        grads = tuple(torch.empty_like(t) for t in (q_nope, q_rope, k_nope, k_rope, v))
    need = vlf_attn_varlen_bwd_latent_workspace_size(tq, tk, hq, hkv, rh, q_nope.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q_nope.device)
    st = _lib.vlf_attn_varlen_bwd_latent(
        _ptr(q_nope), _ptr(q_rope), _ptr(k_nope), _ptr(k_rope), _ptr(v), _ptr(out), _ptr(lse),
        _ptr(dout), _ptr(cu_seqlens_q), _ptr(cu_seqlens_kv), cu_seqlens_q.numel() - 1, tq, tk,
        int(max_seqlen_q), int(max_seqlen_kv), hq, hkv, rh, q_nope.shape[2], q_rope.shape[2],
        v.shape[2], _DTYPE[q_nope.dtype], float(scale) if scale else 0.0, int(bool(causal)),
        int(window or 0), _ptr(bias), bh, *[_ptr(g) for g in grads], _ptr(workspace),
        workspace.numel(), _stream(stream, q_nope), int(flags), *_events(stage_events))
    _check(st, "vlf_attn_varlen_bwd_latent")
    return grads


def vlf_noalloc_scratch_bytes() -> int:
    return int(_lib.vlf_noalloc_scratch_bytes())


def vlf_attn_varlen_bwd_noalloc(dout, q, k, v, out, lse, cu_seqlens_q, cu_seqlens_kv,
                                max_seqlen_q, max_seqlen_kv=None, scale=None, causal=False,
                                window=0, bias=None, dq=None, dk=None, dv=None, stream=None):
    """Backward through the entry point that allocates nothing on the device: the library keeps
    the row-dot workspace in a fixed array of its own (vlf_noalloc_scratch_bytes() bytes per
    GPU), for callers that cannot allocate device memory when they call.  Calls that overlap on
    the GPU share that array and race; problems with h_q * total_q above the array's size are
    refused.  The gradient outputs are allocated here with torch only when not passed in."""
    for t, n in ((dout, "dout"), (q, "q"), (k, "k"), (v, "v"), (out, "out")):
        _req(t, n, q.dtype)
    _req(lse, "lse", torch.float32)
    _req(cu_seqlens_q, "cu_seqlens_q", torch.int32), _req(cu_seqlens_kv, "cu_seqlens_kv", torch.int32)
    tq, hq, dqk = q.shape
    tk, hkv, dvv = v.shape
    if max_seqlen_kv is None:
        max_seqlen_kv = int(bias.shape[2]) if bias is not None else _max_len(cu_seqlens_kv)
    bias, bh = _bias_args(bias, tq, hq)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    st = _lib.vlf_attn_varlen_bwd_noalloc(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), _ptr(cu_seqlens_q),
        _ptr(cu_seqlens_kv), cu_seqlens_q.numel() - 1, tq, tk, int(max_seqlen_q),
        int(max_seqlen_kv), hq, hkv, dqk, dvv, _DTYPE[q.dtype], float(scale) if scale else 0.0,
        int(bool(causal)), int(window or 0), _ptr(bias), bh, _ptr(dq), _ptr(dk), _ptr(dv),
        _stream(stream, q))
    _check(st, "vlf_attn_varlen_bwd_noalloc")
    return dq, dk, dv


# ------------------------------------------------------------------ decoding on a bounded cache
# Host time counts in a decode step, whose kernels take microseconds: the common case (plain CUDA
# tensors, outputs allocated here, the current stream) is one native call (csrc/calls.cpp), which
# returns None for everything else and for what it refuses.  What follows it tests its conditions in
# one expression (a tensor attribute costs ~0.1 us), and only where that fails takes the checks that
# say which one it was.
def _same_device(like, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != like.device:
            raise VlfError(VLF_ERR_INVALID, f"{name} is on {t.device}, not on {like.device}")


def _another(stream, like):
    """Whether the caller's stream is another than the current one of like's device."""
    if stream is None or not like.is_cuda:
        return False
    if stream.device != like.device:
        raise VlfError(VLF_ERR_INVALID, f"stream is on {stream.device}, the tensors on {like.device}")
    return stream.cuda_stream != _stream(None, like)


def _under(stream, given, call):
    """call() with the caller's stream as the current one: what it allocates or reads on the host is in
    that stream's order.  (A block allocated on the current stream may still be read or written by
    what is queued there, which the caller's stream does not wait for.)  The outputs that the caller
    did not give are told of the stream they are returned to, so that they outlive its work on them."""
    here = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        got = call()
    for t in got if isinstance(got, tuple) else (got,):
        if t is not None and t.numel() and not any(t is g for g in given):
            t.record_stream(here)
    return got


def _elsewhere(t):
    """Whether t is on another device than the current one, where a kernel would be launched whatever
    its stream and pointers say."""
    return t.is_cuda and t.get_device() != torch.cuda.current_device()


def _given(t, name, shape, dtype):
    """A caller's output tensor."""
    _req(t, name, dtype)
    if tuple(t.shape) != tuple(shape):
        raise VlfError(VLF_ERR_INVALID, f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _c_int(x, name):
    """x as the C int an entry point takes (ctypes would cut off what does not fit)."""
    x = int(x)
    if not -0x80000000 <= x <= 0x7fffffff:
        raise VlfError(VLF_ERR_INVALID, f"{name} = {x} is out of range")
    return x


def _fits(*sizes):
    """Refuses shapes that no C int holds (ctypes would cut them off)."""
    if max(sizes) > 0x7fffffff:
        raise VlfError(VLF_ERR_UNSUPPORTED, f"a size of {max(sizes)} is out of range")


_WORKSPACES = {}  # (entry point, shape, device) -> bytes of workspace


def _workspace_size(fn, key):
    """fn(*key[1:-1], 0 SMs given), remembered: it depends on the shape and the device alone."""
    need = _WORKSPACES.get(key)
    if need is None:
        need = int(fn(*key[1:-1], 0))
        if len(_WORKSPACES) < 4096:
            _WORKSPACES[key] = need
    return need


def _rope_rows(t, name, dtype, total=None):
    """Checks a rope operand [tokens, heads, d] (tokens may be strided, heads and columns are
    dense) and returns its token stride."""
    if t is None or not t.is_cuda:
        raise VlfError(VLF_ERR_INVALID, f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise VlfError(VLF_ERR_INVALID, f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3 or (total is not None and t.shape[0] != total):
        raise VlfError(VLF_ERR_INVALID, f"{name} must be [tokens, heads, head_dim]")
    n, h, d = t.shape
    s0, s1, s2 = t.stride()
    if (d > 1 and s2 != 1) or (h > 1 and s1 != d):
        raise VlfError(VLF_ERR_INVALID, f"{name}: the heads and columns of a token must be dense")
    return s0 if n > 1 else h * d


_SECTIONS = {}  # section counts -> the C array of them


def _sections(sections):
    key = tuple(map(int, sections))
    arr = _SECTIONS.get(key)
    if arr is None:
        arr = (ctypes.c_int * len(key))(*key)
        if len(_SECTIONS) < 256:
            _SECTIONS[key] = arr
    return arr


def vlf_rope(q, k, positions, inv_freq, sections=None, interleaved=False, inverse=False, q_out=None,
             k_out=None, stream=None):
    """Rotary positions of q [T,Hq,D] and k [T,Hk,D] (k may be None) with one or several position
    axes.  ``positions`` int32 [T] or [axes, T]; ``inv_freq`` fp32 [rot / 2], the radians a pair
    turns per unit of its position; ``sections``: how many consecutive pairs each axis turns (None:
    one axis).  Pair c is columns (c, c + rot / 2), or (2 c, 2 c + 1) when ``interleaved``; columns
    from rot on pass through.  ``inverse`` turns back, which is also the gradient.  q and k may be
    slices of a packed projection (their tokens may be strided); ``q_out`` / ``k_out`` may be q / k
    themselves.  Returns (q_out, k_out)."""
    if q_out is None and k_out is None and stream is None:
        done = _calls.rope(q, k, positions, inv_freq, sections, interleaved, inverse)
        if done is not None:
            return done
    if _elsewhere(q):
        with torch.cuda.device(q.device):
            return vlf_rope(q, k, positions, inv_freq, sections, interleaved, inverse, q_out, k_out,
                            stream)
    if _another(stream, q):
        return _under(stream, (q_out, k_out), lambda: vlf_rope(
            q, k, positions, inv_freq, sections, interleaved, inverse, q_out, k_out))
    dtype = q.dtype
    dt = _DTYPE.get(dtype)
    if dt is None:
        raise VlfError(VLF_ERR_INVALID, f"unsupported dtype {dtype}")
    shape, stride, dev = q.shape, q.stride(), q.get_device()
    if dev >= 0 and len(shape) == 3 and stride[2] == 1 and stride[1] == shape[2] and shape[0] > 1:
        sq = stride[0]
    else:
        sq = _rope_rows(q, "q", dtype)
    total, hq, d = shape
    hk, sk, sko, k_p, ko_p = 0, 0, 0, None, None
    if k is not None:
        shape, stride = k.shape, k.stride()
        if (k.get_device() == dev and k.dtype is dtype and len(shape) == 3 and stride[2] == 1
                and stride[1] == d and shape[0] == total and shape[2] == d and total > 1):
            sk = stride[0]
        else:
            sk = _rope_rows(k, "k", dtype, total)
            if shape[2] != d:
                raise VlfError(VLF_ERR_INVALID, "q and k must have the same head_dim")
        hk = shape[1]
        k_p = k.data_ptr()
    shape = positions.shape
    if not (positions.dtype is torch.int32 and inv_freq.dtype is torch.float32
            and positions.get_device() == dev and inv_freq.get_device() == dev
            and positions.is_contiguous() and inv_freq.is_contiguous() and inv_freq.dim() == 1
            and 1 <= len(shape) <= 2 and shape[-1] == total):
        _req(positions, "positions", torch.int32), _req(inv_freq, "inv_freq", torch.float32)
        _same_device(q, positions=positions, inv_freq=inv_freq)
        raise VlfError(VLF_ERR_INVALID, "positions must be [tokens] or [axes, tokens], inv_freq [rot / 2]")
    _fits(total, hq, hk, d, 2 * inv_freq.shape[0])
    # (slices of them start anywhere; the library takes 16-byte aligned pointers)
    if positions.data_ptr() % 16:
        positions = positions.clone()
    if inv_freq.data_ptr() % 16:
        inv_freq = inv_freq.clone()
    axes = 1 if len(shape) == 1 else shape[0]
    if sections is None:
        if axes != 1:
            raise VlfError(VLF_ERR_INVALID, "several position axes need sections")
        sec = None
    else:
        if len(sections) != axes:
            raise VlfError(VLF_ERR_INVALID, f"{len(sections)} sections for {axes} position axes")
        sec = _sections(sections)
    if q_out is None:
        q_out = torch.empty((total, hq, d), dtype=dtype, device=q.device)
        sqo = hq * d
    else:
        sqo = _rope_rows(q_out, "q_out", dtype, total)
        if q_out.shape != q.shape:
            raise VlfError(VLF_ERR_INVALID, "q_out must have q's shape")
        _same_device(q, q_out=q_out)
    if k is not None:
        if k_out is None:
            k_out = torch.empty((total, hk, d), dtype=dtype, device=q.device)
            sko = hk * d
        else:
            sko = _rope_rows(k_out, "k_out", dtype, total)
            if k_out.shape != k.shape:
                raise VlfError(VLF_ERR_INVALID, "k_out must have k's shape")
        if k.get_device() != dev or k_out.get_device() != dev:
            _same_device(q, k=k, k_out=k_out)
        ko_p = k_out.data_ptr()
    elif k_out is not None:
        raise VlfError(VLF_ERR_INVALID, "k_out without k")
    st = _lib.vlf_rope(q.data_ptr(), sq, k_p, sk, positions.data_ptr(), axes, sec, inv_freq.data_ptr(),
                       total, hq, hk, d, 2 * inv_freq.shape[0], dt, 1 if interleaved else 0,
                       1 if inverse else 0, q_out.data_ptr(), sqo, ko_p, sko, _stream(stream, q))
    if st != VLF_OK:
        _check(st, "vlf_rope")
    return q_out, k_out


def vlf_attn_varlen_fwd_prefix_workspace_size(num_seqs, total_q, max_seqlen_q, max_seqlen_kv,
                                              prefix_len, h_q, h_kv, d_qk, d_v, dtype, flags=0,
                                              num_sms=0) -> int:
    dt = _DTYPE[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(_lib.vlf_attn_varlen_fwd_prefix_workspace_size(
        num_seqs, total_q, max_seqlen_q, max_seqlen_kv, prefix_len, h_q, h_kv, d_qk, d_v, dt, flags,
        num_sms))


def vlf_attn_varlen_fwd_prefix(q, k_prefix, v_prefix, k, v, cu_seqlens_q, cu_seqlens_kv,
                               max_seqlen_q, max_seqlen_kv=None, scale=None, causal=False, window=0,
                               out=None, lse=None, workspace=None, stream=None, flags=0):
    """Attention of a batch whose sequences share their first keys: every sequence attends over
    ``k_prefix`` / ``v_prefix`` [P, Hkv, D] and then its own keys.  Equals vlf_attn_varlen_fwd on
    the concatenated keys, with the prefix read once.  Returns out [Tq, Hq, Dv] and lse fp32
    [Hq, Tq].  ``workspace``: at least vlf_attn_varlen_fwd_prefix_workspace_size bytes, allocated
    here when not given."""
    if out is None and lse is None and workspace is None and stream is None:
        done = _calls.prefix(q, k_prefix, v_prefix, k, v, cu_seqlens_q, cu_seqlens_kv, max_seqlen_q,
                             max_seqlen_kv, scale, causal, window, flags)
        if done is not None:
            return done
    if _elsewhere(q):
        with torch.cuda.device(q.device):
            return vlf_attn_varlen_fwd_prefix(q, k_prefix, v_prefix, k, v, cu_seqlens_q,
                                              cu_seqlens_kv, max_seqlen_q, max_seqlen_kv, scale,
                                              causal, window, out, lse, workspace, stream, flags)
    if _another(stream, q):
        return _under(stream, (out, lse), lambda: vlf_attn_varlen_fwd_prefix(
            q, k_prefix, v_prefix, k, v, cu_seqlens_q, cu_seqlens_kv, max_seqlen_q, max_seqlen_kv, scale,
            causal, window, out, lse, workspace, flags=flags))
    dtype, dev = q.dtype, q.get_device()
    i32 = torch.int32
    if not (dtype in _DTYPE and dev >= 0 and q.is_contiguous()
            and k.dtype is dtype and k.get_device() == dev and k.is_contiguous()
            and v.dtype is dtype and v.get_device() == dev and v.is_contiguous()
            and k_prefix.dtype is dtype and k_prefix.get_device() == dev and k_prefix.is_contiguous()
            and v_prefix.dtype is dtype and v_prefix.get_device() == dev and v_prefix.is_contiguous()
            and cu_seqlens_q.dtype is i32 and cu_seqlens_q.get_device() == dev and cu_seqlens_q.is_contiguous()
            and cu_seqlens_kv.dtype is i32 and cu_seqlens_kv.get_device() == dev and cu_seqlens_kv.is_contiguous()
            and q.dim() == 3 and k.dim() == 3 and v.dim() == 3):
        _fwd_checks(q, k, v, cu_seqlens_q, cu_seqlens_kv)
        _req(k_prefix, "k_prefix", dtype), _req(v_prefix, "v_prefix", dtype)
        _same_device(q, k_prefix=k_prefix, v_prefix=v_prefix, k=k, v=v, cu_seqlens_q=cu_seqlens_q,
                     cu_seqlens_kv=cu_seqlens_kv)
    tq, hq, dqk = q.shape
    tk, hkv, dv = v.shape
    if k.shape != (tk, hkv, dqk):
        raise VlfError(VLF_ERR_INVALID, "k shape")
    n = k_prefix.shape[0]
    if k_prefix.shape != (n, hkv, dqk) or v_prefix.shape != (n, hkv, dv):
        raise VlfError(VLF_ERR_INVALID, "k_prefix / v_prefix must be [prefix_len, H_kv, D]")
    nseq = cu_seqlens_q.numel() - 1
    if nseq != cu_seqlens_kv.numel() - 1 or nseq < 0:
        raise VlfError(VLF_ERR_INVALID, "cu_seqlens_q and cu_seqlens_kv must have num_seqs + 1 entries")
    _fits(tq, tk, n, nseq, hq, hkv, dqk, dv)
    if max_seqlen_kv is None:
        max_seqlen_kv = _max_len(cu_seqlens_kv)
    if out is None:
        out = torch.empty((tq, hq, dv), dtype=dtype, device=q.device)
    else:
        _given(out, "out", (tq, hq, dv), dtype), _same_device(q, out=out)
    if lse is None:
        lse = torch.empty((hq, tq), dtype=torch.float32, device=q.device)
    else:
        _given(lse, "lse", (hq, tq), torch.float32), _same_device(q, lse=lse)
    mq, mk = _c_int(max_seqlen_q, "max_seqlen_q"), _c_int(max_seqlen_kv, "max_seqlen_kv")
    window = _c_int(window or 0, "window")
    dt, flags = _DTYPE[dtype], int(flags)
    need = _workspace_size(_lib.vlf_attn_varlen_fwd_prefix_workspace_size,
                           ("prefix", nseq, tq, mq, mk, n, hq, hkv, dqk, dv, dt, flags, dev))
    ws_p, ws_n = None, 0
    if workspace is not None:
        _req(workspace, "workspace"), _same_device(q, workspace=workspace)
        ws_p, ws_n = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    elif need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        ws_p, ws_n = workspace.data_ptr(), need
    st = _lib.vlf_attn_varlen_fwd_prefix(
        q.data_ptr(), k_prefix.data_ptr(), v_prefix.data_ptr(), n, k.data_ptr(), v.data_ptr(),
        cu_seqlens_q.data_ptr(), cu_seqlens_kv.data_ptr(), nseq, tq, tk, mq, mk, hq, hkv, dqk, dv, dt,
        float(scale) if scale else 0.0, 1 if causal else 0, window,
        out.data_ptr(), lse.data_ptr(), ws_p, ws_n, _stream(stream, q), flags)
    if st != VLF_OK:
        _check(st, "vlf_attn_varlen_fwd_prefix")
    return out, lse


def vlf_attn_key_weights_workspace_size(num_seqs, total_kv, max_seqlen_q, max_seqlen_kv, h_q, h_kv, d,
                                        dtype, flags=0, num_sms=0) -> int:
    dt = _DTYPE[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(_lib.vlf_attn_key_weights_workspace_size(num_seqs, total_kv, max_seqlen_q,
                                                        max_seqlen_kv, h_q, h_kv, d, dt, flags, num_sms))


def vlf_attn_key_weights(q, k, lse, cu_seqlens_q, cu_seqlens_kv, max_seqlen_q, max_seqlen_kv=None,
                         scale=None, causal=False, window=0, prev=None, weights=None, workspace=None,
                         stream=None, flags=0):
    """The attention weight each key received, fp32 [Hkv, Tkv]: the sum over the rows that see it and
    the heads of its group of exp(logit - lse), plus ``prev`` (fp32 [Hkv, Tkv], or None).  ``lse``
    [Hq, Tq] comes from the forward with the same scale, causal and window.  ``weights`` (the
    output) may be ``prev``."""
    if weights is None and workspace is None and stream is None:
        done = _calls.weights(q, k, lse, cu_seqlens_q, cu_seqlens_kv, max_seqlen_q, max_seqlen_kv,
                              scale, causal, window, prev, flags)
        if done is not None:
            return done
    if _elsewhere(q):
        with torch.cuda.device(q.device):
            return vlf_attn_key_weights(q, k, lse, cu_seqlens_q, cu_seqlens_kv, max_seqlen_q,
                                        max_seqlen_kv, scale, causal, window, prev, weights,
                                        workspace, stream, flags)
    if _another(stream, q):
        return _under(stream, (weights,), lambda: vlf_attn_key_weights(
            q, k, lse, cu_seqlens_q, cu_seqlens_kv, max_seqlen_q, max_seqlen_kv, scale, causal, window,
            prev, weights, workspace, flags=flags))
    dtype, dev = q.dtype, q.get_device()
    i32, f32 = torch.int32, torch.float32
    if not (dtype in _DTYPE and dev >= 0 and q.is_contiguous()
            and k.dtype is dtype and k.get_device() == dev and k.is_contiguous()
            and lse.dtype is f32 and lse.get_device() == dev and lse.is_contiguous()
            and cu_seqlens_q.dtype is i32 and cu_seqlens_q.get_device() == dev and cu_seqlens_q.is_contiguous()
            and cu_seqlens_kv.dtype is i32 and cu_seqlens_kv.get_device() == dev and cu_seqlens_kv.is_contiguous()
            and q.dim() == 3 and k.dim() == 3):
        _fwd_checks(q, k, k, cu_seqlens_q, cu_seqlens_kv)
        _req(lse, "lse", f32)
        _same_device(q, k=k, lse=lse, cu_seqlens_q=cu_seqlens_q, cu_seqlens_kv=cu_seqlens_kv)
    tq, hq, d = q.shape
    tk, hkv, _ = k.shape
    if k.shape[2] != d or lse.shape != (hq, tq):
        raise VlfError(VLF_ERR_INVALID, "k must be [Tkv, Hkv, D] and lse [Hq, Tq]")
    nseq = cu_seqlens_q.numel() - 1
    if nseq != cu_seqlens_kv.numel() - 1 or nseq < 0:
        raise VlfError(VLF_ERR_INVALID, "cu_seqlens_q and cu_seqlens_kv must have num_seqs + 1 entries")
    _fits(tq, tk, nseq, hq, hkv, d)
    if max_seqlen_kv is None:
        max_seqlen_kv = _max_len(cu_seqlens_kv)
    prev_p = None
    if prev is not None:
        _given(prev, "prev", (hkv, tk), f32)
        if prev.get_device() != dev:
            _same_device(q, prev=prev)
        prev_p = prev.data_ptr()
    if weights is None:
        weights = torch.empty((hkv, tk), dtype=f32, device=q.device)
    else:
        _given(weights, "weights", (hkv, tk), f32), _same_device(q, weights=weights)
    mq, mk = _c_int(max_seqlen_q, "max_seqlen_q"), _c_int(max_seqlen_kv, "max_seqlen_kv")
    window = _c_int(window or 0, "window")
    dt, flags = _DTYPE[dtype], int(flags)
    need = _workspace_size(_lib.vlf_attn_key_weights_workspace_size,
                           ("weights", nseq, tk, mq, mk, hq, hkv, d, dt, flags, dev))
    ws_p, ws_n = None, 0
    if workspace is not None:
        _req(workspace, "workspace"), _same_device(q, workspace=workspace)
        ws_p, ws_n = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    elif need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        ws_p, ws_n = workspace.data_ptr(), need
    st = _lib.vlf_attn_key_weights(
        q.data_ptr(), k.data_ptr(), lse.data_ptr(), cu_seqlens_q.data_ptr(), cu_seqlens_kv.data_ptr(),
        nseq, tq, tk, mq, mk, hq, hkv, d, dt, float(scale) if scale else 0.0, 1 if causal else 0,
        window, prev_p, weights.data_ptr(), ws_p, ws_n, _stream(stream, q), flags)
    if st != VLF_OK:
        _check(st, "vlf_attn_key_weights")
    return weights


def vlf_cache_evict(k, v, weights, cu_seqlens_kv, budget, sink=0, recent=0, max_seqlen_kv=None,
                    total_out=None, k_out=None, v_out=None, weights_out=None, index_out=None,
                    cu_out=None, stream=None):
    """Cuts each sequence's cache to at most ``budget`` keys: the first ``sink``, the last ``recent``
    and, between them, the ones with the largest weight (per kv head; ties keep the lower index).
    k [Tkv,Hkv,Dk], v [Tkv,Hkv,Dv], weights fp32 [Hkv,Tkv].  Returns the compacted (k, v, weights),
    index int32 [Hkv, total_out] (the sequence-local key each row came from) and cu int32 [n + 1].
    ``total_out``: rows of the outputs, the sum of min(length, budget) where the caller knows the
    lengths (None: min(Tkv, n * budget), whose last rows may stay unwritten)."""
    if stream is None and k_out is None and v_out is None and weights_out is None and index_out is None \
            and cu_out is None:
        done = _calls.evict(k, v, weights, cu_seqlens_kv, budget, sink, recent, max_seqlen_kv, total_out)
        if done is not None:
            return done
    if _elsewhere(k):
        with torch.cuda.device(k.device):
            return vlf_cache_evict(k, v, weights, cu_seqlens_kv, budget, sink, recent,
                                   max_seqlen_kv, total_out, k_out, v_out, weights_out, index_out,
                                   cu_out, stream)
    if _another(stream, k):
        return _under(stream, (k_out, v_out, weights_out, index_out, cu_out), lambda: vlf_cache_evict(
            k, v, weights, cu_seqlens_kv, budget, sink, recent, max_seqlen_kv, total_out, k_out, v_out,
            weights_out, index_out, cu_out))
    dtype, dev = k.dtype, k.get_device()
    if not (dtype in _DTYPE and dev >= 0 and k.is_contiguous() and v.dtype is dtype
            and v.get_device() == dev and v.is_contiguous() and weights.dtype is torch.float32
            and weights.get_device() == dev and weights.is_contiguous()
            and cu_seqlens_kv.dtype is torch.int32 and cu_seqlens_kv.get_device() == dev
            and cu_seqlens_kv.is_contiguous()):
        _req(k, "k"), _req(v, "v", dtype), _req(weights, "weights", torch.float32)
        _req(cu_seqlens_kv, "cu_seqlens_kv", torch.int32)
        _same_device(k, v=v, weights=weights, cu_seqlens_kv=cu_seqlens_kv)
        raise VlfError(VLF_ERR_INVALID, f"unsupported dtype {dtype}")
    ks, vs = k.shape, v.shape
    if len(ks) != 3 or len(vs) != 3 or ks[:2] != vs[:2] or cu_seqlens_kv.numel() < 1:
        raise VlfError(VLF_ERR_INVALID, "k, v must be [tokens, heads, head_dim]")
    tk, h, dk = ks
    dv = vs[2]
    if weights.shape != (h, tk):
        raise VlfError(VLF_ERR_INVALID, "weights must be [H_kv, total_kv]")
    _fits(tk, h, dk, dv, cu_seqlens_kv.numel())
    if max_seqlen_kv is None:
        max_seqlen_kv = _max_len(cu_seqlens_kv)
    n, budget, sink, recent = cu_seqlens_kv.numel() - 1, int(budget), int(sink), int(recent)
    if sink < 0 or recent < 0 or sink + recent > budget:
        raise VlfError(VLF_ERR_INVALID, "sink and recent must be at least 0, their sum at most budget")
    budget = min(budget, 0x7fffffff)  # (more than any sequence has)
    sink, recent = _c_int(sink, "sink"), _c_int(recent, "recent")
    total_out = min(tk, n * budget) if total_out is None else _c_int(total_out, "total_out")
    given = (k_out, v_out, weights_out, index_out, cu_out)
    empty, device = torch.empty, k.device
    if k_out is None:
        k_out = empty((total_out, h, dk), dtype=dtype, device=device)
    if v_out is None:
        v_out = empty((total_out, h, dv), dtype=dtype, device=device)
    if weights_out is None:
        weights_out = empty((h, total_out), dtype=torch.float32, device=device)
    if index_out is None:
        index_out = empty((h, total_out), dtype=torch.int32, device=device)
    if cu_out is None:
        cu_out = empty((n + 1,), dtype=torch.int32, device=device)
    outs = (k_out, v_out, weights_out, index_out, cu_out)
    if not all(t is None for t in given):
        for t, name, like in zip(given, ("k_out", "v_out", "weights_out", "index_out", "cu_out"),
                                 ((total_out, h, dk, dtype), (total_out, h, dv, dtype),
                                  (h, total_out, torch.float32), (h, total_out, torch.int32),
                                  (n + 1, torch.int32))):
            if t is not None:
                _given(t, name, like[:-1], like[-1]), _same_device(k, **{name: t})
    st = _lib.vlf_cache_evict(
        k.data_ptr(), v.data_ptr(), weights.data_ptr(), cu_seqlens_kv.data_ptr(), n, tk,
        _c_int(max_seqlen_kv, "max_seqlen_kv"), h, dk, dv, _DTYPE[dtype], budget, sink, recent, total_out,
        k_out.data_ptr(), v_out.data_ptr(), weights_out.data_ptr(), index_out.data_ptr(),
        cu_out.data_ptr(), _stream(stream, k))
    if st != VLF_OK:
        _check(st, "vlf_cache_evict")
    if n == 0:  # (for an empty batch the library enqueues nothing)
        cu_out.zero_()
    return outs


# ------------------------------------------------------------------ serving from a cache of pages in 8 bits
_I32, _F32, _E4M3 = torch.int32, torch.float32, getattr(torch, "float8_e4m3fn", None)


def _at16(t):
    """t, or a copy of a slice that starts anywhere: the library takes 16-byte aligned pointers."""
    return t if t is None or t.data_ptr() % 16 == 0 else t.clone()


def _room(workspace, need, like):
    """(pointer, bytes) of the caller's workspace, or of one allocated here, and the tensor to keep."""
    if workspace is None:
        if need <= 0:
            return None, 0, None
        workspace = torch.empty(need, dtype=torch.uint8, device=like.device)
    else:
        _req(workspace, "workspace"), _same_device(like, workspace=workspace)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _turns(like, total, positions, inv_freq, sections):
    """The arguments of the rotary positions, checked: (positions, axes, sections, inv_freq, rot); positions
    and inv_freq may be None, for none."""
    if positions is None or inv_freq is None:
        if positions is not None or inv_freq is not None or sections is not None:
            raise VlfError(VLF_ERR_INVALID, "positions and inv_freq go together")
        return None, 1, None, None, 0
    _req(positions, "positions", _I32), _req(inv_freq, "inv_freq", _F32)
    _same_device(like, positions=positions, inv_freq=inv_freq)
    if not 1 <= positions.dim() <= 2 or positions.shape[-1] != total or inv_freq.dim() != 1:
        raise VlfError(VLF_ERR_INVALID, "positions must be [tokens] or [axes, tokens], inv_freq [rot / 2]")
    axes = 1 if positions.dim() == 1 else positions.shape[0]
    if sections is None:
        if axes != 1:
            raise VlfError(VLF_ERR_INVALID, "several position axes need sections")
    elif len(sections) != axes:
        raise VlfError(VLF_ERR_INVALID, f"{len(sections)} sections for {axes} position axes")
    _fits(axes, 2 * inv_freq.shape[0])
    return positions, axes, None if sections is None else _sections(sections), inv_freq, 2 * inv_freq.shape[0]


def _norm_weights(like, q_weight, k_weight, d):
    """Checks the weights and returns their type (the same for both)."""
    dtype = None
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is None:
            continue
        _given(w, name, (d,), dtype)
        if w.dtype not in (like.dtype, _F32):
            raise VlfError(VLF_ERR_INVALID, f"{name} must be {like.dtype} or {_F32}, got {w.dtype}")
        _same_device(like, **{name: w})
        dtype = w.dtype
    return like.dtype if dtype is None else dtype


def _eps(eps):
    eps = float(eps)
    if not 0.0 <= eps < 3.4e38:
        raise VlfError(VLF_ERR_INVALID, f"eps = {eps} is out of range")
    return eps


def _rows_like(out, name, like, strides):
    """The caller's output of ``like``'s shape and type, or a dense one; its token stride is appended."""
    if out is None:
        out = torch.empty(like.shape, dtype=like.dtype, device=like.device)
    stride = _rope_rows(out, name, like.dtype, like.shape[0])
    if out.shape != like.shape:
        raise VlfError(VLF_ERR_INVALID, f"{name} must have the shape {tuple(like.shape)}")
    _same_device(like, **{name: out})
    strides.append(stride)
    return out


def _norm_rows(q, k):
    """Checks q and k [tokens, heads, d] of one type; (token strides, total, h_q, h_k, d)."""
    if q.dtype not in _DTYPE:
        raise VlfError(VLF_ERR_INVALID, f"unsupported dtype {q.dtype}")
    strides = [_rope_rows(q, "q", q.dtype)]
    total, hq, d = q.shape
    hk = 0
    if k is not None:
        strides.append(_rope_rows(k, "k", q.dtype, total))
        if k.shape[2] != d:
            raise VlfError(VLF_ERR_INVALID, "q and k must have the same head_dim")
        _same_device(q, k=k)
        hk = k.shape[1]
    else:
        strides.append(0)
    _fits(total, hq, hk, d)
    return strides, total, hq, hk, d


def vlf_norm_rope(q, k, q_weight, k_weight, positions=None, inv_freq=None, sections=None,
                  interleaved=False, eps=1e-6, q_out=None, k_out=None, stream=None):
    """Root-mean-square norm of each head of q [T,Hq,D] and k [T,Hk,D] (k may be None), times the weights
    ``q_weight`` / ``k_weight`` [D] (None: ones; q's type or fp32), and the rotary positions of ``vlf_rope``
    in the same pass (``positions`` and ``inv_freq`` None: the norm alone).  q and k may be slices of a
    packed projection, the outputs q / k themselves.  Returns (q_out, k_out)."""
    if q_out is None and k_out is None and stream is None:
        done = _calls.norm_rope(q, k, q_weight, k_weight, positions, inv_freq, sections, interleaved, eps)
        if done is not None:
            return done
    if _elsewhere(q):
        with torch.cuda.device(q.device):
            return vlf_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, sections, interleaved, eps,
                                 q_out, k_out, stream)
    if _another(stream, q):
        return _under(stream, (q_out, k_out), lambda: vlf_norm_rope(
            q, k, q_weight, k_weight, positions, inv_freq, sections, interleaved, eps, q_out, k_out))
    (sq, sk), total, hq, hk, d = _norm_rows(q, k)
    if k is None and (k_out is not None or k_weight is not None):
        raise VlfError(VLF_ERR_INVALID, "k_out or k_weight without k")
    w_dtype = _norm_weights(q, q_weight, k_weight, d)
    positions, axes, sec, inv_freq, rot = _turns(q, total, positions, inv_freq, sections)
    q_weight, k_weight, positions, inv_freq = map(_at16, (q_weight, k_weight, positions, inv_freq))
    so = []
    q_out = _rows_like(q_out, "q_out", q, so)
    k_out = _rows_like(k_out, "k_out", k, so) if k is not None else so.append(0)
    _check(_lib.vlf_norm_rope(
        _ptr(q), sq, _ptr(k), sk, _ptr(q_weight), _ptr(k_weight), _DTYPE[w_dtype], _eps(eps), _ptr(positions),
        axes, sec, _ptr(inv_freq), total, hq, hk, d, rot, _DTYPE[q.dtype], int(bool(interleaved)),
        _ptr(q_out), so[0], _ptr(k_out), so[1], _stream(stream, q)), "vlf_norm_rope")
    return q_out, k_out


def vlf_norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, positions=None, inv_freq=None,
                      sections=None, interleaved=False, eps=1e-6, dq=None, dk=None, dq_weight=None,
                      dk_weight=None, workspace=None, stream=None):
    """Gradients of vlf_norm_rope: ``dq_out`` / ``dk_out`` are those of its outputs, the other arguments its
    own.  Returns (dq, dk, dq_weight, dk_weight), None where the input is None.  ``workspace``: at least
    vlf_norm_rope_bwd_workspace_size bytes, allocated here when not given."""
    if dq is None and dk is None and dq_weight is None and dk_weight is None and workspace is None and stream is None:
        done = _calls.norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, positions, inv_freq, sections,
                                    interleaved, eps)
        if done is not None:
            return done
    if _elsewhere(q):
        with torch.cuda.device(q.device):
            return vlf_norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, positions, inv_freq, sections,
                                     interleaved, eps, dq, dk, dq_weight, dk_weight, workspace, stream)
    if _another(stream, q):
        return _under(stream, (dq, dk, dq_weight, dk_weight), lambda: vlf_norm_rope_bwd(
            dq_out, dk_out, q, k, q_weight, k_weight, positions, inv_freq, sections, interleaved, eps, dq, dk,
            dq_weight, dk_weight, workspace))
    (sq, sk), total, hq, hk, d = _norm_rows(q, k)
    if k is None and any(t is not None for t in (dk_out, dk, k_weight, dk_weight)):
        raise VlfError(VLF_ERR_INVALID, "dk_out, dk, k_weight or dk_weight without k")
    w_dtype = _norm_weights(q, q_weight, k_weight, d)
    positions, axes, sec, inv_freq, rot = _turns(q, total, positions, inv_freq, sections)
    q_weight, k_weight, positions, inv_freq = map(_at16, (q_weight, k_weight, positions, inv_freq))
    sg, so = [], []
    for t, name, x in ((dq_out, "dq_out", q), (dk_out, "dk_out", k)):
        if x is not None:
            if t is None:
                raise VlfError(VLF_ERR_INVALID, f"{name} is None")
            _rows_like(t, name, x, sg)
    dq = _rows_like(dq, "dq", q, so)
    dk = _rows_like(dk, "dk", k, so) if k is not None else so.append(0)
    grads = []
    for w, dw, name in ((q_weight, dq_weight, "dq_weight"), (k_weight, dk_weight, "dk_weight")):
        if w is None and dw is not None:
            raise VlfError(VLF_ERR_INVALID, f"{name} without its weight")
        if w is not None and dw is None:
            dw = torch.empty_like(w)
        if w is not None:
            _given(dw, name, (d,), w_dtype), _same_device(q, **{name: dw})
        grads.append(dw)
    need = vlf_norm_rope_bwd_workspace_size(d) if q_weight is not None or k_weight is not None else 0
    ws_p, ws_n, workspace = _room(workspace, need, q)
    _check(_lib.vlf_norm_rope_bwd(
        _ptr(dq_out), sg[0], _ptr(dk_out), sg[1] if k is not None else 0, _ptr(q), sq, _ptr(k), sk, _ptr(q_weight),
        _ptr(k_weight), _DTYPE[w_dtype], _eps(eps), _ptr(positions), axes, sec, _ptr(inv_freq), total, hq, hk, d,
        rot, _DTYPE[q.dtype], int(bool(interleaved)), _ptr(dq), so[0], _ptr(dk), so[1], _ptr(grads[0]),
        _ptr(grads[1]), ws_p, ws_n, _stream(stream, q)), "vlf_norm_rope_bwd")
    return dq, dk, grads[0], grads[1]


def vlf_norm_rope_bwd_workspace_size(d) -> int:
    return int(_lib.vlf_norm_rope_bwd_workspace_size(_c_int(d, "d")))


def _pool(k_pages, v_pages, k_scale, v_scale):
    """Checks a layer's pages and scales; (num_pages, h_kv, page, d_qk, d_v)."""
    for t, name in ((k_pages, "k_pages"), (v_pages, "v_pages")):
        _req(t, name)
        if t.dtype not in (torch.uint8, _E4M3):
            raise VlfError(VLF_ERR_INVALID, f"{name} must be {_E4M3} or {torch.uint8}, got {t.dtype}")
        if t.dim() != 4:
            raise VlfError(VLF_ERR_INVALID, f"{name} must be [num_pages, H_kv, page, head_dim]")
    n, h, page, dk = k_pages.shape
    dv = v_pages.shape[3]
    if v_pages.shape[:3] != k_pages.shape[:3]:
        raise VlfError(VLF_ERR_INVALID, "k_pages and v_pages must have the same pages, heads and page size")
    _given(k_scale, "k_scale", (n, h), _F32), _given(v_scale, "v_scale", (n, h), _F32)
    _same_device(k_pages, v_pages=v_pages, k_scale=k_scale, v_scale=v_scale)
    _fits(n, h, page, dk, dv)
    return n, h, page, dk, dv


def _table(like, page_table, lens, names=("page_table", "seqlens_kv")):
    """Checks a page table [num_seqs, max_pages] and its sequences' lengths; (num_seqs, max_pages)."""
    _req(page_table, names[0], _I32), _req(lens, names[1], _I32)
    _same_device(like, **{names[0]: page_table, names[1]: lens})
    if page_table.dim() != 2 or lens.shape != page_table.shape[:1]:
        raise VlfError(VLF_ERR_INVALID, f"{names[0]} must be [num_seqs, max_pages] and {names[1]} [num_seqs]")
    _fits(*page_table.shape)
    return page_table.shape


def vlf_pages_write(k, v, k_pages, v_pages, k_scale, v_scale, page_table, cu_seqlens, seqlens_kv, stream=None):
    """New keys and values into their pages.  k [T,Hkv,Dk], v [T,Hkv,Dv] (tokens may be strided) packed by
    ``cu_seqlens`` int32 [n + 1]; ``seqlens_kv`` int32 [n] are the sequences' lengths with them;
    ``page_table`` int32 [n, max_pages].  The cache (``k_pages`` [pages,Hkv,page,Dk] and ``v_pages`` in e4m3 or
    uint8, ``k_scale`` / ``v_scale`` fp32 [pages,Hkv]) is written in place: each page has, for each head, one
    power of two as its scale, which grows where a new value needs it (include/vlf.h)."""
    if stream is None and _calls.pages_write(k, v, k_pages, v_pages, k_scale, v_scale, page_table, cu_seqlens,
                                             seqlens_kv):
        return
    if _elsewhere(k):
        with torch.cuda.device(k.device):
            return vlf_pages_write(k, v, k_pages, v_pages, k_scale, v_scale, page_table, cu_seqlens, seqlens_kv,
                                   stream)
    if _another(stream, k):
        return _under(stream, (), lambda: vlf_pages_write(
            k, v, k_pages, v_pages, k_scale, v_scale, page_table, cu_seqlens, seqlens_kv))
    if k.dtype not in _DTYPE:
        raise VlfError(VLF_ERR_INVALID, f"unsupported dtype {k.dtype}")
    sk, sv = _rope_rows(k, "k", k.dtype), _rope_rows(v, "v", k.dtype, k.shape[0])
    pages, h, page, dk, dv = _pool(k_pages, v_pages, k_scale, v_scale)
    total = k.shape[0]
    if k.shape[1:] != (h, dk) or v.shape[1:] != (h, dv):
        raise VlfError(VLF_ERR_INVALID, "k, v must be [tokens, H_kv, head_dim] of the pages' heads and widths")
    _same_device(k, v=v, k_pages=k_pages)
    n, most = _table(k, page_table, seqlens_kv)
    _given(cu_seqlens, "cu_seqlens", (n + 1,), _I32), _same_device(k, cu_seqlens=cu_seqlens)
    _fits(total)
    page_table, cu_seqlens, seqlens_kv = map(_at16, (page_table, cu_seqlens, seqlens_kv))
    _check(_lib.vlf_pages_write(
        _ptr(k), sk, _ptr(v), sv, _ptr(k_pages), _ptr(v_pages), _ptr(k_scale), _ptr(v_scale), _ptr(page_table),
        _ptr(cu_seqlens), _ptr(seqlens_kv), n, total, most, pages, page, h, dk, dv, _DTYPE[k.dtype],
        _stream(stream, k)), "vlf_pages_write")


def vlf_attn_varlen_fwd_pages_workspace_size(num_seqs, total_q, max_seqlen_q, h_q, h_kv, d_qk, d_v, dtype, flags=0,
                                             num_sms=0) -> int:
    dt = _DTYPE[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(_lib.vlf_attn_varlen_fwd_pages_workspace_size(num_seqs, total_q, max_seqlen_q, h_q, h_kv, d_qk, d_v,
                                                             dt, flags, num_sms))


def vlf_attn_varlen_fwd_pages(q, k_pages, v_pages, k_scale, v_scale, page_table, cu_seqlens_q, seqlens_kv,
                              max_seqlen_q, scale=None, causal=False, window=0, out=None, lse=None,
                              workspace=None, stream=None, flags=0):
    """Attention of q [Tq,Hq,Dk] over a cache of pages in e4m3 (see vlf_pages_write for its tensors): sequence
    s has the first ``seqlens_kv[s]`` keys of its row of ``page_table``.  Equals vlf_attn_varlen_fwd on the
    values that the bytes stand for.  Returns out [Tq,Hq,Dv] and lse fp32 [Hq,Tq].  ``workspace``: at least
    vlf_attn_varlen_fwd_pages_workspace_size bytes, allocated here when not given."""
    if out is None and lse is None and workspace is None and stream is None:
        done = _calls.pages_attn(q, k_pages, v_pages, k_scale, v_scale, page_table, cu_seqlens_q, seqlens_kv,
                                 max_seqlen_q, scale, causal, window, flags)
        if done is not None:
            return done
    if _elsewhere(q):
        with torch.cuda.device(q.device):
            return vlf_attn_varlen_fwd_pages(q, k_pages, v_pages, k_scale, v_scale, page_table, cu_seqlens_q,
                                             seqlens_kv, max_seqlen_q, scale, causal, window, out, lse, workspace,
                                             stream, flags)
    if _another(stream, q):
        return _under(stream, (out, lse), lambda: vlf_attn_varlen_fwd_pages(
            q, k_pages, v_pages, k_scale, v_scale, page_table, cu_seqlens_q, seqlens_kv, max_seqlen_q, scale, causal,
            window, out, lse, workspace, flags=flags))
    _req(q, "q")
    if q.dtype not in _DTYPE or q.dim() != 3:
        raise VlfError(VLF_ERR_INVALID, f"q must be [tokens, heads, head_dim] in fp16, bf16 or fp32, got {q.dtype}")
    pages, hkv, page, dqk, dv = _pool(k_pages, v_pages, k_scale, v_scale)
    tq, hq, d = q.shape
    if d != dqk:
        raise VlfError(VLF_ERR_INVALID, "q and k_pages must have the same head_dim")
    _same_device(q, k_pages=k_pages)
    n, most = _table(q, page_table, seqlens_kv)
    _given(cu_seqlens_q, "cu_seqlens_q", (n + 1,), _I32), _same_device(q, cu_seqlens_q=cu_seqlens_q)
    _fits(tq, hq)
    if out is None:
        out = torch.empty((tq, hq, dv), dtype=q.dtype, device=q.device)
    else:
        _given(out, "out", (tq, hq, dv), q.dtype), _same_device(q, out=out)
    if lse is None:
        lse = torch.empty((hq, tq), dtype=_F32, device=q.device)
    else:
        _given(lse, "lse", (hq, tq), _F32), _same_device(q, lse=lse)
    mq, window, dt, flags = _c_int(max_seqlen_q, "max_seqlen_q"), _c_int(window or 0, "window"), _DTYPE[q.dtype], int(flags)
    page_table, cu_seqlens_q, seqlens_kv = map(_at16, (page_table, cu_seqlens_q, seqlens_kv))
    need = _workspace_size(_lib.vlf_attn_varlen_fwd_pages_workspace_size,
                           ("pages", n, tq, mq, hq, hkv, dqk, dv, dt, flags, q.get_device()))
    ws_p, ws_n, workspace = _room(workspace, need, q)
    _check(_lib.vlf_attn_varlen_fwd_pages(
        _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(k_scale), _ptr(v_scale), _ptr(page_table), _ptr(cu_seqlens_q),
        _ptr(seqlens_kv), n, tq, mq, most, pages, page, hq, hkv, dqk, dv, dt, float(scale) if scale else 0.0,
        int(bool(causal)), window, _ptr(out), _ptr(lse), ws_p, ws_n, _stream(stream, q), flags),
        "vlf_attn_varlen_fwd_pages")
    return out, lse


def vlf_pages_copy(k_pages, v_pages, k_scale, v_scale, src, dst, stream=None):
    """Copies page src[i] (keys, values and scales) over page dst[i] for each i with src[i] >= 0; ``src`` and
    ``dst`` int32 [n], as vlf_pages_fork and vlf_pages_compact return them (a page is in dst once at most,
    and not in src as well).  In place; called for each layer's cache."""
    if stream is None and _calls.pages_copy(k_pages, v_pages, k_scale, v_scale, src, dst):
        return
    if _elsewhere(k_pages):
        with torch.cuda.device(k_pages.device):
            return vlf_pages_copy(k_pages, v_pages, k_scale, v_scale, src, dst, stream)
    if _another(stream, k_pages):
        return _under(stream, (), lambda: vlf_pages_copy(k_pages, v_pages, k_scale, v_scale, src, dst))
    pages, h, page, dk, dv = _pool(k_pages, v_pages, k_scale, v_scale)
    _req(src, "src", _I32), _req(dst, "dst", _I32), _same_device(k_pages, src=src, dst=dst)
    if src.dim() != 1 or dst.shape != src.shape:
        raise VlfError(VLF_ERR_INVALID, "src and dst must be [n]")
    _fits(src.shape[0])
    src, dst = _at16(src), _at16(dst)
    _check(_lib.vlf_pages_copy(
        _ptr(k_pages), _ptr(v_pages), _ptr(k_scale), _ptr(v_scale), _ptr(src), _ptr(dst), src.shape[0], pages, page, h,
        dk, dv, _stream(stream, k_pages)), "vlf_pages_copy")


def vlf_pages_fork_workspace_size(num_pages, num_out) -> int:
    return int(_lib.vlf_pages_fork_workspace_size(_c_int(num_pages, "num_pages"), _c_int(num_out, "num_out")))


def vlf_pages_fork(page_table, seqlens, refs, parents, grow, page_size, table_out=None, seqlens_out=None,
                   refs_out=None, src=None, dst=None, left=None, workspace=None, stream=None):
    """The page tables of the next step: new row s follows old row ``parents[s]`` (-1: it begins empty) and has
    room for ``grow[s]`` more tokens.  ``page_table`` int32 [n, max_pages], ``seqlens`` [n], ``refs`` [pages]
    (how many hold each page), ``parents`` and ``grow`` [m].  A row that is no one's parent gives its pages
    back, whole pages are shared, and a page that is not full has one holder: the other rows get
    copies.  Returns (table [m, max_pages], seqlens [m] with the growth, refs [pages], src [m], dst [m],
    left [1]); src and dst are for vlf_pages_copy of every layer, before anything is written; left, the free
    pages that are left, is negative where there were too few: nothing has changed then, and the tables
    returned are empty (include/vlf.h).  Nothing is read on the host.  Outputs that the call makes may share one
    allocation, its workspace (up to 256 KB) behind them: one that is kept, or saved to a file, keeps or saves all, so
    clone what outlives the step."""
    if all(t is None for t in (table_out, seqlens_out, refs_out, src, dst, left, workspace, stream)):
        done = _calls.pages_fork(page_table, seqlens, refs, parents, grow, page_size)
        if done is not None:
            return done
    if _elsewhere(refs):
        with torch.cuda.device(refs.device):
            return vlf_pages_fork(page_table, seqlens, refs, parents, grow, page_size, table_out, seqlens_out,
                                  refs_out, src, dst, left, workspace, stream)
    if _another(stream, refs):
        return _under(stream, (table_out, seqlens_out, refs_out, src, dst, left), lambda: vlf_pages_fork(
            page_table, seqlens, refs, parents, grow, page_size, table_out, seqlens_out, refs_out, src, dst, left,
            workspace))
    _req(refs, "refs", _I32), _req(parents, "parents", _I32), _req(grow, "grow", _I32)
    n, most = _table(refs, page_table, seqlens, ("page_table", "seqlens"))
    _same_device(refs, parents=parents, grow=grow)
    if refs.dim() != 1 or parents.dim() != 1 or grow.shape != parents.shape:
        raise VlfError(VLF_ERR_INVALID, "refs must be [num_pages], parents and grow [m]")
    m, pages = parents.shape[0], refs.shape[0]
    _fits(m, pages)
    outs = []
    for t, name, shape in ((table_out, "table_out", (m, most)), (seqlens_out, "seqlens_out", (m,)),
                           (refs_out, "refs_out", (pages,)), (src, "src", (m,)), (dst, "dst", (m,)),
                           (left, "left", (1,))):
        if t is None:
            t = torch.empty(shape, dtype=_I32, device=refs.device)
        _given(t, name, shape, _I32), _same_device(refs, **{name: t})
        outs.append(t)
    page_table, seqlens, refs, parents, grow = map(_at16, (page_table, seqlens, refs, parents, grow))
    ws_p, ws_n, workspace = _room(workspace, vlf_pages_fork_workspace_size(pages, m), refs)
    _check(_lib.vlf_pages_fork(
        _ptr(page_table), _ptr(seqlens), _ptr(refs), _ptr(parents), _ptr(grow), n, m, most, pages,
        _c_int(page_size, "page_size"), *map(_ptr, outs), ws_p, ws_n, _stream(stream, refs)), "vlf_pages_fork")
    return tuple(outs)


def vlf_pages_compact_workspace_size(num_pages) -> int:
    return int(_lib.vlf_pages_compact_workspace_size(_c_int(num_pages, "num_pages")))


def vlf_pages_compact(page_table, refs, table_out=None, refs_out=None, to=None, src=None, dst=None, used=None,
                      workspace=None, stream=None):
    """The pages in use (``refs`` [pages] above 0) moved to the front of the pool.  Returns (table, refs, to, src,
    dst, used): the tables and counts afterwards, where each page in use then is (-1: it was free), the
    copies to make (int32 [pages // 2], -1 behind them) with vlf_pages_copy of every layer, and int32 [1]
    how many pages are in use.  Nothing is read on the host.  Outputs share their memory as vlf_pages_fork's do."""
    if all(t is None for t in (table_out, refs_out, to, src, dst, used, workspace, stream)):
        done = _calls.pages_compact(page_table, refs)
        if done is not None:
            return done
    if _elsewhere(refs):
        with torch.cuda.device(refs.device):
            return vlf_pages_compact(page_table, refs, table_out, refs_out, to, src, dst, used, workspace, stream)
    if _another(stream, refs):
        return _under(stream, (table_out, refs_out, to, src, dst, used), lambda: vlf_pages_compact(
            page_table, refs, table_out, refs_out, to, src, dst, used, workspace))
    _req(page_table, "page_table", _I32), _req(refs, "refs", _I32), _same_device(refs, page_table=page_table)
    if page_table.dim() != 2 or refs.dim() != 1:
        raise VlfError(VLF_ERR_INVALID, "page_table must be [num_seqs, max_pages], refs [num_pages]")
    n, most = page_table.shape
    pages = refs.shape[0]
    _fits(n, most, pages)
    outs = []
    for t, name, shape in ((table_out, "table_out", (n, most)), (refs_out, "refs_out", (pages,)), (to, "to", (pages,)),
                           (src, "src", (pages // 2,)), (dst, "dst", (pages // 2,)), (used, "used", (1,))):
        if t is None:
            t = torch.empty(shape, dtype=_I32, device=refs.device)
        _given(t, name, shape, _I32), _same_device(refs, **{name: t})
        outs.append(t)
    page_table, refs = _at16(page_table), _at16(refs)
    ws_p, ws_n, workspace = _room(workspace, vlf_pages_compact_workspace_size(pages), refs)
    _check(_lib.vlf_pages_compact(_ptr(page_table), _ptr(refs), n, most, pages, *map(_ptr, outs), ws_p, ws_n,
                                  _stream(stream, refs)), "vlf_pages_compact")
    return tuple(outs)


__all__ = ["vlf_attn_varlen_fwd", "vlf_attn_varlen_bwd", "vlf_attn_varlen_bwd_workspace_size",
           "vlf_bias_bands", "vlf_bias_bands_size",
           "vlf_check_error", "vlf_status_string", "vlf_sched_kv_band", "vlf_sched_q_band",
           "vlf_version", "vlf_launch_count", "vlf_fwd_path", "vlf_bwd_path",
           "vlf_attn_varlen_bwd_noalloc", "vlf_noalloc_scratch_bytes", "VlfError",
           "vlf_rope", "vlf_attn_varlen_fwd_prefix", "vlf_attn_varlen_fwd_prefix_workspace_size",
           "vlf_attn_key_weights", "vlf_attn_key_weights_workspace_size", "vlf_cache_evict",
           "vlf_norm_rope", "vlf_norm_rope_bwd", "vlf_norm_rope_bwd_workspace_size", "vlf_pages_write",
           "vlf_attn_varlen_fwd_pages", "vlf_attn_varlen_fwd_pages_workspace_size", "vlf_pages_copy",
           "vlf_pages_fork", "vlf_pages_fork_workspace_size", "vlf_pages_compact",
           "vlf_pages_compact_workspace_size",
           "LIB_PATH", "EXPORTS"]

# differentiable entry points (autograd over the two calls above)
from .functional import (flash_attn_varlen_func, flash_attn_varlen_kvpacked_func,  # noqa: E402
                         flash_attn_varlen_qkvpacked_func, latent_attention,
                         norm_rotary_embedding, rotary_embedding, varlen_attention)

__all__ += ["varlen_attention", "latent_attention", "rotary_embedding", "norm_rotary_embedding", "flash_attn_varlen_func", "flash_attn_varlen_qkvpacked_func",
            "flash_attn_varlen_kvpacked_func"]
