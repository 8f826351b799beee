"""ctypes binding of libfa.so (include/fa.h).

Two layers:

* ``fa_*`` (every name in ``EXPORTS``: forward, packed forward, the
  backward and its three launches, the packed and allocation-free
  backwards, dropout forward/backward, decode, rotary positions, the paged
  cache and decode over it, status and error helpers):
  the C entry points under the same names, taking raw device pointers (ints)
  and sizes, returning the ``fa_status`` code (or a size).
* ``forward``, ``forward_varlen``, ``backward``, ``backward_varlen``,
  ``backward_noalloc``, ``decode``, ``rope_freqs``, ``rope``,
  ``rope_backward``, ``append_paged``, ``decode_paged``, ``decode_prefix``:
  tensor conveniences that check shapes/dtypes, allocate outputs and workspace with torch unless given
  (device memory and streams are all torch provides) and raise ``FAError``
  on a non-zero status.

Every step of the attention itself runs in the library's CUDA kernels; there
is no fallback.  If ``libfa.so`` is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfa.so")

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT = range(5)
FA_BF16, FA_FP16 = 0, 1

EXPORTS = ("fa_fwd", "fa_fwd_varlen", "fa_bwd_workspace_size", "fa_bwd", "fa_bwd_preprocess", "fa_bwd_main",
           "fa_bwd_finish", "fa_bwd_noalloc", "fa_bwd_varlen_workspace_size", "fa_bwd_varlen", "fa_status_string",
           "fa_check_device_error", "fa_launch_count", "fa_selftest_timeout", "fa_decode_num_splits",
           "fa_decode_workspace_size", "fa_decode", "fa_fwd_dropout", "fa_bwd_dropout", "fa_fwd_varlen_dropout",
           "fa_bwd_varlen_dropout", "fa_rope_freqs", "fa_rope", "fa_rope_fill", "fa_append_paged", "fa_append_paged_fill",
           "fa_decode_paged_workspace_size",
           "fa_decode_paged", "fa_decode_prefix_workspace_size", "fa_decode_prefix")

# fa_rope_scaling, and the layouts of the structs fa_rows and fa_pages of include/fa.h
ROPE_SCALING = {None: 0, "linear": 1, "ntk": 2, "yarn": 3}
_ROWS = struct.Struct("@Pqqqi4x")   # data; batch, head, row stride; heads
_PAGES = struct.Struct("@PPqPqiiii")  # k, v; page stride; table, its stride; n_pages, page_size, heads, max_pages

# Fixed scratch size of fa_bwd_noalloc (FA_BWD_NOALLOC_SCRATCH_BYTES in include/fa.h).
NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024

_lib = None


class FAError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {fa_status_string(status)} ({status})")
        self.status = status


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libfa.so once; raise loudly if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build it with `python -m exact_tiled_attention_31_b200.build` "
            "(there is no non-CUDA implementation to fall back to)")
    lib = ctypes.CDLL(path)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, i, vp]
    lib.fa_fwd.restype = i
    lib.fa_fwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp]
    lib.fa_fwd_varlen.restype = i
    lib.fa_bwd_workspace_size.argtypes = [i, i, i, i]
    lib.fa_bwd_workspace_size.restype = sz
    lib.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, i, i, vp, sz, vp]
    lib.fa_bwd.restype = i
    lib.fa_bwd_preprocess.argtypes = [vp, vp, vp, i, i, i, i, i, vp, sz, vp]
    lib.fa_bwd_preprocess.restype = i
    lib.fa_bwd_main.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, i, i, vp, sz, vp]
    lib.fa_bwd_main.restype = i
    lib.fa_bwd_finish.argtypes = [vp, i, i, i, i, f, i, i, vp, sz, vp]
    lib.fa_bwd_finish.restype = i
    lib.fa_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, i, i, vp]
    lib.fa_bwd_noalloc.restype = i
    lib.fa_bwd_varlen_workspace_size.argtypes = [i, i, i, i, i]
    lib.fa_bwd_varlen_workspace_size.restype = sz
    lib.fa_bwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, i, vp, sz, vp]
    lib.fa_bwd_varlen.restype = i
    lib.fa_status_string.argtypes = [i]
    lib.fa_status_string.restype = ctypes.c_char_p
    lib.fa_check_device_error.argtypes = [vp]
    lib.fa_check_device_error.restype = i
    lib.fa_selftest_timeout.argtypes = [vp]
    lib.fa_selftest_timeout.restype = i
    lib.fa_decode_num_splits.argtypes = [i, i, i]
    lib.fa_decode_num_splits.restype = i
    lib.fa_decode_workspace_size.argtypes = [i, i, i, i]
    lib.fa_decode_workspace_size.restype = sz
    lib.fa_decode.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp, sz, vp]
    lib.fa_decode.restype = i
    u64 = ctypes.c_uint64
    lib.fa_fwd_dropout.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, i, f, u64, u64, vp]
    lib.fa_fwd_dropout.restype = i
    lib.fa_bwd_dropout.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, i, i, f, u64, u64, vp, sz, vp]
    lib.fa_bwd_dropout.restype = i
    lib.fa_fwd_varlen_dropout.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, f, u64, u64, vp]
    lib.fa_fwd_varlen_dropout.restype = i
    lib.fa_bwd_varlen_dropout.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, i, f, u64,
                                          u64, vp, sz, vp]
    lib.fa_bwd_varlen_dropout.restype = i
    d, i64 = ctypes.c_double, ctypes.c_longlong
    lib.fa_rope_freqs.argtypes = [i, d, i, d, i, d, d, vp, vp]
    lib.fa_rope_freqs.restype = i
    lib.fa_rope.argtypes = [vp, vp, i, vp, i, i, f, i, vp, i64, vp, i, i, i, i, i, vp]
    lib.fa_rope.restype = i
    lib.fa_rope_fill.argtypes, lib.fa_rope_fill.restype = lib.fa_rope.argtypes, i
    lib.fa_append_paged.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, vp, i, i, f, vp, i, i, vp]
    lib.fa_append_paged.restype = i
    lib.fa_append_paged_fill.argtypes, lib.fa_append_paged_fill.restype = lib.fa_append_paged.argtypes, i
    lib.fa_decode_paged_workspace_size.argtypes = [i, i, i, i]
    lib.fa_decode_paged_workspace_size.restype = sz
    lib.fa_decode_paged.argtypes = [vp, vp, vp, vp, vp, i, i, i, f, i, vp, sz, vp]
    lib.fa_decode_paged.restype = i
    lib.fa_decode_prefix_workspace_size.argtypes = [i, i, i, i, i]
    lib.fa_decode_prefix_workspace_size.restype = sz
    lib.fa_decode_prefix.argtypes = [vp, vp, vp, i, vp, vp, vp, i, i, i, f, i, vp, sz, vp]
    lib.fa_decode_prefix.restype = i
    lib.fa_launch_count.argtypes = []
    lib.fa_launch_count.restype = ctypes.c_uint64
    _lib = lib
    return lib


# ---------------------------------------------------------------- raw entry points

def fa_fwd(q, k, v, o, lse, B, H, S, D, scale, causal, dt, stream) -> int:
    return load_library().fa_fwd(q, k, v, o, lse, B, H, S, D, scale, int(causal), dt, stream)


def fa_fwd_varlen(q, k, v, o, lse, cu_seqlens, nseq, max_seqlen, total, H, D, scale, causal, dt, stream) -> int:
    return load_library().fa_fwd_varlen(q, k, v, o, lse, cu_seqlens, nseq, max_seqlen, total, H, D, scale,
                                        int(causal), dt, stream)


def fa_bwd_workspace_size(B, H, S, D) -> int:
    return load_library().fa_bwd_workspace_size(B, H, S, D)


def fa_bwd(q, k, v, o, dO, lse, dq, dk, dv, B, H, S, D, scale, causal, dt, deterministic, workspace,
           workspace_bytes, stream) -> int:
    return load_library().fa_bwd(q, k, v, o, dO, lse, dq, dk, dv, B, H, S, D, scale, int(causal), dt,
                                 int(deterministic), workspace, workspace_bytes, stream)


def fa_bwd_preprocess(o, dO, lse, B, H, S, D, dt, workspace, workspace_bytes, stream) -> int:
    return load_library().fa_bwd_preprocess(o, dO, lse, B, H, S, D, dt, workspace, workspace_bytes, stream)


def fa_bwd_main(q, k, v, dO, dk, dv, B, H, S, D, scale, causal, dt, deterministic, workspace, workspace_bytes,
                stream) -> int:
    return load_library().fa_bwd_main(q, k, v, dO, dk, dv, B, H, S, D, scale, int(causal), dt, int(deterministic),
                                      workspace, workspace_bytes, stream)


def fa_bwd_finish(dq, B, H, S, D, scale, dt, deterministic, workspace, workspace_bytes, stream) -> int:
    return load_library().fa_bwd_finish(dq, B, H, S, D, scale, dt, int(deterministic), workspace, workspace_bytes,
                                        stream)


def fa_bwd_noalloc(q, k, v, o, dO, lse, dq, dk, dv, B, H, S, D, scale, causal, dt, deterministic,
                   stream) -> int:
    return load_library().fa_bwd_noalloc(q, k, v, o, dO, lse, dq, dk, dv, B, H, S, D, scale, int(causal), dt,
                                         int(deterministic), stream)


def fa_bwd_varlen_workspace_size(nseq, max_seqlen, total, H, D) -> int:
    return load_library().fa_bwd_varlen_workspace_size(nseq, max_seqlen, total, H, D)


def fa_bwd_varlen(q, k, v, o, dO, lse, dq, dk, dv, cu_seqlens, nseq, max_seqlen, total, H, D, scale, causal, dt,
                  deterministic, workspace, workspace_bytes, stream) -> int:
    return load_library().fa_bwd_varlen(q, k, v, o, dO, lse, dq, dk, dv, cu_seqlens, nseq, max_seqlen, total, H, D,
                                        scale, int(causal), dt, int(deterministic), workspace, workspace_bytes,
                                        stream)


def fa_fwd_dropout(q, k, v, o, lse, B, H, S, D, scale, causal, dt, dropout_p, seed, offset, stream) -> int:
    return load_library().fa_fwd_dropout(q, k, v, o, lse, B, H, S, D, scale, int(causal), dt, dropout_p, seed, offset,
                                         stream)


def fa_bwd_dropout(q, k, v, o, dO, lse, dq, dk, dv, B, H, S, D, scale, causal, dt, deterministic, dropout_p, seed,
                   offset, workspace, workspace_bytes, stream) -> int:
    return load_library().fa_bwd_dropout(q, k, v, o, dO, lse, dq, dk, dv, B, H, S, D, scale, int(causal), dt,
                                         int(deterministic), dropout_p, seed, offset, workspace, workspace_bytes,
                                         stream)


def fa_fwd_varlen_dropout(q, k, v, o, lse, cu_seqlens, nseq, max_seqlen, total, H, D, scale, causal, dt, dropout_p,
                          seed, offset, stream) -> int:
    return load_library().fa_fwd_varlen_dropout(q, k, v, o, lse, cu_seqlens, nseq, max_seqlen, total, H, D, scale,
                                                int(causal), dt, dropout_p, seed, offset, stream)


def fa_bwd_varlen_dropout(q, k, v, o, dO, lse, dq, dk, dv, cu_seqlens, nseq, max_seqlen, total, H, D, scale, causal,
                          dt, deterministic, dropout_p, seed, offset, workspace, workspace_bytes, stream) -> int:
    return load_library().fa_bwd_varlen_dropout(q, k, v, o, dO, lse, dq, dk, dv, cu_seqlens, nseq, max_seqlen, total,
                                                H, D, scale, int(causal), dt, int(deterministic), dropout_p, seed,
                                                offset, workspace, workspace_bytes, stream)


def fa_decode_num_splits(B, Hkv, L_max) -> int:
    return load_library().fa_decode_num_splits(B, Hkv, L_max)


def fa_decode_workspace_size(B, Hq, n_splits, D) -> int:
    return load_library().fa_decode_workspace_size(B, Hq, n_splits, D)


def fa_decode(q, k_cache, v_cache, seq_lens, o, lse, B, Hq, Hkv, L_max, D, scale, dt, n_splits, workspace,
              workspace_bytes, stream) -> int:
    return load_library().fa_decode(q, k_cache, v_cache, seq_lens, o, lse, B, Hq, Hkv, L_max, D, scale, dt, n_splits,
                                    workspace, workspace_bytes, stream)


def fa_rope_freqs(rot_dim, base, scaling, factor, original_len, beta_fast, beta_slow, freqs, amp) -> int:
    return load_library().fa_rope_freqs(rot_dim, base, scaling, factor, original_len, beta_fast, beta_slow, freqs, amp)


def fa_rope(x, y, n, freqs, rot_dim, interleaved, amp, backward, positions, positions_stride, cu_seqlens, nseq, B, S,
            D, dt, stream) -> int:
    """``x`` and ``y``: the bytes of n ``fa_rows`` each (or a pointer to them)."""
    return load_library().fa_rope(x, y, n, freqs, rot_dim, int(interleaved), amp, int(backward), positions,
                                  positions_stride, cu_seqlens, nseq, B, S, D, dt, stream)


def fa_rope_fill(x, y, n, freqs, rot_dim, interleaved, amp, backward, positions, positions_stride, cu_seqlens, nseq, B,
                 S, D, dt, stream) -> int:
    return load_library().fa_rope_fill(x, y, n, freqs, rot_dim, int(interleaved), amp, int(backward), positions,
                                       positions_stride, cu_seqlens, nseq, B, S, D, dt, stream)


def fa_append_paged(k, v, q, q_out, pages, seq_lens, cu_seqlens, nseq, total, freqs, rot_dim, interleaved, amp,
                    positions, D, dt, stream) -> int:
    """``k``, ``v``, ``q``, ``q_out``: the bytes of one ``fa_rows`` each, ``pages``: of an ``fa_pages``."""
    return load_library().fa_append_paged(k, v, q, q_out, pages, seq_lens, cu_seqlens, nseq, total, freqs, rot_dim,
                                          int(interleaved), amp, positions, D, dt, stream)


def fa_append_paged_fill(k, v, q, q_out, pages, seq_lens, cu_seqlens, nseq, total, freqs, rot_dim, interleaved, amp,
                         positions, D, dt, stream) -> int:
    return load_library().fa_append_paged_fill(k, v, q, q_out, pages, seq_lens, cu_seqlens, nseq, total, freqs, rot_dim,
                                               int(interleaved), amp, positions, D, dt, stream)


def fa_decode_paged_workspace_size(B, Hq, Hkv, D) -> int:
    return load_library().fa_decode_paged_workspace_size(B, Hq, Hkv, D)


def fa_decode_paged(q, pages, seq_lens, o, lse, B, Hq, D, scale, dt, workspace, workspace_bytes, stream) -> int:
    """``pages``: the bytes of an ``fa_pages`` (or a pointer to it)."""
    return load_library().fa_decode_paged(q, pages, seq_lens, o, lse, B, Hq, D, scale, dt, workspace, workspace_bytes,
                                          stream)


def fa_decode_prefix_workspace_size(B, Hq, Hkv, prefix_len, D) -> int:
    return load_library().fa_decode_prefix_workspace_size(B, Hq, Hkv, prefix_len, D)


def fa_decode_prefix(q, pages, seq_lens, prefix_len, prefix_table, o, lse, B, Hq, D, scale, dt, workspace,
                     workspace_bytes, stream) -> int:
    """``pages``: the bytes of an ``fa_pages`` (or a pointer to it)."""
    return load_library().fa_decode_prefix(q, pages, seq_lens, prefix_len, prefix_table, o, lse, B, Hq, D, scale, dt,
                                           workspace, workspace_bytes, stream)


def fa_status_string(status: int) -> str:
    return load_library().fa_status_string(status).decode()


def fa_check_device_error(stream) -> int:
    return load_library().fa_check_device_error(stream)


def fa_selftest_timeout(stream) -> int:
    return load_library().fa_selftest_timeout(stream)


def fa_launch_count() -> int:
    return load_library().fa_launch_count()


# ---------------------------------------------------------------- tensor conveniences

def _dt(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return FA_BF16
    if t.dtype == torch.float16:
        return FA_FP16
    raise TypeError(f"expected bf16 or fp16 tensors, got {t.dtype}")


def _check(ts, shape):
    for t in ts:
        if not t.is_cuda:
            raise ValueError("tensors must live on a CUDA device")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"shape {tuple(t.shape)} != {tuple(shape)}")
        if t.dtype != ts[0].dtype:
            raise TypeError("all tensors must share one dtype")


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def forward(q, k, v, causal: bool, scale: float | None = None, out=None, lse=None, stream=None,
            dropout_p: float = 0.0, seed: int = 0, offset: int = 0):
    """O, LSE of [B, H, S, D] inputs; LSE is fp32 [B, H, S].  ``dropout_p`` > 0
    drops attention probabilities with the counter-based mask of (seed, offset)."""
    import torch
    B, H, S, D = q.shape
    _check((q, k, v), q.shape)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    o = torch.empty_like(q) if out is None else out
    lse = torch.empty((B, H, S), device=q.device, dtype=torch.float32) if lse is None else lse
    if dropout_p:
        st = fa_fwd_dropout(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, H, S, D,
                            scale, causal, _dt(q), float(dropout_p), int(seed), int(offset), _stream(stream))
        if st != FA_OK:
            raise FAError(st, "fa_fwd_dropout")
        return o, lse
    st = fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, H, S, D, scale,
                causal, _dt(q), _stream(stream))
    if st != FA_OK:
        raise FAError(st, "fa_fwd")
    return o, lse


def forward_varlen(q, k, v, cu_seqlens, max_seqlen: int, causal: bool, scale: float | None = None,
                   stream=None, dropout_p: float = 0.0, seed: int = 0, offset: int = 0):
    """Packed [H, T, D] forward; ``cu_seqlens`` is a device int32 tensor.
    ``dropout_p`` > 0 drops P with sequence s taking the mask of batch index
    s of a dense batch (fa_fwd_varlen_dropout)."""
    import torch
    H, T, D = q.shape
    _check((q, k, v), q.shape)
    if cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_cuda:
        raise TypeError("cu_seqlens must be a CUDA int32 tensor")
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    o = torch.empty_like(q)
    lse = torch.empty((H, T), device=q.device, dtype=torch.float32)
    if dropout_p:
        st = fa_fwd_varlen_dropout(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                   cu_seqlens.data_ptr(), cu_seqlens.numel() - 1, int(max_seqlen), T, H, D, scale,
                                   causal, _dt(q), float(dropout_p), int(seed), int(offset), _stream(stream))
        if st != FA_OK:
            raise FAError(st, "fa_fwd_varlen_dropout")
        return o, lse
    st = fa_fwd_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                       cu_seqlens.data_ptr(), cu_seqlens.numel() - 1, int(max_seqlen), T, H, D, scale, causal,
                       _dt(q), _stream(stream))
    if st != FA_OK:
        raise FAError(st, "fa_fwd_varlen")
    return o, lse


def backward(q, k, v, o, do, lse, causal: bool, scale: float | None = None, deterministic: bool = False,
             workspace=None, stream=None, dropout_p: float = 0.0, seed: int = 0, offset: int = 0, out=None):
    """dQ, dK, dV of [B, H, S, D] inputs given the forward's O and LSE (and
    the forward's dropout_p, seed and offset, if it dropped).  ``out`` may
    give the three output tensors to fill."""
    import torch
    B, H, S, D = q.shape
    _check((q, k, v, o, do), q.shape)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    if out is None:
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    else:
        dq, dk, dv = out
        _check((q, dq, dk, dv), q.shape)
    nbytes = fa_bwd_workspace_size(B, H, S, D)
    if workspace is None or workspace.numel() < nbytes:
        workspace = torch.empty(max(nbytes, 1), device=q.device, dtype=torch.uint8)
    if dropout_p:
        st = fa_bwd_dropout(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(), lse.data_ptr(),
                            dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, S, D, scale, causal, _dt(q),
                            deterministic, float(dropout_p), int(seed), int(offset), workspace.data_ptr(),
                            workspace.numel(), _stream(stream))
        if st != FA_OK:
            raise FAError(st, "fa_bwd_dropout")
        return dq, dk, dv
    st = fa_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(), lse.data_ptr(),
                dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, S, D, scale, causal, _dt(q), deterministic,
                workspace.data_ptr(), workspace.numel(), _stream(stream))
    if st != FA_OK:
        raise FAError(st, "fa_bwd")
    return dq, dk, dv


def backward_varlen(q, k, v, o, do, lse, cu_seqlens, max_seqlen: int, causal: bool, scale: float | None = None,
                    deterministic: bool = False, workspace=None, stream=None, dropout_p: float = 0.0, seed: int = 0,
                    offset: int = 0):
    """dQ, dK, dV of a packed [H, T, D] batch given fa_fwd_varlen's O and LSE
    (with the forward's dropout_p, seed and offset, if it dropped)."""
    import torch
    H, T, D = q.shape
    _check((q, k, v, o, do), q.shape)
    if cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_cuda:
        raise TypeError("cu_seqlens must be a CUDA int32 tensor")
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    nseq = cu_seqlens.numel() - 1
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    nbytes = fa_bwd_varlen_workspace_size(nseq, int(max_seqlen), T, H, D)
    if workspace is None or workspace.numel() < nbytes:
        workspace = torch.empty(max(nbytes, 1), device=q.device, dtype=torch.uint8)
    args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(), lse.data_ptr(), dq.data_ptr(),
            dk.data_ptr(), dv.data_ptr(), cu_seqlens.data_ptr(), nseq, int(max_seqlen), T, H, D, scale, causal, _dt(q),
            deterministic)
    if dropout_p:
        st = fa_bwd_varlen_dropout(*args, float(dropout_p), int(seed), int(offset), workspace.data_ptr(),
                                   workspace.numel(), _stream(stream))
        if st != FA_OK:
            raise FAError(st, "fa_bwd_varlen_dropout")
        return dq, dk, dv
    st = fa_bwd_varlen(*args, workspace.data_ptr(), workspace.numel(), _stream(stream))
    if st != FA_OK:
        raise FAError(st, "fa_bwd_varlen")
    return dq, dk, dv


def backward_noalloc(q, k, v, o, do, lse, dq, dk, dv, causal: bool, scale: float | None = None,
                     deterministic: bool = False, stream=None):
    """Backward into caller-provided dq, dk, dv with no allocation at all:
    the library's fixed device scratch replaces the workspace (for callers
    that must not allocate device memory; sizes beyond the scratch raise)."""
    B, H, S, D = q.shape
    _check((q, k, v, o, do, dq, dk, dv), q.shape)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    st = fa_bwd_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(), lse.data_ptr(),
                        dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, S, D, scale, causal, _dt(q),
                        deterministic, _stream(stream))
    if st != FA_OK:
        raise FAError(st, "fa_bwd_noalloc")
    return dq, dk, dv


def decode(q, k_cache, v_cache, seq_lens, scale: float | None = None, n_splits: int | None = None, out=None,
           lse=None, workspace=None, stream=None):
    """One decode step: q [B, Hq, D] against caches [B, Hkv, L_max, D] holding
    ``seq_lens`` (CUDA int32 [B]) valid keys each.  Returns O [B, Hq, D] and
    fp32 LSE [B, Hq].  ``n_splits`` defaults to the library's choice."""
    import torch
    B, Hq, D = q.shape
    _check((q,), q.shape)
    _check((k_cache, v_cache), k_cache.shape)
    if k_cache.dtype != q.dtype:
        raise TypeError("q and the caches must share one dtype")
    Bk, Hkv, L, Dk = k_cache.shape
    if Bk != B or Dk != D:
        raise ValueError(f"cache shape {tuple(k_cache.shape)} does not match q {tuple(q.shape)}")
    if not seq_lens.is_cuda or seq_lens.dtype != torch.int32 or tuple(seq_lens.shape) != (B,):
        raise ValueError("seq_lens must be a CUDA int32 tensor of shape [B]")
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    n = fa_decode_num_splits(B, Hkv, L) if n_splits is None else int(n_splits)
    o = torch.empty_like(q) if out is None else out
    lse = torch.empty((B, Hq), device=q.device, dtype=torch.float32) if lse is None else lse
    need = fa_decode_workspace_size(B, Hq, n, D)
    if workspace is None:
        workspace = torch.empty(max(need, 1), device=q.device, dtype=torch.uint8)
    st = fa_decode(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), seq_lens.data_ptr(), o.data_ptr(),
                   lse.data_ptr(), B, Hq, Hkv, L, D, scale, _dt(q), n, workspace.data_ptr(), workspace.numel(),
                   _stream(stream))
    if st != FA_OK:
        raise FAError(st, "fa_decode")
    return o, lse


# ---- rotary positions and the paged cache
#
# A decode step is a few microseconds on the GPU, so its checks must not cost
# more: everything about a call that follows from the layout of its tensors
# (dtype, device, shape, strides) is checked and worked out once per layout.
# What is kept are sizes and strides: no tensor and no address.

_layouts: dict = {}


def _known(key, make, *args):
    got = _layouts.get(key)
    if got is None:
        if len(_layouts) >= 1024:
            _layouts.clear()
        got = _layouts[key] = make(*args)
    return got


def _c_int(x, what):
    """``x`` as the C entries take it: ctypes would cut it to 32 bits without a word."""
    x = int(x)
    if not -(1 << 31) <= x < 1 << 31:
        raise ValueError(f"{what} does not fit 32 bits: {x}")
    return x


def _sig(t):
    return None if t is None else (t.dtype, t.get_device(), t.shape, t.stride())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _same_device(first, *ts):
    """Every given tensor on ``first``'s CUDA device; returns its index."""
    if not first.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    for t in ts:
        if t is not None and t.device != first.device:
            raise ValueError(f"tensors must share one device: {t.device} != {first.device}")
    return first.get_device()


_torch = _current_device = _current_stream = None


def _bind():
    """torch's cheapest calls for the current device and stream (as numbers;
    the public ones take 0.2 and 1.2 us), with the public ones where this
    torch has no others."""
    global _torch, _current_device, _current_stream
    import torch
    _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    _current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda device: torch.cuda.current_stream(device).cuda_stream)
    _torch = torch


def _on(device, stream, call, *args):
    """``call(raw stream, *args)`` with ``device`` current, and on ``stream``
    if one is given, so that what is allocated inside belongs to the stream
    that the kernels run on."""
    if _lib is None:
        load_library()
    if _torch is None:
        _bind()
    if stream is None:
        if _current_device() == device:
            return call(_current_stream(device), *args)
        with _torch.cuda.device(device):
            return call(_current_stream(device), *args)
    cuda = _torch.cuda
    if not hasattr(stream, "cuda_stream"):
        raw = int(stream)
        stream = cuda.ExternalStream(raw, device=device) if raw else cuda.default_stream(device)
    if stream.device.index != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{device}")
    with cuda.device(device), cuda.stream(stream):
        return call(stream.cuda_stream, *args)


def _int32(t, what, shape=None):
    import torch
    if t.dtype != torch.int32 or not t.is_contiguous() or (shape is not None and t.shape != shape):
        raise ValueError(f"{what} must be a contiguous CUDA int32 tensor" + (f" of shape {list(shape)}" if shape else ""))


def _contiguous(shape):
    st, n = [], 1
    for s in reversed(shape):
        st.append(n)
        n *= max(s, 1)
    return tuple(reversed(st))


def _row_strides(shape, strides, dims, out=False):
    """The strides of ``dims`` (0 for dimensions of one element), rows contiguous."""
    if strides[-1] != 1:
        raise ValueError("rows must be contiguous in the last dimension")
    got = []
    for d in dims:
        s = strides[d] if shape[d] > 1 else 0
        if s % 8 or (out and s == 0 and shape[d] > 1):
            raise ValueError("strides must be multiples of 8 elements" + (" and not zero in an output" if out else ""))
        got.append(s)
    return got


def _rows_layout(x, y, order):
    """Of rows x and where they go, y (None: a new contiguous tensor): what
    fa_rows says behind the pointer, for both.  ``order``: the dimensions of
    batch (or None), heads and tokens."""
    if y is not None and (y.shape != x.shape or y.dtype != x.dtype):
        raise ValueError(f"output {tuple(y.shape)} {y.dtype} does not match {tuple(x.shape)} {x.dtype}")
    heads, said = x.shape[order[1]], []
    for st, out in ((x.stride(), False), (_contiguous(x.shape) if y is None else y.stride(), True)):
        s = _row_strides(x.shape, st, [d for d in order if d is not None], out)
        said.append((*(s if order[0] is not None else (0, *s)), heads))
    return said


def _refused(status, what, pairs, others=()):
    """Raise for a status that is not FA_OK, of a call with these (output,
    input) pairs.  The C entries decide whether outputs overlap anything (views
    of one buffer may lie between one another); where they refuse a call whose
    outputs reach into another tensor, say so."""
    def span(t):
        at = t.data_ptr()
        return at, at + t.element_size() * (1 + sum((n - 1) * k for n, k in zip(t.shape, t.stride())))
    if status == FA_ERR_INVALID_ARG:
        for i, (y, x) in enumerate(pairs):
            rest = [o for o, _ in pairs[:i]] + [z for j, (_, z) in enumerate(pairs) if j != i] + list(others)
            if y.data_ptr() != x.data_ptr() or y.stride() != x.stride():
                rest.append(x)
            for z in rest:
                (c, d), (e, f) = span(y), span(z)
                if y.numel() and z.numel() and c < f and e < d:
                    raise ValueError(f"{what}: an output overlaps another tensor of the call, other than its input in place")
    raise FAError(status, what)


def _check_freqs(freqs):
    import torch
    if freqs.dtype != torch.float64 or not freqs.is_contiguous() or freqs.dim() != 1:
        raise ValueError("freqs must be a contiguous CUDA float64 tensor of rot_dim / 2 radians per position")
    return 2 * freqs.shape[0]


def rope_freqs(rot_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
               original_len: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda"):
    """The frequencies of ``rope`` and ``append_paged``: a float64 tensor of
    rot_dim / 2 radians per position, and the factor ``amp`` to pass with it.
    ``scaling``: None, "linear" (positions divided by ``factor``), "ntk" (a
    larger base) or "yarn" (by parts; takes ``original_len``)."""
    import torch
    if scaling not in ROPE_SCALING:
        raise ValueError(f"scaling must be one of {list(ROPE_SCALING)}")
    rot_dim, original_len = _c_int(rot_dim, "rot_dim"), _c_int(original_len, "original_len")
    out = (ctypes.c_double * max(rot_dim // 2, 1))()
    amp = ctypes.c_float()
    st = fa_rope_freqs(rot_dim, float(base), ROPE_SCALING[scaling], float(factor), original_len, float(beta_fast),
                       float(beta_slow), out, ctypes.byref(amp))
    if st != FA_OK:
        raise FAError(st, "fa_rope_freqs")
    return torch.tensor(list(out), dtype=torch.float64).to(device), amp.value


def _rope_layout(q, k, freqs, positions, cu_seqlens, outs):
    import torch
    dev = _same_device(q, k, freqs, positions, cu_seqlens, *outs)
    packed = q.dim() == 3
    if not packed and q.dim() != 4:
        raise ValueError("q must be [B, H, S, D], or packed [H, T, D]")
    order = (None, 0, 1) if packed else (0, 1, 2)
    B, S = (1, q.shape[1]) if packed else (q.shape[0], q.shape[2])
    if k is not None and (k.dtype != q.dtype or k.dim() != q.dim() or
                          any(a != b for d, (a, b) in enumerate(zip(k.shape, q.shape)) if d != order[1])):
        raise ValueError(f"k {tuple(k.shape)} {k.dtype} does not match q {tuple(q.shape)} {q.dtype}")
    nseq = pos_stride = 0
    if cu_seqlens is not None:
        if not packed:
            raise ValueError("cu_seqlens goes with packed [H, T, D] tensors")
        _int32(cu_seqlens, "cu_seqlens")
        nseq = cu_seqlens.numel() - 1
        if nseq < 0:
            raise ValueError("cu_seqlens must hold at least one offset")
    if positions is not None:
        if positions.dtype != torch.int32 or positions.dim() not in (1, 2) or positions.shape[-1] != S or \
                (positions.dim() == 2 and positions.shape[0] not in (1, B)) or \
                (S > 1 and positions.stride(-1) != 1):
            raise ValueError(f"positions must be a CUDA int32 tensor of shape [{S}] or [{B}, {S}]")
        pos_stride = positions.stride(0) if positions.dim() == 2 and positions.shape[0] > 1 else 0
    elif packed and cu_seqlens is None:
        raise ValueError("packed tensors need cu_seqlens or positions")
    rows = [_rows_layout(x, y, order) for x, y in zip((q, k), outs) if x is not None]
    empty = q.numel() == 0 and (k is None or k.numel() == 0)
    return dev, _dt(q), _check_freqs(freqs), B, S, q.shape[-1], nseq, pos_stride, rows, empty


def _rope(q, k, freqs, positions, cu_seqlens, interleaved, amp, out, stream, backward):
    if out is None:
        q_out = k_out = None
    else:
        q_out, k_out = out if isinstance(out, (tuple, list)) else (out, None)
        if q_out is None or (k is None) != (k_out is None):
            raise ValueError("out must give a tensor for each input")
    known = _known(("rope", _sig(q), _sig(k), _sig(freqs), _sig(positions), _sig(cu_seqlens), _sig(q_out), _sig(k_out)),
                   _rope_layout, q, k, freqs, positions, cu_seqlens, (q_out, k_out))
    return _on(known[0], stream, _rope_call, known, q, k, freqs, positions, cu_seqlens, interleaved, amp, q_out, k_out,
               backward)


def _rope_call(raw, known, q, k, freqs, positions, cu_seqlens, interleaved, amp, yq, yk, backward):
    _, dt, rot, B, S, D, nseq, pos_stride, rows, empty = known
    given = yq is not None
    if not given:
        yq = _torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if k is not None:
            yk = _torch.empty(k.shape, dtype=k.dtype, device=k.device)
    xp, yp = q.data_ptr(), yq.data_ptr()
    x, y = _ROWS.pack(xp, *rows[0][0]), _ROWS.pack(yp, *rows[0][1])
    if k is not None:
        kp, ykp = k.data_ptr(), yk.data_ptr()
        x += _ROWS.pack(kp, *rows[1][0])
        y += _ROWS.pack(ykp, *rows[1][1])
    if not empty:
        call = _lib.fa_rope if given else _lib.fa_rope_fill
        st = call(x, y, len(rows), freqs.data_ptr(), rot, interleaved, amp, backward, _ptr(positions), pos_stride,
                  _ptr(cu_seqlens), nseq, B, S, D, dt, raw)
        if st != FA_OK:
            _refused(st, "fa_rope", [p for p in ((yq, q), (yk, k)) if given and p[0] is not None])
    return yq, yk


def rope(q, k, freqs, positions=None, cu_seqlens=None, interleaved: bool = False, amp: float = 1.0, out=None,
         stream=None):
    """q and k (or None) with rotary positions, in one launch: [B, H, S, D]
    tensors, or packed [H, T, D] ones with ``cu_seqlens``.  Inputs may be any
    views whose rows are contiguous (a transposed projection, say); the
    outputs are contiguous, or ``out`` = (q_out, k_out), which may be the
    inputs themselves but not overlap anything else of the call.  Rows behind
    the last sequence are zero in new outputs and left as they were in
    ``out``.  ``freqs`` and ``amp`` come from ``rope_freqs``; ``positions``
    (int32 [S] or [B, S]; packed [T]) defaults to the index in
    the sequence.  The columns past the rotated ones are copied."""
    return _rope(q, k, freqs, positions, cu_seqlens, interleaved, amp, out, stream, False)


def rope_backward(dq, dk, freqs, positions=None, cu_seqlens=None, interleaved: bool = False, amp: float = 1.0,
                  out=None, stream=None):
    """The gradients of ``rope``'s q and k from those of its outputs (as
    ``backward`` / ``backward_varlen`` return them); arguments as ``rope``."""
    return _rope(dq, dk, freqs, positions, cu_seqlens, interleaved, amp, out, stream, True)


def _pages_layout(k_pages, v_pages, block_table, B, dtype, D):
    """What fa_pages says of these tensors: (page stride, row stride of the
    table, n_pages, page_size, heads, max_pages)."""
    import torch
    if k_pages.dim() != 4 or k_pages.shape != v_pages.shape or k_pages.dtype != dtype or v_pages.dtype != dtype:
        raise ValueError("k_pages and v_pages must be [n_pages, Hkv, page_size, D] of the queries' dtype")
    n, heads, page, Dk = k_pages.shape
    if Dk != D:
        raise ValueError(f"pages of D = {Dk} do not match D = {D}")
    strides = []
    for x in (k_pages, v_pages):
        if n and not x[0].is_contiguous():
            raise ValueError("each page must be contiguous")
        strides.append(x.stride(0) if n > 1 else heads * page * D)
    if strides[0] != strides[1]:
        raise ValueError("k_pages and v_pages must have the same stride from page to page")
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] != B or \
            (block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError(f"block_table must be a CUDA int32 tensor of shape [{B}, max_pages]")
    return strides[0], block_table.stride(0) if B > 1 else 0, n, page, heads, block_table.shape[1]


def _pack_pages(k_pages, v_pages, block_table, layout):
    return _PAGES.pack(k_pages.data_ptr(), v_pages.data_ptr(), layout[0], block_table.data_ptr(), *layout[1:])


def _append_layout(k, v, k_pages, v_pages, block_table, seq_lens, cu_seqlens, q, freqs, positions, q_out):
    dev = _same_device(k, v, k_pages, v_pages, block_table, seq_lens, cu_seqlens, q, freqs, positions, q_out)
    dt = _dt(k)
    if k.dim() != 3 or k.shape != v.shape or v.dtype != k.dtype:
        raise ValueError("k and v must be equal in shape and dtype: [B, Hkv, D], or packed [Hkv, T, D]")
    one, D = cu_seqlens is None, k.shape[-1]
    order = (None, 1, 0) if one else (None, 0, 1)
    T = k.shape[order[2]]
    B = T if one else cu_seqlens.numel() - 1
    if B < 0:
        raise ValueError("cu_seqlens must hold at least one offset")
    pages = _pages_layout(k_pages, v_pages, block_table, B, k.dtype, D)
    if k.shape[order[1]] != pages[4]:
        raise ValueError(f"k has {k.shape[order[1]]} heads, the pages {pages[4]}")
    _int32(seq_lens, "seq_lens", (B,))
    if not one:
        _int32(cu_seqlens, "cu_seqlens")
    if positions is not None:
        _int32(positions, "positions", (T,))
    if q is None and q_out is not None:
        raise ValueError("q_out goes with q")
    q_rows = None
    if q is not None:
        if freqs is None:
            raise ValueError("q is only rotated: it takes freqs")
        if q.dim() != 3 or q.dtype != k.dtype or q.shape[order[2]] != T or q.shape[-1] != D:
            raise ValueError(f"q {tuple(q.shape)} {q.dtype} does not match k {tuple(k.shape)} {k.dtype}")
        q_rows = _rows_layout(q, q_out, order)
    k_rows, v_rows = ((0, *_row_strides(x.shape, x.stride(), order[1:]), x.shape[order[1]]) for x in (k, v))
    return dev, dt, B, T, D, pages, k_rows, v_rows, q_rows, 0 if freqs is None else _check_freqs(freqs)


def append_paged(k, v, k_pages, v_pages, block_table, seq_lens, cu_seqlens=None, q=None, freqs=None, positions=None,
                 interleaved: bool = False, amp: float = 1.0, q_out=None, stream=None):
    """Write new keys and values into the pages of their sequences, the keys
    (and the queries ``q`` of the same tokens) rotated on the way.

    A decode step gives k, v [B, Hkv, D] (q [B, Hq, D]), one token per
    sequence; with ``cu_seqlens`` they are packed [H, T, D].  ``seq_lens``
    (CUDA int32 [B]) are the lengths with the new tokens, as ``decode_paged``
    takes them next.  Without ``freqs`` nothing is rotated.  Returns the
    rotated q (``q_out``, which may be q) or None.  Tokens of a sequence of
    length 0 and tokens behind the last sequence write nothing (their rows of
    a new q are zero); a row past
    the table or a page outside the pool is reported by
    ``check_device_error``."""
    known = _known(
        ("append", _sig(k), _sig(v), _sig(k_pages), _sig(v_pages), _sig(block_table), _sig(seq_lens), _sig(cu_seqlens),
         _sig(q), _sig(freqs), _sig(positions), _sig(q_out)),
        _append_layout, k, v, k_pages, v_pages, block_table, seq_lens, cu_seqlens, q, freqs, positions, q_out)
    return _on(known[0], stream, _append_call, known, k, v, k_pages, v_pages, block_table, seq_lens, cu_seqlens, q,
               freqs, positions, interleaved, amp, q_out)


def _append_call(raw, known, k, v, k_pages, v_pages, block_table, seq_lens, cu_seqlens, q, freqs, positions,
                 interleaved, amp, q_out):
    _, dt, B, T, D, pages, k_rows, v_rows, q_rows, rot = known
    to, qx, qy = q_out, None, None
    if q is not None:
        if q_out is None:
            to = _torch.empty(q.shape, dtype=q.dtype, device=q.device)
        xp, yp = q.data_ptr(), to.data_ptr()
        qx, qy = _ROWS.pack(xp, *q_rows[0]), _ROWS.pack(yp, *q_rows[1])
    if T:
        call = _lib.fa_append_paged_fill if q_out is None else _lib.fa_append_paged
        st = call(_ROWS.pack(k.data_ptr(), *k_rows), _ROWS.pack(v.data_ptr(), *v_rows), qx, qy,
                  _pack_pages(k_pages, v_pages, block_table, pages), seq_lens.data_ptr(), _ptr(cu_seqlens), B, T,
                  _ptr(freqs), rot, interleaved, amp, _ptr(positions), D, dt, raw)
        if st != FA_OK:
            _refused(st, "fa_append_paged", [] if q_out is None else [(q_out, q)], (k, v, k_pages, v_pages))
    return to


def _decode_layout(q, k_pages, v_pages, block_table, seq_lens, prefix_len, prefix_table, out, lse, workspace):
    import torch
    dev = _same_device(q, k_pages, v_pages, block_table, seq_lens, prefix_table, out, lse, workspace)
    dt = _dt(q)
    if q.dim() != 3 or not q.is_contiguous():
        raise ValueError("q must be a contiguous [B, Hq, D] tensor")
    B, Hq, D = q.shape
    pages = _pages_layout(k_pages, v_pages, block_table, B, q.dtype, D)
    _int32(seq_lens, "seq_lens", (B,))
    if prefix_table is not None:
        _int32(prefix_table, "prefix_table")
        if prefix_table.dim() != 1 or prefix_table.shape[0] * pages[3] < prefix_len:
            raise ValueError(f"prefix_table must name the pages of {prefix_len} rows")
    if out is not None:
        _check((out,), q.shape)
        if out.dtype != q.dtype:
            raise TypeError("out must have q's dtype")
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != (B, Hq) or not lse.is_contiguous()):
        raise ValueError(f"lse must be a contiguous fp32 tensor of shape [{B}, {Hq}]")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    with torch.cuda.device(dev):  # the size is that of the device
        need = fa_decode_prefix_workspace_size(B, Hq, pages[4], prefix_len, D)
    size = need if workspace is None else workspace.numel() * workspace.element_size()
    return dev, dt, B, Hq, D, pages, need, size


def _decode_pages(q, k_pages, v_pages, block_table, seq_lens, prefix_len, prefix_table, scale, out, lse, workspace,
                  stream):
    known = _known(
        ("decode", _sig(q), _sig(k_pages), _sig(v_pages), _sig(block_table), _sig(seq_lens), prefix_len,
         _sig(prefix_table), _sig(out), _sig(lse), _sig(workspace)),
        _decode_layout, q, k_pages, v_pages, block_table, seq_lens, prefix_len, prefix_table, out, lse, workspace)
    return _on(known[0], stream, _decode_call, known, q, k_pages, v_pages, block_table, seq_lens, prefix_len,
               prefix_table, scale, out, lse, workspace)


def _decode_call(raw, known, q, k_pages, v_pages, block_table, seq_lens, prefix_len, prefix_table, scale, o, lse, ws):
    _, dt, B, Hq, D, pages, need, size = known
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if o is None:
        o = _torch.empty_like(q)
    if lse is None:
        lse = _torch.empty((B, Hq), device=q.device, dtype=_torch.float32)
    if ws is None:
        ws = _torch.empty(max(need, 1), device=q.device, dtype=_torch.uint8)
    at = _pack_pages(k_pages, v_pages, block_table, pages)
    if prefix_len:
        st = _lib.fa_decode_prefix(q.data_ptr(), at, seq_lens.data_ptr(), prefix_len, _ptr(prefix_table), o.data_ptr(),
                                   lse.data_ptr(), B, Hq, D, scale, dt, ws.data_ptr(), size, raw)
    else:
        st = _lib.fa_decode_paged(q.data_ptr(), at, seq_lens.data_ptr(), o.data_ptr(), lse.data_ptr(), B, Hq, D, scale,
                                  dt, ws.data_ptr(), size, raw)
    if st != FA_OK:
        raise FAError(st, "fa_decode_prefix" if prefix_len else "fa_decode_paged")
    return o, lse


def decode_paged(q, k_pages, v_pages, block_table, seq_lens, scale: float | None = None, out=None, lse=None,
                 workspace=None, stream=None):
    """One decode step over a paged cache: q [B, Hq, D] against pages
    [n_pages, Hkv, page_size, D] that ``block_table`` (CUDA int32
    [B, max_pages]) names, ``seq_lens`` (CUDA int32 [B]) rows of each
    sequence.  Returns O [B, Hq, D] and fp32 LSE [B, Hq]."""
    return _decode_pages(q, k_pages, v_pages, block_table, seq_lens, 0, None, scale, out, lse, workspace, stream)


def decode_prefix(q, k_pages, v_pages, block_table, seq_lens, prefix_len: int, prefix_table=None,
                  scale: float | None = None, out=None, lse=None, workspace=None, stream=None):
    """``decode_paged`` for sequences whose first ``prefix_len`` rows (a
    multiple of the page size) are the same pages: those named by
    ``prefix_table``, or by ``block_table`` for the first sequence that has
    them all (its other rows are not asked for them).  The shared rows
    are read once for the whole batch; a sequence shorter than ``prefix_len``
    sees those up to its length, whatever the others hold."""
    return _decode_pages(q, k_pages, v_pages, block_table, seq_lens, _c_int(prefix_len, "prefix_len"), prefix_table,
                         scale, out, lse, workspace, stream)


def check_device_error(stream=None):
    """Synchronise and raise FAError if a kernel recorded an error (a wait
    that timed out, split backward calls that disagreed on the mode, or a
    page table that named a page outside its pool)."""
    st = fa_check_device_error(_stream(stream))
    if st != FA_OK:
        raise FAError(st, "device")
