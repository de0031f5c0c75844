"""Index-selection sparse attention over a paged KV cache on GB300 (sm_103a): Python binding.

A thin ctypes layer over ``libdsa.so`` (C ABI in ``include/dsa.h``). It only marshals
arguments: torch tensors are passed as device pointers together with the current CUDA stream,
and every step of the computation runs in the library's kernels. There is no fallback: if the
library is missing or fails to load, :func:`lib` raises.

Entry points (same names as the C ABI):

* :func:`indexer_topk` -- lightning indexer + Top-K: ``idx[T][K]`` of the selected positions.
* :func:`sparse_attn` -- sparse attention over the rows ``idx`` selects.
* :func:`decode` -- both, fused on one stream, for one query row per sequence.
* :func:`cache_append` -- new tokens' indexer keys and latent rows into the paged caches (FP8 keys:
  block requantisation; FP8 latent rows: per-tile quantisation).
* :func:`indexer_prolog` -- the cache append and the MXFP8 query quantisation in one launch.
* :func:`rope`, :func:`rope_frequencies` -- rotary positions of queries, in place or into another tensor, and
  the frequencies of long contexts.
* :func:`cache_append_rope` -- the cache append of rows whose rotary columns are not turned yet.
* :func:`cache_read` -- ranges of the paged caches read back as dense, dequantised rows.
* :func:`prompt_attn` -- dense causal attention over packed prompts (grouped heads, prefixes).
* :func:`grouped_append`, :func:`grouped_attn`, :func:`grouped_evict` -- a paged cache of grouped heads in 8 bits:
  its append, decode attention over it (with the weight each position receives, if wanted), and eviction by it.
* :func:`block_summaries`, :func:`indexer_topk_hier` -- hierarchical (coarse -> fine) selection over
  per-block summary keys.
* :func:`indexer_topk_noalloc` -- :func:`indexer_topk` with the library's static scratch instead of
  a workspace, for callers that cannot allocate device memory.

Every tensor argument is a contiguous CUDA tensor in the layout ``include/dsa.h`` gives (:func:`rope`,
:func:`prompt_attn` and the new rows and queries of the grouped-head calls may be strided views); the calls are enqueued on the current stream (or
``stream=``). Nothing is recorded for autograd: :func:`rope`, :func:`cache_append_rope`, :func:`cache_read`,
:func:`prompt_attn` and the grouped-head calls refuse tensors that require gradients outside ``torch.no_grad()``, and
the caller's outputs of all but the appends count as changed in place (the paged caches, which belong to the library's
calls, do not).
A decode step over a batch of B sequences, bf16 everywhere, 64 indexer heads of 128, 128 heads over 576-wide latent
rows::

    dims = make_dims("bf16", B, max_blocks, num_blocks, H_I=64, d_I=128, H=128, d=576, d_v=512, K=2048)
    ws = workspace(dims, B)                      # sized for calls of B rows (the library checks it)
    idx, out, lse = decode(dims, q_I, w, k_I_cache, None, block_table, seq_lens, q, kv_cache,
                           576 ** -0.5, ws=ws)  # idx [B][K] int32, out [B][128][512] bf16
    assert read_error(ws) == 0                   # device-side fault bits (synchronises)
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch
from torch.autograd.graph import increment_version

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdsa.so")
_lib = None

MODES = {"f32": 0, "bf16": 1, "bf16_kfp8": 2, "mxfp8": 3}
STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "workspace", 4: "launch", 5: "device fault",
          6: "timeout", 7: "too large for the static scratch"}


class Dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("mode", "B", "max_blocks", "num_blocks", "block_size", "H_I", "d_I", "H", "d", "d_v", "K")]


class RopeTensor(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p), ("heads", ctypes.c_int32), ("layout", ctypes.c_int32)] + \
        [(n, ctypes.c_int64) for n in ("x_stride_t", "x_stride_h", "out_stride_t", "out_stride_h")]


_ROPE_TENSOR = struct.Struct("@PPiiqqqq")  # the same bytes, made faster


class RopeAppend(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rot", "k_offset", "k_layout", "kv_offset", "kv_layout")] + \
        [("scale", ctypes.c_float)]


class PromptDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("type", "B", "H", "H_kv", "d_qk", "d_v", "causal")] + \
        [(n, ctypes.c_int64) for n in ("q_stride_t", "q_stride_h", "k_stride_t", "k_stride_h", "v_stride_t", "v_stride_h")]


class GroupedDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("type", "B", "max_blocks", "num_blocks", "block_size", "H", "H_kv", "d_qk", "d_v")]


class DsaError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {lib().dsa_status_string(status).decode()} (status {status})")


def lib():
    """The loaded libdsa.so (built by ``__graft_entry__.build()``); raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m indexer_top_sparse_paged_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        D = ctypes.POINTER(Dims)
        L.dsa_workspace_size.restype = SZ
        L.dsa_workspace_size.argtypes = [D, I32]
        L.dsa_workspace_init.restype = ctypes.c_int
        L.dsa_workspace_init.argtypes = [P, SZ, P]
        L.dsa_indexer_topk.restype = ctypes.c_int
        L.dsa_indexer_topk.argtypes = [D, P, P, P, P, P, P, P, P, I32, P, P, SZ, P]
        L.dsa_sparse_attn.restype = ctypes.c_int
        L.dsa_sparse_attn.argtypes = [D, P, P, P, P, P, P, I32, ctypes.c_float, P, P, P, SZ, P]
        L.dsa_decode.restype = ctypes.c_int
        L.dsa_decode.argtypes = [D, P, P, P, P, P, P, P, P, ctypes.c_float, P, P, P, P, SZ, P]
        L.dsa_hier_workspace_size.restype = SZ
        L.dsa_hier_workspace_size.argtypes = [D, I32, I32]
        L.dsa_block_summaries.restype = ctypes.c_int
        L.dsa_block_summaries.argtypes = [D, P, P, P, P, P, P, SZ, P]
        L.dsa_block_summaries_append.restype = ctypes.c_int
        L.dsa_block_summaries_append.argtypes = [D, P, P, P, P, P, P, I32, P, P, SZ, P]
        L.dsa_indexer_topk_hier.restype = ctypes.c_int
        L.dsa_indexer_topk_hier.argtypes = [D, P, P, P, P, P, P, P, P, I32, P, I32, P, P, P, SZ, P]
        L.dsa_cache_append.restype = ctypes.c_int
        L.dsa_cache_append.argtypes = [D, P, P, P, P, P, P, I32, P, P, P, P, SZ, P]
        L.dsa_indexer_prolog.restype = ctypes.c_int
        L.dsa_indexer_prolog.argtypes = [D, P, P, P, P, P, P, I32, P, P, P, P, I32, P, P, SZ, P]
        F32, F64 = ctypes.c_float, ctypes.c_double
        L.dsa_rope_frequencies.restype = ctypes.c_int
        L.dsa_rope_frequencies.argtypes = [I32, F64, I32, F64, F64, F64, F64, ctypes.POINTER(F64)]
        L.dsa_rope.restype = ctypes.c_int
        L.dsa_rope.argtypes = [I32, P, I32, I32, P, P, P, I32, F32, I32, P]
        L.dsa_cache_append_rope.restype = ctypes.c_int
        L.dsa_cache_append_rope.argtypes = [D, ctypes.POINTER(RopeAppend), P, P, P, P, P, P, P, I32, P, P, P, P, SZ, P]
        L.dsa_cache_read.restype = ctypes.c_int
        L.dsa_cache_read.argtypes = [D, P, P, P, P, P, P, P, I32, P, P, P, SZ, P]
        PD = ctypes.POINTER(PromptDims)
        L.dsa_prompt_workspace_size.restype = SZ
        L.dsa_prompt_workspace_size.argtypes = [PD, I32]
        L.dsa_prompt_attn.restype = ctypes.c_int
        L.dsa_prompt_attn.argtypes = [PD, P, P, P, P, P, I32, I32, F32, P, P, P, SZ, P]
        GD, I64 = ctypes.POINTER(GroupedDims), ctypes.c_int64
        L.dsa_grouped_append.restype = ctypes.c_int
        L.dsa_grouped_append.argtypes = [GD, P, I64, I64, P, I64, I64, P, P, P, I32, P, P, P, P, P, SZ, P]
        L.dsa_grouped_workspace_size.restype = SZ
        L.dsa_grouped_workspace_size.argtypes = [GD, I32, I32]
        L.dsa_grouped_attn.restype = ctypes.c_int
        L.dsa_grouped_attn.argtypes = [GD, P, I64, I64, P, P, P, P, P, P, P, I32, F32, P, P, P, P, P, SZ, P]
        L.dsa_grouped_evict.restype = ctypes.c_int
        L.dsa_grouped_evict.argtypes = [GD, P, I32, I32, I32, P, P, P, I32, P, P, P, P, P, P, P, P, SZ, P]
        L.dsa_indexer_topk_noalloc.restype = ctypes.c_int
        L.dsa_indexer_topk_noalloc.argtypes = [D, P, P, P, P, P, P, P, P, I32, P, P, P]
        L.dsa_read_error.restype = ctypes.c_int
        L.dsa_read_error.argtypes = [P, ctypes.POINTER(I32), P]
        L.dsa_selftest_wait_timeout.restype = ctypes.c_int
        L.dsa_selftest_wait_timeout.argtypes = [P, SZ, P]
        L.dsa_last_launch_count.restype = I32
        L.dsa_last_launch_count.argtypes = []
        L.dsa_status_string.restype = ctypes.c_char_p
        L.dsa_status_string.argtypes = [ctypes.c_int]
        L.dsa_version.restype = I32
        L.dsa_version.argtypes = []
        _lib = L
    return _lib


KV_FP8 = 0x10  # DSA_KV_FP8: the latent cache holds FP8 records (e4m3 codes, one fp32 scale per 128 elements)
Q_MX_READY = 0x20  # DSA_Q_MX_READY: q_I already holds MXFP8 values (from indexer_prolog)


def kv_record_bytes(d: int) -> int:
    """DSA_KV_FP8_RECORD_BYTES(d): bytes of one FP8 latent record."""
    return (d + 4 * ((d + 127) // 128) + 15) // 16 * 16


def make_dims(mode: str, B: int, max_blocks: int, num_blocks: int, H_I: int, d_I: int, H: int, d: int, d_v: int,
              K: int, block_size: int = 64, kv: str = "act", q_ready: bool = False) -> Dims:
    """kv="fp8" sets DSA_KV_FP8 (the latent cache holds FP8 records); q_ready sets DSA_Q_MX_READY."""
    m = MODES[mode] if isinstance(mode, str) else int(mode)
    if q_ready:
        m |= Q_MX_READY
    if kv == "fp8":
        m |= KV_FP8
    elif kv != "act":
        raise ValueError(f"unknown latent-cache storage {kv!r}")
    return Dims(m, B, max_blocks, num_blocks, block_size, H_I, d_I, H, d, d_v, K)


def _p(t):
    """The device address of a tensor argument (None: NULL). The library reads and writes densely
    packed data through raw device pointers, so a strided view or a host tensor is refused here:
    passed on, it would be read with the wrong layout or dereferenced on the GPU as a bad address."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensor arguments must be contiguous (the library reads densely packed rows)")
    if not t.is_cuda:
        raise ValueError("tensor arguments must be CUDA tensors (the library takes device pointers)")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn: str, status: int):
    if status != 0:
        raise DsaError(fn, status)


def _check_out(dims: Dims, T: int, out, lse):
    """The output buffers the library writes must have its dtype and size (it takes raw pointers)."""
    odt = torch.float32 if dims.mode == MODES["f32"] else torch.bfloat16
    if out.dtype != odt or out.numel() < T * dims.H * dims.d_v or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {odt} tensor of T x H x d_v elements")
    if lse is not None and (lse.dtype != torch.float32 or lse.numel() < T * dims.H or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 tensor of T x H elements")


def _check_idx(dims: Dims, T: int, idx):
    if idx.dtype != torch.int32 or idx.numel() < T * dims.K or not idx.is_contiguous():
        raise ValueError("idx must be a contiguous int32 tensor of T x K elements")


def workspace_size(dims: Dims, T: int) -> int:
    return int(lib().dsa_workspace_size(ctypes.byref(dims), T))


def workspace(dims: Dims, T: int, device="cuda", stream=None) -> torch.Tensor:
    """Allocates (with torch) and initialises a workspace for calls with T query rows."""
    n = workspace_size(dims, T)
    if n == 0:
        raise ValueError("invalid dims")
    ws = torch.empty(n + 256, dtype=torch.uint8, device=device)
    off = (-ws.data_ptr()) % 256
    ws = ws[off: off + n]
    _check("dsa_workspace_init", lib().dsa_workspace_init(_p(ws), n, _stream(stream)))
    return ws


def indexer_topk(dims: Dims, q_I, w, k_I_cache, k_I_scale, block_table, seq_lens, q_seq=None, q_pos=None, *, ws,
                 idx=None, stream=None) -> torch.Tensor:
    """idx[T][K] int32: the Top-K causal positions of every query row (ascending, -1 padded)."""
    T = q_I.shape[0]
    if idx is None:
        idx = torch.empty((T, dims.K), dtype=torch.int32, device=q_I.device)
    _check_idx(dims, T, idx)
    st = lib().dsa_indexer_topk(ctypes.byref(dims), _p(q_I), _p(w), _p(k_I_cache), _p(k_I_scale), _p(block_table),
                                _p(seq_lens), _p(q_seq), _p(q_pos), T, _p(idx), _p(ws), ws.numel(), _stream(stream))
    _check("dsa_indexer_topk", st)
    return idx


def indexer_topk_noalloc(dims: Dims, q_I, w, k_I_cache, k_I_scale, block_table, seq_lens, q_seq=None, q_pos=None,
                         *, idx=None, fault_word=None, stream=None) -> torch.Tensor:
    """As :func:`indexer_topk`, without a workspace: the library's static scratch is used.

    ``fault_word`` (optional int32 device tensor of one element) receives the call's fault bits.
    Calls must be ordered on one stream (they share the scratch).
    """
    T = q_I.shape[0]
    if idx is None:
        idx = torch.empty((T, dims.K), dtype=torch.int32, device=q_I.device)
    _check_idx(dims, T, idx)
    st = lib().dsa_indexer_topk_noalloc(ctypes.byref(dims), _p(q_I), _p(w), _p(k_I_cache), _p(k_I_scale),
                                        _p(block_table), _p(seq_lens), _p(q_seq), _p(q_pos), T, _p(idx),
                                        _p(fault_word), _stream(stream))
    _check("dsa_indexer_topk_noalloc", st)
    return idx


def sparse_attn(dims: Dims, q, kv_cache, block_table, seq_lens, idx, sm_scale: float, q_seq=None, *, ws, out=None,
                lse=None, stream=None):
    """(out[T][H][d_v], lse[T][H]) of softmax attention over the rows idx selects."""
    T = q.shape[0]
    odt = torch.float32 if dims.mode == MODES["f32"] else torch.bfloat16
    if out is None:
        out = torch.empty((T, dims.H, dims.d_v), dtype=odt, device=q.device)
    if lse is None:
        lse = torch.empty((T, dims.H), dtype=torch.float32, device=q.device)
    _check_out(dims, T, out, lse)
    st = lib().dsa_sparse_attn(ctypes.byref(dims), _p(q), _p(kv_cache), _p(block_table), _p(seq_lens), _p(q_seq),
                               _p(idx), T, float(sm_scale), _p(out), _p(lse), _p(ws), ws.numel(), _stream(stream))
    _check("dsa_sparse_attn", st)
    return out, lse


def decode(dims: Dims, q_I, w, k_I_cache, k_I_scale, block_table, seq_lens, q, kv_cache, sm_scale: float, *, ws,
           idx=None, out=None, lse=None, want_idx: bool = True, stream=None):
    """Fused decode step (one query row per sequence): (idx or None, out, lse)."""
    T = dims.B
    odt = torch.float32 if dims.mode == MODES["f32"] else torch.bfloat16
    if idx is None and want_idx:
        idx = torch.empty((T, dims.K), dtype=torch.int32, device=q.device)
    if out is None:
        out = torch.empty((T, dims.H, dims.d_v), dtype=odt, device=q.device)
    if lse is None:
        lse = torch.empty((T, dims.H), dtype=torch.float32, device=q.device)
    _check_out(dims, T, out, lse)
    if idx is not None and (idx.dtype != torch.int32 or idx.numel() < T * dims.K or not idx.is_contiguous()):
        raise ValueError("idx must be a contiguous int32 tensor of T x K elements")
    st = lib().dsa_decode(ctypes.byref(dims), _p(q_I), _p(w), _p(k_I_cache), _p(k_I_scale), _p(block_table),
                          _p(seq_lens), _p(q), _p(kv_cache), float(sm_scale), _p(idx), _p(out), _p(lse), _p(ws),
                          ws.numel(), _stream(stream))
    _check("dsa_decode", st)
    return idx, out, lse


def cache_append(dims: Dims, k_I_new, kv_new, block_table, seq_lens, k_I_cache, k_I_scale, kv_cache, q_seq=None,
                 q_pos=None, *, ws, stream=None) -> None:
    """Writes new tokens (rows of k_I_new / kv_new) into the paged caches in place."""
    T = kv_new.shape[0]
    st = lib().dsa_cache_append(ctypes.byref(dims), _p(k_I_new), _p(kv_new), _p(block_table), _p(seq_lens), _p(q_seq),
                                _p(q_pos), T, _p(k_I_cache), _p(k_I_scale), _p(kv_cache), _p(ws), ws.numel(),
                                _stream(stream))
    _check("dsa_cache_append", st)


def indexer_prolog(dims: Dims, k_I_new, kv_new, block_table, seq_lens, k_I_cache, k_I_scale, kv_cache, q_I=None,
                   q_seq=None, q_pos=None, *, ws, q_out=None, stream=None):
    """One launch: the cache append of the new tokens (as cache_append) and, when q_I is given
    (DSA_MXFP8), its MXFP8 quantisation into q_out (returned; bf16, q_I's shape)."""
    T_new = 0 if kv_new is None else kv_new.shape[0]
    T_q = 0
    if q_I is not None:
        T_q = q_I.shape[0]
        if q_out is None:
            q_out = torch.empty_like(q_I)
        if q_out.dtype != torch.bfloat16 or q_out.numel() < q_I.numel() or not q_out.is_contiguous():
            raise ValueError("q_out must be a contiguous bf16 tensor of q_I's size")
    st = lib().dsa_indexer_prolog(ctypes.byref(dims), _p(k_I_new), _p(kv_new), _p(block_table), _p(seq_lens),
                                  _p(q_seq), _p(q_pos), T_new, _p(k_I_cache), _p(k_I_scale), _p(kv_cache), _p(q_I), T_q,
                                  _p(q_out), _p(ws), ws.numel(), _stream(stream))
    _check("dsa_indexer_prolog", st)
    return q_out


ROPE_LAYOUTS = {"interleaved": 0, "half": 1}
ROPE_SCALINGS = {"linear": 0, "base": 1, "yarn": 2}
_TYPES = {torch.float32: 0, torch.bfloat16: 1}


_F32, _I32, _U8 = torch.float32, torch.int32, torch.uint8


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _device(*tensors) -> int:
    """The current CUDA device's index, on which the library launches; every tensor must be there. Nothing is
    recorded for autograd, so a tensor whose gradient would get lost is refused."""
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                raise ValueError("tensor arguments must not record gradients (none would arrive: call under torch.no_grad(), "
                                 "or from an autograd.Function)")
    dev = None
    for t in tensors:
        if t is not None:
            d = t.get_device()
            if d != dev:
                _need(d >= 0, "tensor arguments must be CUDA tensors (the library takes device pointers)")
                _need(dev is None, "tensor arguments must be on one CUDA device")
                dev = d
    _need(dev == torch.cuda.current_device(), "tensor arguments must be on the current CUDA device")
    return dev


def _at(t):
    """The address of a contiguous tensor whose device has been checked (None: NULL)."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensor arguments must be contiguous (the library reads densely packed rows)")
    return t.data_ptr()


def _raw_stream(dev: int, stream):
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _int32(t, n: int, name: str):
    if t is not None and (t.dtype is not torch.int32 or t.numel() < n):
        raise ValueError(f"{name} must be an int32 tensor of {n} elements")


def _empty(shape, dtype, device, stream):
    """A new output that belongs to the stream the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _layout(name) -> int:
    _need(name in ROPE_LAYOUTS, f"unknown rotary layout {name!r}")
    return ROPE_LAYOUTS[name]


def rope_frequencies(rot: int, base: float = 10000.0, *, scaling: str = "linear", factor: float = 1.0,
                     original_length: float = 4096.0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                     device="cuda") -> torch.Tensor:
    """The rot / 2 angular frequencies (radians per position, float64) :func:`rope` takes, for contexts
    ``factor`` times the trained length: "linear", "base" or "yarn" (factor 1: unscaled)."""
    _need(scaling in ROPE_SCALINGS, f"unknown rotary scaling {scaling!r}")
    f = (ctypes.c_double * max(1, rot // 2))()
    _check("dsa_rope_frequencies", lib().dsa_rope_frequencies(rot, base, ROPE_SCALINGS[scaling], factor, original_length,
                                                              beta_fast, beta_slow, f))
    return torch.tensor(list(f), dtype=torch.float64, device=device)


def rope(x, freq, seq_lens=None, q_pos=None, *, layout="interleaved", out=None, scale: float = 1.0,
         transpose: bool = False, stream=None):
    """Turns the columns of ``x`` ([T][heads][rot], fp32 or bf16; rot = 2 freq.numel()) by the rows'
    positions ``q_pos`` (or seq_lens - 1), in place or into ``out``, and returns the result.

    ``x`` may be a view of part of wider heads (``q[..., 512:]``), or a list of up to four tensors of the
    same tokens, with ``out`` and ``layout`` lists as well. ``transpose=True`` is the backward pass, for an
    autograd.Function of the caller's: nothing is recorded here, and tensors that record gradients are refused."""
    many = isinstance(x, (list, tuple))
    xs = x if many else (x,)
    outs = xs if out is None else out if many else (out,)
    n = len(xs)
    layouts = layout if isinstance(layout, (list, tuple)) else (layout,) * n
    if not 0 < n == len(outs) == len(layouts):
        raise ValueError("x, out and layout must have the same number of tensors")
    dev = _device(freq, seq_lens, q_pos, *xs) if out is None else _device(freq, seq_lens, q_pos, *xs, *outs)
    if freq.dtype is not torch.float64 or freq.dim() != 1:
        raise ValueError("freq must be a float64 tensor of rot / 2 elements")
    dt, T, rot = xs[0].dtype, xs[0].shape[0], 2 * freq.shape[0]
    if dt not in _TYPES:
        raise ValueError("x must be float32 or bfloat16")
    if q_pos is None:
        _need(seq_lens is not None, "rope needs q_pos or seq_lens")
        _int32(seq_lens, T, "seq_lens")
    else:
        _int32(q_pos, T, "q_pos")
    arr = b""  # dsa_rope_tensor [n]
    for i in range(n):
        s, d = xs[i], outs[i]
        shape, st = s.shape, s.stride()
        if len(shape) != 3 or shape[0] != T or shape[2] != rot or s.dtype is not dt:
            raise ValueError("rope tensors must be [T][heads][rot] of one type and one T")
        if d is s:
            so = st
        else:
            so = d.stride()
            if d.shape != shape or d.dtype is not dt:
                raise ValueError("out must have x's shape and type")
        H = shape[1]
        if T and H:
            if st[2] != 1 or so[2] != 1:
                raise ValueError("a head's rotated columns must be dense")
            if (T > 1 and so[0] == 0) or (H > 1 and so[1] == 0):
                raise ValueError("out must not repeat rows (expanded views)")
        arr += _ROPE_TENSOR.pack(s.data_ptr(), d.data_ptr(), H, _layout(layouts[i]), st[0], st[1], so[0], so[1])
    st = lib().dsa_rope(_TYPES[dt], arr, n, rot, _at(freq), _at(seq_lens), _at(q_pos), T, scale, transpose,
                        _raw_stream(dev, stream))
    if st:
        _check("dsa_rope", st)
    increment_version(outs)  # a backward pass that kept what was here fails, and does not go on with the new values
    return outs if many else outs[0]


def cache_append_rope(dims: Dims, freq, k_I_new, kv_new, block_table, seq_lens, k_I_cache, k_I_scale, kv_cache,
                      q_seq=None, q_pos=None, *, k_offset=0, k_layout="half", kv_offset=None, kv_layout="interleaved",
                      scale: float = 1.0, ws, stream=None) -> None:
    """:func:`cache_append` of rows whose rotary columns are not turned yet: ``rot`` = 2 freq.numel()
    columns from ``k_offset`` of the indexer keys and from ``kv_offset`` of the latent rows (default: their
    last columns; -1: none) turn by the rows' positions in the same launch."""
    T, rot = kv_new.shape[0], 2 * freq.numel()
    dev = _device(freq, k_I_new, kv_new, block_table, seq_lens, k_I_cache, k_I_scale, kv_cache, q_seq, q_pos, ws)
    if freq.dtype is not torch.float64:
        raise ValueError("freq must be a float64 tensor of rot / 2 elements")
    act = torch.float32 if dims.mode == 0 else torch.bfloat16
    if k_I_new.dtype is not act or k_I_new.numel() != T * dims.d_I:
        raise ValueError(f"k_I_new must be a {act} tensor of T x d_I elements")
    if kv_new.dtype is not act or kv_new.numel() != T * dims.d:
        raise ValueError(f"kv_new must be a {act} tensor of T x d elements")
    _int32(block_table, dims.B * dims.max_blocks, "block_table")
    _int32(seq_lens, dims.B, "seq_lens")
    _int32(q_seq, T, "q_seq")
    _int32(q_pos, T, "q_pos")
    r = RopeAppend(rot, k_offset, _layout(k_layout), dims.d - rot if kv_offset is None else kv_offset, _layout(kv_layout),
                   float(scale))
    st = lib().dsa_cache_append_rope(ctypes.byref(dims), ctypes.byref(r), _at(freq), _at(k_I_new), _at(kv_new),
                                     _at(block_table), _at(seq_lens), _at(q_seq), _at(q_pos), T, _at(k_I_cache),
                                     _at(k_I_scale), _at(kv_cache), _at(ws), ws.numel(), _raw_stream(dev, stream))
    if st:
        _check("dsa_cache_append_rope", st)


def cache_read(dims: Dims, k_I_cache, k_I_scale, kv_cache, block_table, seq_lens, cu_rows, R: int, start=None, *,
               k_out=None, kv_out=None, want_k: bool = True, want_kv: bool = True, ws, stream=None):
    """(k[R][d_I], kv[R][d]) of the positions start[b], start[b] + 1, ... of every sequence b, dequantised,
    in rows cu_rows[b] .. cu_rows[b + 1] - 1 (fp32 or bf16). An output not wanted is None."""
    dev = _device(k_I_cache, k_I_scale, kv_cache, block_table, seq_lens, cu_rows, start, k_out, kv_out, ws)
    act = torch.float32 if dims.mode == 0 else torch.bfloat16
    if k_out is None and want_k:
        k_out = _empty((R, dims.d_I), act, ws.device, stream)
    if kv_out is None and want_kv:
        kv_out = _empty((R, dims.d), act, ws.device, stream)
    for t, d, name in ((k_out, dims.d_I, "k_out"), (kv_out, dims.d, "kv_out")):
        if t is not None and (t.dtype is not act or t.numel() < R * d):
            raise ValueError(f"{name} must be a {act} tensor of R x {d} elements")
    _int32(block_table, dims.B * dims.max_blocks, "block_table")
    _int32(seq_lens, dims.B, "seq_lens")
    _int32(cu_rows, dims.B + 1, "cu_rows")
    _int32(start, dims.B, "start")
    st = lib().dsa_cache_read(ctypes.byref(dims), _at(k_I_cache), _at(k_I_scale), _at(kv_cache), _at(block_table),
                              _at(seq_lens), _at(start), _at(cu_rows), R, _at(k_out), _at(kv_out), _at(ws), ws.numel(),
                              _raw_stream(dev, stream))
    if st:
        _check("dsa_cache_read", st)
    increment_version([t for t in (k_out, kv_out) if t is not None])
    return k_out, kv_out


def prompt_dims(q, k, v, B: int, causal: bool = True) -> PromptDims:
    """The dims of :func:`prompt_attn` for B sequences packed in q [Tq][H][d_qk], k [Tk][H_kv][d_qk] and
    v [Tk][H_kv][d_v] (strided views allowed; a head's columns are dense)."""
    return PromptDims(*_prompt_fields(q, k, v, B, causal))


_PROMPT_DIMS = struct.Struct("@7i4x6q")  # dsa_prompt_dims


def _prompt_fields(q, k, v, B, causal):
    qn, kn, vn, qs, ks, vs, dt = q.shape, k.shape, v.shape, q.stride(), k.stride(), v.stride(), q.dtype
    if not len(qn) == len(kn) == len(vn) == 3 or (qs[2] != 1 and q.numel()) or (ks[2] != 1 and k.numel()) or (vs[2] != 1 and v.numel()):
        raise ValueError("q, k and v must be [tokens][heads][width] with dense columns")
    if dt not in _TYPES or k.dtype is not dt or v.dtype is not dt:
        raise ValueError("q, k and v must be all float32 or all bfloat16")
    if kn[:2] != vn[:2] or qn[2] != kn[2]:
        raise ValueError("k and v must have the same tokens and heads, q and k the same width")
    return (_TYPES[dt], B, qn[1], kn[1], qn[2], vn[2], int(causal), qs[0], qs[1], ks[0], ks[1], vs[0], vs[1])


def prompt_workspace(dims: PromptDims, Tq: int, device="cuda", stream=None) -> torch.Tensor:
    """Allocates and initialises a workspace for :func:`prompt_attn` calls of up to Tq query tokens."""
    n = int(lib().dsa_prompt_workspace_size(ctypes.byref(dims), Tq))
    if n == 0:
        raise ValueError("invalid dims")
    ws = _empty(n + 256, torch.uint8, device, stream)
    off = (-ws.data_ptr()) % 256
    ws = ws[off: off + n]
    _check("dsa_workspace_init", lib().dsa_workspace_init(_p(ws), n, _stream(stream)))
    return ws


def prompt_attn(dims: PromptDims, q, k, v, cu_q, cu_k, sm_scale: float, *, ws, out=None, lse=None, stream=None):
    """(out[Tq][H][d_v], lse[Tq][H]) of dense attention over packed sequences: sequence b has the queries
    cu_q[b] .. cu_q[b + 1] - 1, the last of its positions, and the keys cu_k[b] .. cu_k[b + 1] - 1."""
    if bytes(dims) != _PROMPT_DIMS.pack(*_prompt_fields(q, k, v, dims.B, dims.causal)):
        raise ValueError("q, k and v differ from the tensors dims was made for")
    dev = _device(q, k, v, cu_q, cu_k, out, lse, ws)
    _int32(cu_q, dims.B + 1, "cu_q")
    _int32(cu_k, dims.B + 1, "cu_k")
    Tq, H = q.shape[:2]
    if out is None:
        out = _empty((Tq, H, dims.d_v), q.dtype, q.device, stream)
    elif out.dtype is not q.dtype or out.numel() < Tq * H * dims.d_v:
        raise ValueError("out must be a tensor of Tq x H x d_v elements in q's type")
    if lse is None:
        lse = _empty((Tq, H), torch.float32, q.device, stream)
    elif lse.dtype is not torch.float32 or lse.numel() < Tq * H:
        raise ValueError("lse must be a float32 tensor of Tq x H elements")
    st = lib().dsa_prompt_attn(ctypes.byref(dims), q.data_ptr(), k.data_ptr(), v.data_ptr(), _at(cu_q), _at(cu_k), Tq,
                               k.shape[0], sm_scale, _at(out), _at(lse), _at(ws), ws.numel(), _raw_stream(dev, stream))
    if st:
        _check("dsa_prompt_attn", st)
    increment_version((out, lse))
    return out, lse


def grouped_dims(type: str, B: int, max_blocks: int, num_blocks: int, H: int, H_kv: int, d_qk: int, d_v: int,
                 block_size: int = 64) -> GroupedDims:
    """The dims of the grouped-head calls: ``type`` ("f32" or "bf16") is that of q, out and the new keys and values."""
    _need(type in ("f32", "bf16"), f"unknown type {type!r}")
    return GroupedDims(MODES[type], B, max_blocks, num_blocks, block_size, H, H_kv, d_qk, d_v)


def grouped_workspace(dims: GroupedDims, T: int, weights: bool = False, device="cuda", stream=None) -> torch.Tensor:
    """Allocates and initialises a workspace for the grouped-head calls of up to T query tokens (``weights``:
    :func:`grouped_attn` with weights_out as well)."""
    n = int(lib().dsa_grouped_workspace_size(ctypes.byref(dims), T, weights))
    if n == 0:
        raise ValueError("invalid dims")
    ws = _empty(n + 256, torch.uint8, device, stream)
    off = (-ws.data_ptr()) % 256
    ws = ws[off: off + n]
    _check("dsa_workspace_init", lib().dsa_workspace_init(_p(ws), n, _stream(stream)))
    return ws


def _grouped_rows(x, T: int, heads: int, width: int, dims: GroupedDims, name: str):
    """Address and strides of [T][heads][width] rows, which may be a strided view."""
    t, shape, st = torch.bfloat16 if dims.type else torch.float32, x.shape, x.stride()
    if x.dtype is not t or len(shape) != 3 or shape[0] != T or shape[1] != heads or shape[2] != width:
        raise ValueError(f"{name} must be a {t} tensor of [{T}][{heads}][{width}]")
    if st[2] != 1 and T:
        raise ValueError(f"a head's columns of {name} must be dense")
    return x.data_ptr(), st[0], st[1]


def _grouped_caches(dims: GroupedDims, k_cache, k_scale, v_cache, v_scale, block_table, seq_lens, cu, T: int):
    rows = dims.num_blocks * dims.H_kv
    for t, n, name in ((k_cache, rows * 64 * dims.d_qk, "k_cache"), (v_cache, rows * 64 * dims.d_v, "v_cache")):
        if t.element_size() != 1 or t.numel() < n:
            raise ValueError(f"{name} must be a tensor of {n} bytes")
    for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if t.dtype is not torch.float32 or t.numel() < rows:
            raise ValueError(f"{name} must be a float32 tensor of num_blocks x H_kv elements")
    _int32(block_table, dims.B * dims.max_blocks, "block_table")
    _int32(seq_lens, dims.B, "seq_lens")
    _int32(cu, dims.B + 1, "cu")
    if cu is None and T >= 0:
        _need(T == dims.B, "without cu there is one row for each sequence")


def _row_width(t, n: int, total: int, name: str):
    """A tensor of more than one dimension and more elements than the call needs has them in further rows, not in longer ones:
    its last dimensions make up rows of n elements."""
    if t.numel() == total or t.dim() < 2:
        return
    p = 1
    for s in reversed(t.shape):
        p *= s
        if p >= n:
            break
    if p != n:
        raise ValueError(f"rows of {name} must have {n} elements")


def _fp32(t, n: int, name: str):
    if t.dtype is not torch.float32 or t.numel() < n:
        raise ValueError(f"{name} must be a float32 tensor of {n} elements")


def _all_fit(wanted, dev: int):
    """The addresses of tensors that all are as they should be -- (tensor, type, elements) -- or None: the checks one by
    one, which take longer, then say what is wrong."""
    grad = torch.is_grad_enabled()
    at = []
    for t, dtype, n in wanted:
        if t.dtype is not dtype or t.numel() < n or t.get_device() != dev or not t.is_contiguous() or (grad and t.requires_grad):
            return None
        at.append(t.data_ptr())
    return at


def grouped_append(dims: GroupedDims, k_new, v_new, block_table, seq_lens, k_cache, k_scale, v_cache, v_scale, cu=None, *,
                   ws, stream=None) -> None:
    """Writes new tokens (k_new[T][H_kv][d_qk], v_new[T][H_kv][d_v], strided views allowed) into the caches as e4m3 codes
    with one scale per block and head: rows cu[b] .. cu[b + 1] - 1 are the last of sequence b's seq_lens[b] positions."""
    T = k_new.shape[0]
    dev = _device(k_new, v_new, cu)
    k = _grouped_rows(k_new, T, dims.H_kv, dims.d_qk, dims, "k_new")
    v = _grouped_rows(v_new, T, dims.H_kv, dims.d_v, dims, "v_new")
    rows = dims.num_blocks * dims.H_kv
    at = _all_fit(((block_table, _I32, dims.B * dims.max_blocks), (seq_lens, _I32, dims.B), (k_cache, _U8, 64 * rows * dims.d_qk),
                   (k_scale, _F32, rows), (v_cache, _U8, 64 * rows * dims.d_v), (v_scale, _F32, rows), (ws, _U8, 0)), dev)
    if at is None or (T != dims.B if cu is None else cu.dtype is not _I32 or cu.numel() <= dims.B):
        _device(k_new, v_new, block_table, seq_lens, k_cache, k_scale, v_cache, v_scale, cu, ws)
        _grouped_caches(dims, k_cache, k_scale, v_cache, v_scale, block_table, seq_lens, cu, T)
        at = [_at(t) for t in (block_table, seq_lens, k_cache, k_scale, v_cache, v_scale, ws)]
    _row_width(block_table, dims.max_blocks, dims.B * dims.max_blocks, "block_table")
    st = lib().dsa_grouped_append(dims, *k, *v, at[0], at[1], _at(cu), T, at[2], at[3], at[4], at[5], at[6], ws.numel(),
                                  _raw_stream(dev, stream))
    if st:
        _check("dsa_grouped_append", st)


def grouped_attn(dims: GroupedDims, q, k_cache, k_scale, v_cache, v_scale, block_table, seq_lens, sm_scale: float, cu=None,
                 *, weights=None, weights_out=None, ws, out=None, lse=None, stream=None):
    """(out[T][H][d_v], lse[T][H]) of attention over the cached positions: queries cu[b] .. cu[b + 1] - 1 (default: one for
    each sequence) are the last of sequence b's positions, and each sees those up to its own.

    ``weights_out`` ([B][H_kv][max_blocks * 64] fp32; default: ``weights`` itself, in place) receives ``weights`` plus the
    attention weight of every position, summed over the sequence's queries and the heads of its group."""
    T = q.shape[0]
    if weights_out is None:
        weights_out = weights
    dev = _device(q, cu, weights, weights_out, out, lse)
    row = _grouped_rows(q, T, dims.H, dims.d_qk, dims, "q")
    rows = dims.num_blocks * dims.H_kv
    at = _all_fit(((k_cache, _U8, 64 * rows * dims.d_qk), (k_scale, _F32, rows), (v_cache, _U8, 64 * rows * dims.d_v),
                   (v_scale, _F32, rows), (block_table, _I32, dims.B * dims.max_blocks), (seq_lens, _I32, dims.B), (ws, _U8, 0)), dev)
    if at is None or (T != dims.B if cu is None else cu.dtype is not _I32 or cu.numel() <= dims.B):
        _device(q, k_cache, k_scale, v_cache, v_scale, block_table, seq_lens, cu, ws)
        _grouped_caches(dims, k_cache, k_scale, v_cache, v_scale, block_table, seq_lens, cu, T)
        at = [_at(t) for t in (k_cache, k_scale, v_cache, v_scale, block_table, seq_lens, ws)]
    _row_width(block_table, dims.max_blocks, dims.B * dims.max_blocks, "block_table")
    for t, name in ((weights, "weights"), (weights_out, "weights_out")):
        if t is not None:
            n = dims.max_blocks * 64
            _fp32(t, dims.B * dims.H_kv * n, name)
            _row_width(t, n, dims.B * dims.H_kv * n, name)
    if out is None:
        out = _empty((T, dims.H, dims.d_v), q.dtype, q.device, stream)
    elif out.dtype is not q.dtype or out.numel() < T * dims.H * dims.d_v:
        raise ValueError("out must be a tensor of T x H x d_v elements in q's type")
    if lse is None:
        lse = _empty((T, dims.H), torch.float32, q.device, stream)
    else:
        _fp32(lse, T * dims.H, "lse")
    st = lib().dsa_grouped_attn(dims, *row, at[0], at[1], at[2], at[3], at[4], at[5], _at(cu), T, sm_scale, _at(out), _at(lse),
                                _at(weights), _at(weights_out), at[6], ws.numel(), _raw_stream(dev, stream))
    if st:
        _check("dsa_grouped_attn", st)
    increment_version((out, lse) if weights_out is None else (out, lse, weights_out))
    return out, lse


def grouped_evict(dims: GroupedDims, weights, keep: int, block_table, seq_lens, new_table, k_cache, k_scale, v_cache, v_scale,
                  *, sink: int = 0, recent: int = 0, ws, kept=None, new_lens=None, weights_out=None, stream=None):
    """(kept[B][H_kv][keep], new_lens[B], weights_out[B][H_kv][blocks * 64]): every sequence cut to ``keep`` positions for each
    key head -- the first ``sink``, the last ``recent`` and the heaviest of the rest by ``weights`` -- and the kept rows
    copied into the blocks of ``new_table`` ([B][blocks]), requantised. Go on with new_table (dims of its width), new_lens as
    seq_lens, and weights_out; rotate later queries and keys at their own positions (``rope(..., q_pos=)``), not by new_lens."""
    _need(new_table.dim() == 2 and new_table.shape[0] == dims.B, "new_table must be [B][blocks]")
    dev = _device(weights, block_table, seq_lens, new_table, k_cache, k_scale, v_cache, v_scale, ws, kept, new_lens, weights_out)
    _grouped_caches(dims, k_cache, k_scale, v_cache, v_scale, block_table, seq_lens, None, -1)
    _int32(new_table, 0, "new_table")
    heads = dims.B * dims.H_kv
    _fp32(weights, heads * dims.max_blocks * 64, "weights")
    _row_width(block_table, dims.max_blocks, dims.B * dims.max_blocks, "block_table")
    _row_width(weights, dims.max_blocks * 64, heads * dims.max_blocks * 64, "weights")
    blocks = new_table.shape[1]
    if kept is None:
        kept = _empty((dims.B, dims.H_kv, max(0, keep)), torch.int32, ws.device, stream)
    else:
        _int32(kept, heads * keep, "kept")
        _row_width(kept, keep, heads * keep, "kept")
    if new_lens is None:
        new_lens = _empty((dims.B,), torch.int32, ws.device, stream)
    _int32(new_lens, dims.B, "new_lens")
    if weights_out is None:
        weights_out = _empty((dims.B, dims.H_kv, blocks * 64), torch.float32, ws.device, stream)
    else:
        _fp32(weights_out, heads * blocks * 64, "weights_out")
        _row_width(weights_out, blocks * 64, heads * blocks * 64, "weights_out")
    st = lib().dsa_grouped_evict(dims, _at(weights), keep, sink, recent, _at(block_table), _at(seq_lens), _at(new_table), blocks,
                                 _at(k_cache), _at(k_scale), _at(v_cache), _at(v_scale), _at(kept), _at(new_lens),
                                 _at(weights_out), _at(ws), ws.numel(), _raw_stream(dev, stream))
    if st:
        _check("dsa_grouped_evict", st)
    increment_version((kept, new_lens, weights_out))
    return kept, new_lens, weights_out


def summaries_buffer(dims: Dims, device="cuda") -> torch.Tensor:
    """A bf16 [B][pages * 64][d_I] tensor for dsa_block_summaries (pages = ceil(max_blocks / 64))."""
    pages = (dims.max_blocks + 63) // 64
    return torch.zeros((dims.B, pages * 64, dims.d_I), dtype=torch.bfloat16, device=device)


def block_summaries(dims: Dims, k_I_cache, k_I_scale, block_table, seq_lens, summaries, *, ws, stream=None) -> None:
    """Writes the mean key of every valid 64-token block into ``summaries``."""
    st = lib().dsa_block_summaries(ctypes.byref(dims), _p(k_I_cache), _p(k_I_scale), _p(block_table), _p(seq_lens),
                                   _p(summaries), _p(ws), ws.numel(), _stream(stream))
    _check("dsa_block_summaries", st)


def block_summaries_append(dims: Dims, k_I_cache, k_I_scale, block_table, seq_lens, T: int, summaries, q_seq=None,
                           q_pos=None, *, ws, stream=None) -> None:
    """Recomputes the summaries of the blocks that T appended tokens touched."""
    st = lib().dsa_block_summaries_append(ctypes.byref(dims), _p(k_I_cache), _p(k_I_scale), _p(block_table),
                                          _p(seq_lens), _p(q_seq), _p(q_pos), T, _p(summaries), _p(ws), ws.numel(),
                                          _stream(stream))
    _check("dsa_block_summaries_append", st)


def hier_workspace(dims: Dims, T: int, n_sel: int, device="cuda", stream=None) -> torch.Tensor:
    n = int(lib().dsa_hier_workspace_size(ctypes.byref(dims), T, n_sel))
    if n == 0:
        raise ValueError("invalid dims")
    ws = torch.empty(n + 256, dtype=torch.uint8, device=device)
    off = (-ws.data_ptr()) % 256
    ws = ws[off: off + n]
    _check("dsa_workspace_init", lib().dsa_workspace_init(_p(ws), n, _stream(stream)))
    return ws


def indexer_topk_hier(dims: Dims, q_I, w, k_I_cache, k_I_scale, block_table, seq_lens, summaries, n_sel: int,
                      q_seq=None, q_pos=None, *, ws, idx=None, blocks=None, stream=None):
    """(idx[T][K], blocks[T][n_sel]) of hierarchical selection (coarse blocks, then fine tokens)."""
    T = q_I.shape[0]
    if idx is None:
        idx = torch.empty((T, dims.K), dtype=torch.int32, device=q_I.device)
    if blocks is None:
        blocks = torch.empty((T, n_sel), dtype=torch.int32, device=q_I.device)
    st = lib().dsa_indexer_topk_hier(ctypes.byref(dims), _p(q_I), _p(w), _p(k_I_cache), _p(k_I_scale), _p(block_table),
                                     _p(seq_lens), _p(q_seq), _p(q_pos), T, _p(summaries), n_sel, _p(idx), _p(blocks),
                                     _p(ws), ws.numel(), _stream(stream))
    _check("dsa_indexer_topk_hier", st)
    return idx, blocks


def read_error(ws, stream=None) -> int:
    """Synchronises the stream and returns (then clears) the device fault bits of ``ws``."""
    bits = ctypes.c_int32(0)
    st = lib().dsa_read_error(_p(ws), ctypes.byref(bits), _stream(stream))
    if st not in (0, 5, 6):
        raise DsaError("dsa_read_error", st)
    return int(bits.value)


def selftest_wait_timeout(ws, stream=None) -> None:
    """Runs the bounded-wait self-test (its wait runs out after about a second and sets the
    timeout bit of ``ws``; read it with :func:`read_error`)."""
    _check("dsa_selftest_wait_timeout", lib().dsa_selftest_wait_timeout(_p(ws), ws.numel(), _stream(stream)))


def last_launch_count() -> int:
    return int(lib().dsa_last_launch_count())
