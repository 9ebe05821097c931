"""Python binding of libdsa.so -- the DSA sparse-attention hot path for GB300.

Argument marshalling only: every stage runs in the library's CUDA kernels.
PyTorch supplies device memory and the current CUDA stream; tensors are passed
as raw device pointers to the C ABI declared in ``include/dsa.h``.

Stages (names as in the C ABI):

* :func:`index_score` -- indexer score of every cached position, ReLU-weighted
  over indexer heads ("Day-0 Adaptation of Trillion-Parameter MoE Models on
  Domestic GPUs", section 3 (1));
* :func:`topk` -- exact top-K per query, ties to the lower position ("Day-0
  Adaptation of Ultra-Large-Scale MoE Models on Heterogeneous AI
  Accelerators", section 4);
* :func:`sparse_attn_decode` / :func:`sparse_attn_prefill` -- exact softmax
  attention over the selected rows gathered through the block table (first
  page, section 3 (2)-(3)).

Around them: :func:`head_norm_rope` and :func:`cache_append` (heads of new
tokens), :func:`prefix_attn_decode` (every position, a shared prefix read once)
and, for layers with grouped heads, :func:`prompt_attn` (exact causal attention
of packed prompts) and a cache of 4 bits per element (:func:`cache4_pool`,
:func:`cache4_write`, :func:`cache4_read`, :func:`cache4_attn_decode`).

:func:`decode` and :func:`prefill` chain the three stages with workspaces
allocated through torch.  There is no CPU fallback: importing this package
raises if ``libdsa.so`` has not been built, and every call raises
:class:`DsaError` if the library reports an error.
"""
from __future__ import annotations

import ctypes
import math
import os
from dataclasses import dataclass
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdsa.so")

DSA_OK = 0
DSA_BF16 = 0
DSA_FP8_E4M3 = 1
STATUS_BAD_BLOCK = 0x1
STATUS_BAD_INDEX = 0x2
STATUS_BAD_LENGTH = 0x4
STATUS_TIMEOUT = 0x8
NORMS = {"none": 0, "rms": 1, "layer": 2}
MAX_HEAD_PARTS = 4

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")

_lib = ctypes.CDLL(LIB_PATH)


class DsaError(RuntimeError):
    def __init__(self, code: int, where: str):
        msg = _lib.dsa_last_error_string().decode(errors="replace")
        super().__init__(f"{where} failed with code {code}: {msg}")
        self.code = code


class PagedLayoutC(ctypes.Structure):
    _fields_ = [("block_size", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
                ("max_blocks_per_seq", ctypes.c_int32), ("batch", ctypes.c_int32),
                ("max_seq_len", ctypes.c_int32), ("reserved_", ctypes.c_int32),
                ("block_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p)]


class HeadPartC(ctypes.Structure):
    _fields_ = [("in_", ctypes.c_void_p), ("in_token_stride", ctypes.c_int64),
                ("in_head_stride", ctypes.c_int64), ("out", ctypes.c_void_p),
                ("out_token_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64),
                ("out_dtype", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("dim", ctypes.c_int32), ("norm", ctypes.c_int32), ("norm_dim", ctypes.c_int32),
                ("eps", ctypes.c_float), ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("rope_offset", ctypes.c_int32), ("rope_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("reserved_", ctypes.c_int32),
                ("inv_freq", ctypes.c_void_p)]


_vp, _i, _i64, _sz, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
_LP = ctypes.POINTER(PagedLayoutC)


def _sig(name, restype, argtypes):
    fn = getattr(_lib, name)
    fn.restype = restype
    fn.argtypes = argtypes
    return fn


_sig("dsa_version", _i, [])
_sig("dsa_launch_count", ctypes.c_uint64, [])
_sig("dsa_last_error_string", ctypes.c_char_p, [])
_sig("dsa_get_status", _i, [_vp, _vp, ctypes.POINTER(ctypes.c_int32), _i])
_sig("dsa_selftest_bounded_wait", _i, [_i, ctypes.c_uint64, _vp, _sz, _vp])
_sig("dsa_selftest_warp_wait", _i, [_i, ctypes.c_uint64, _vp, _sz, _vp])
_sig("dsa_index_score_workspace_size", _sz, [_i, _i, _i, _i64])
_sig("dsa_index_score", _i, [_LP, _vp, _vp, _vp, _i, _i, _i, _vp, _vp, _i, _vp, _i64, _vp, _sz, _vp])
_sig("dsa_index_score_prefill_workspace_size", _sz, [_i, _i, _i, _i64])
_sig("dsa_index_score_prefill", _i, [_LP, _i, _vp, _vp, _vp, _i, _i, _i, _vp, _i, _vp, _i64, _vp, _sz,
                                     _vp])
_sig("dsa_topk_workspace_size", _sz, [_i, _i64, _i])
_sig("dsa_topk", _i, [_vp, _i64, _vp, _i, _i, _vp, _vp, _sz, _vp])
_sig("dsa_topk_noalloc", _i, [_vp, _i64, _vp, _i, _i, _vp, _vp])
_sig("dsa_topk_noalloc_scratch_bytes", _sz, [])
_sig("dsa_decode_step_workspace_size", _sz, [_i, _i, _i, _i64, _i, _i, _i, _i])
_sig("dsa_decode_step", _i, [_LP, _vp, _vp, _i64, _vp, _vp, _i64, _vp, _vp, _i, _vp, _vp, _i, _i,
                             _vp, _i, _i, _i, _i, _f, _vp, _i64, _vp, _vp, _vp, _vp, _sz, _vp])
_sig("dsa_prefill_step_workspace_size", _sz, [_i, _i, _i, _i64, _i, _i, _i, _i])
_sig("dsa_prefill_step", _i, [_LP, _i, _vp, _vp, _i, _vp, _vp, _i64, _vp, _vp, _i64, _vp, _vp, _i,
                              _vp, _vp, _i, _i, _vp, _i, _i, _i, _i, _f, _vp, _i64, _vp, _vp, _vp,
                              _vp, _sz, _vp])
_sig("dsa_prefill_step_chunked_workspace_size", _sz, [_i, _i, _i, _i64, _i, _i, _i, _i, _i])
_sig("dsa_prefill_step_chunked", _i, [_LP, _i, _vp, _vp, _i, _vp, _vp, _i64, _vp, _vp, _i64, _vp,
                                      _vp, _i, _vp, _vp, _i, _i, _vp, _i, _i, _i, _i, _f, _i64, _i,
                                      _vp, _vp, _vp, _vp, _sz, _vp])
_sig("dsa_index_bounds_update_workspace_size", _sz, [])
_sig("dsa_index_bounds_update", _i, [_LP, _vp, _vp, _i, _vp, _i, _i, _vp, _vp, _sz, _vp])
_sig("dsa_index_score_bounded_workspace_size", _sz, [_i, _i, _i, _i64, _i])
_sig("dsa_index_score_bounded", _i, [_LP, _vp, _vp, _vp, _i, _i, _i, _vp, _i, _vp, _i64, _vp, _sz,
                                     _vp])
_sig("dsa_index_bounded_stats", _i, [_vp, _vp, ctypes.POINTER(ctypes.c_uint64),
                                     ctypes.POINTER(ctypes.c_uint64)])
_sig("dsa_cache_write_workspace_size", _sz, [])
_sig("dsa_cache_write", _i, [_LP, _vp, _vp, _i, _vp, _i, _vp, _i64, _vp, _i, _i, _vp, _vp, _sz, _vp])
_sig("dsa_sparse_attn_decode_workspace_size", _sz, [_i, _i, _i, _i, _i])
_sig("dsa_sparse_attn_decode", _i, [_LP, _vp, _vp, _i64, _vp, _i64, _i, _i, _i, _vp, _i, _f, _vp,
                                    _vp, _vp, _sz, _vp])
_sig("dsa_sparse_attn_prefill_workspace_size", _sz, [_i, _i, _i, _i, _i])
_sig("dsa_sparse_attn_prefill", _i, [_LP, _vp, _vp, _i64, _vp, _i64, _i, _i, _i, _vp, _vp, _i, _vp,
                                     _i, _f, _vp, _vp, _vp, _sz, _vp])
_sig("dsa_head_norm_rope", _i, [_vp, _i, _vp, _i, _vp])
_sig("dsa_cache_append_workspace_size", _sz, [])
_sig("dsa_cache_append", _i, [_LP, _vp, _vp, _i, _vp, _i, _vp, _i, _vp, _sz, _vp])
_sig("dsa_prefix_attn_decode_workspace_size", _sz, [_i, _i, _i, _i, _i])
_sig("dsa_prefix_attn_decode", _i, [_LP, _vp, _vp, _i64, _vp, _i64, _i, _i, _i, _i, _f, _vp, _vp,
                                    _vp, _sz, _vp])
_sig("dsa_prompt_attn_workspace_size", _sz, [_i, _i, _i, _i, _i, _i])
_sig("dsa_prompt_attn", _i, [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i, _i, _i, _i,
                             _i, _i, _i, _f, _vp, _i64, _i64, _vp, _vp, _sz, _vp])
_sig("dsa_cache4_row_bytes", _sz, [_i, _i])
_sig("dsa_cache4_write_workspace_size", _sz, [])
_sig("dsa_cache4_write", _i, [_LP, _vp, _vp, _i, _vp, _i64, _i64, _vp, _i64, _i64, _i, _i, _i, _vp, _vp,
                              _vp, _vp, _vp, _vp, _sz, _vp])
_sig("dsa_cache4_read_workspace_size", _sz, [])
_sig("dsa_cache4_read", _i, [_LP, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp])
_sig("dsa_cache4_attn_decode_workspace_size", _sz, [_i, _i, _i, _i, _i])
_sig("dsa_cache4_attn_decode", _i, [_LP, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _f, _vp, _vp, _vp, _sz,
                                    _vp])

SYMBOLS = ("dsa_version", "dsa_launch_count", "dsa_last_error_string", "dsa_get_status",
           "dsa_selftest_bounded_wait", "dsa_selftest_warp_wait",
           "dsa_index_score_workspace_size", "dsa_index_score",
           "dsa_index_score_prefill_workspace_size", "dsa_index_score_prefill",
           "dsa_topk_workspace_size",
           "dsa_topk", "dsa_topk_noalloc", "dsa_topk_noalloc_scratch_bytes",
           "dsa_sparse_attn_decode_workspace_size", "dsa_sparse_attn_decode",
           "dsa_sparse_attn_prefill_workspace_size", "dsa_sparse_attn_prefill",
           "dsa_cache_write_workspace_size", "dsa_cache_write",
           "dsa_decode_step_workspace_size", "dsa_decode_step",
           "dsa_prefill_step_workspace_size", "dsa_prefill_step",
           "dsa_prefill_step_chunked_workspace_size", "dsa_prefill_step_chunked",
           "dsa_index_bounds_update_workspace_size", "dsa_index_bounds_update",
           "dsa_index_score_bounded_workspace_size", "dsa_index_score_bounded",
           "dsa_index_bounded_stats",
           "dsa_head_norm_rope", "dsa_cache_append_workspace_size", "dsa_cache_append",
           "dsa_prefix_attn_decode_workspace_size", "dsa_prefix_attn_decode",
           "dsa_prompt_attn_workspace_size", "dsa_prompt_attn",
           "dsa_cache4_row_bytes", "dsa_cache4_write_workspace_size", "dsa_cache4_write",
           "dsa_cache4_read_workspace_size", "dsa_cache4_read",
           "dsa_cache4_attn_decode_workspace_size", "dsa_cache4_attn_decode")


def lib() -> ctypes.CDLL:
    return _lib


def version() -> int:
    return int(_lib.dsa_version())


def launch_count() -> int:
    """Kernels launched by libdsa.so in this process so far."""
    return int(_lib.dsa_launch_count())


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


class _Args:
    """The operands of one call, checked so that no kernel can run outside
    them: as each is added, its element size and element count (at least
    what the call touches); then, in ptrs(), that every one of them and the
    layout live on the GPU.  Sizes are checked for all operands before
    residency for any, so that each check can be exercised with host
    tensors."""

    def __init__(self, layout: Optional["PagedLayout"] = None):
        self._t = []
        self._layout = layout

    def add(self, t: Optional[torch.Tensor], name: str, elt=None, numel: Optional[int] = None):
        if t is not None:
            if elt is not None and t.element_size() not in elt:
                raise TypeError(f"{name}: {t.dtype} has {t.element_size()}-byte elements; "
                                f"the call needs {' or '.join(str(e) for e in elt)}")
            if numel is not None and t.numel() < numel:
                raise ValueError(f"{name}: {t.numel()} elements; the call needs at least "
                                 f"{numel}")
        self._t.append((t, name))
        return self

    def ptrs(self):
        for t, name in self._t:
            if t is not None and not t.is_cuda:
                raise ValueError(f"{name}: a CUDA tensor is required")
        lay = self._layout
        if lay is not None and not (lay.block_table.is_cuda and lay.seq_lens.is_cuda):
            raise ValueError("layout: block_table and seq_lens must be CUDA tensors")
        return [_ptr(t) for t, _ in self._t]


def _rows(layout: "PagedLayout", width: int, kidx_pool=None) -> int:
    """Elements of a paged pool of `width`-element rows (kidx_pool: the pool, to be
    of one head)."""
    if kidx_pool is not None:
        _row_width(layout, kidx_pool, "kidx_pool")
    return int(layout.num_blocks) * int(layout.block_size) * int(width)


def _row_width(layout: "PagedLayout", pool, name: str) -> int:
    """Elements between the rows of a pool [num_blocks, block_size, width]
    (or [.., 1, width]).  A pool of several heads is refused: its last dimension
    is a head, not a row."""
    if (pool.dim() == 4 and pool.shape[2] != 1 and pool.shape[1] == layout.block_size
            and pool.shape[0] >= layout.num_blocks):
        raise ValueError(f"{name}: {pool.shape[2]} heads per row; the call reads rows of one")
    return pool.shape[-1]


_F32, _I32, _BF16, _KEY, _WS = (4,), (4,), (2,), (1, 2), (1,)  # element sizes (bytes)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream=None):
    """The CUDA stream handle to launch on: `stream`, else the current stream
    of the current device (read as a raw handle when torch offers that, which
    costs a fraction of building a torch Stream object on every call)."""
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    if _raw_stream is not None:
        return ctypes.c_void_p(_raw_stream(torch.cuda.current_device()))
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _check(rc: int, where: str):
    if rc != DSA_OK:
        raise DsaError(rc, where)


def _elt_dtype(t: torch.Tensor) -> int:
    return DSA_FP8_E4M3 if t.element_size() == 1 else DSA_BF16


@dataclass
class PagedLayout:
    """Block table + sequence lengths on the device (tensors kept alive here)."""

    block_table: torch.Tensor  # int32 [B, max_blocks]
    seq_lens: torch.Tensor     # int32 [B]
    block_size: int
    num_blocks: int
    max_seq_len: int

    def __post_init__(self):
        if self.block_table.dtype != torch.int32 or self.seq_lens.dtype != torch.int32:
            raise TypeError("block_table and seq_lens must be int32")
        self._c = PagedLayoutC(int(self.block_size), int(self.num_blocks),
                               int(self.block_table.shape[1]), int(self.block_table.shape[0]),
                               int(self.max_seq_len), 0, self.block_table.data_ptr(),
                               self.seq_lens.data_ptr())

    @property
    def batch(self) -> int:
        return int(self.block_table.shape[0])

    def c(self):
        return ctypes.byref(self._c)


def workspace(nbytes: int, device=None) -> torch.Tensor:
    """Zero-filled device workspace (uint8), 256-byte aligned by the allocator."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")


def index_score_workspace_size(Nq, H_i, D_i, ld) -> int:
    return int(_lib.dsa_index_score_workspace_size(Nq, H_i, D_i, ld))


def topk_workspace_size(Nq, ld, K) -> int:
    return int(_lib.dsa_topk_workspace_size(Nq, ld, K))


def sparse_attn_decode_workspace_size(B, Hq, Dqk, Dv, K) -> int:
    return int(_lib.dsa_sparse_attn_decode_workspace_size(B, Hq, Dqk, Dv, K))


def sparse_attn_prefill_workspace_size(Nq, Hq, Dqk, Dv, K) -> int:
    return int(_lib.dsa_sparse_attn_prefill_workspace_size(Nq, Hq, Dqk, Dv, K))


def index_score(layout: PagedLayout, q_idx, w, kidx_pool, scores, ws, q_seq=None, q_pos=None,
                stream=None):
    """scores[Nq, ld] <- indexer scores (see include/dsa.h, dsa_index_score)."""
    Nq, H_i, D_i = q_idx.shape
    ld = scores.shape[1]
    a = _Args(layout).add(q_idx, "q_idx", _KEY).add(w, "w", _F32, Nq * H_i)
    a.add(kidx_pool, "kidx_pool", (q_idx.element_size(),), _rows(layout, D_i, kidx_pool))
    a.add(q_seq, "q_seq", _I32, Nq).add(q_pos, "q_pos", _I32, Nq)
    a.add(scores, "scores", _F32, Nq * ld).add(ws, "ws", _WS)
    pq, pw, pk, pseq, ppos, ps, pws = a.ptrs()
    rc = _lib.dsa_index_score(layout.c(), pq, pw, pk, _elt_dtype(kidx_pool), H_i, D_i, pseq, ppos,
                              Nq, ps, ld, pws, ws.numel(), _stream(stream))
    _check(rc, "dsa_index_score")


def index_score_prefill(layout: PagedLayout, seq, q_idx, w, kidx_pool, scores, ws, q_pos=None,
                        stream=None):
    """scores[Nq, ld] <- indexer scores of Nq queries of sequence `seq`."""
    Nq, H_i, D_i = q_idx.shape
    ld = scores.shape[1]
    a = _Args(layout).add(q_idx, "q_idx", _KEY).add(w, "w", _F32, Nq * H_i)
    a.add(kidx_pool, "kidx_pool", (q_idx.element_size(),), _rows(layout, D_i, kidx_pool))
    a.add(q_pos, "q_pos", _I32, Nq).add(scores, "scores", _F32, Nq * ld).add(ws, "ws", _WS)
    pq, pw, pk, ppos, ps, pws = a.ptrs()
    rc = _lib.dsa_index_score_prefill(layout.c(), int(seq), pq, pw, pk, _elt_dtype(kidx_pool), H_i,
                                      D_i, ppos, Nq, ps, ld, pws, ws.numel(), _stream(stream))
    _check(rc, "dsa_index_score_prefill")


def topk(scores, n_eligible, K, idx, ws, stream=None):
    """idx[Nq, K] <- top-K positions, ascending, -1 padded."""
    Nq, ld = scores.shape
    K = int(K)
    a = _Args().add(scores, "scores", _F32).add(n_eligible, "n_eligible", _I32, Nq)
    a.add(idx, "idx", _I32, Nq * K).add(ws, "ws", _WS)
    ps, pn, pi, pws = a.ptrs()
    rc = _lib.dsa_topk(ps, ld, pn, Nq, K, pi, pws, ws.numel(), _stream(stream))
    _check(rc, "dsa_topk")


# Size of the fixed scratch array dsa_topk_noalloc uses, as the loaded library
# reports it (DSA_TOPK_NOALLOC_SCRATCH_BYTES in include/dsa.h).
TOPK_NOALLOC_SCRATCH_BYTES = int(_lib.dsa_topk_noalloc_scratch_bytes())


def topk_noalloc(scores, n_eligible, K, idx, stream=None):
    """dsa_topk without a workspace, for callers that may not allocate device
    memory: the scratch is a fixed array inside the library, shared by every
    call (calls that overlap on the GPU race)."""
    Nq, ld = scores.shape
    K = int(K)
    a = _Args().add(scores, "scores", _F32).add(n_eligible, "n_eligible", _I32, Nq)
    a.add(idx, "idx", _I32, Nq * K)
    ps, pn, pi = a.ptrs()
    rc = _lib.dsa_topk_noalloc(ps, ld, pn, Nq, K, pi, _stream(stream))
    _check(rc, "dsa_topk_noalloc")


def sparse_attn_decode(layout: PagedLayout, q, k_pool, v_pool, idx, sm_scale, out, lse, ws,
                       stream=None):
    B, Hq, Dqk = q.shape
    Dv, K = out.shape[2], idx.shape[1]
    ks, vs = _row_width(layout, k_pool, "k_pool"), _row_width(layout, v_pool, "v_pool")
    a = _Args(layout).add(q, "q", _BF16).add(k_pool, "k_pool", _BF16, _rows(layout, ks))
    a.add(v_pool, "v_pool", _BF16, _rows(layout, vs)).add(idx, "idx", _I32, B * K)
    a.add(out, "out", _BF16, B * Hq * Dv).add(lse, "lse", _F32, B * Hq)
    a.add(ws, "ws", _WS)
    pq, pk, pv, pi, po, pl, pws = a.ptrs()
    rc = _lib.dsa_sparse_attn_decode(layout.c(), pq, pk, ks, pv, vs, Hq, Dqk, Dv, pi, K,
                                     float(sm_scale), po, pl, pws, ws.numel(), _stream(stream))
    _check(rc, "dsa_sparse_attn_decode")


def sparse_attn_prefill(layout: PagedLayout, q, k_pool, v_pool, idx, sm_scale, out, lse, ws,
                        q_seq=None, q_pos=None, stream=None):
    Nq, Hq, Dqk = q.shape
    Dv, K = out.shape[2], idx.shape[1]
    ks, vs = _row_width(layout, k_pool, "k_pool"), _row_width(layout, v_pool, "v_pool")
    a = _Args(layout).add(q, "q", _BF16).add(k_pool, "k_pool", _BF16, _rows(layout, ks))
    a.add(v_pool, "v_pool", _BF16, _rows(layout, vs)).add(idx, "idx", _I32, Nq * K)
    a.add(out, "out", _BF16, Nq * Hq * Dv).add(lse, "lse", _F32, Nq * Hq)
    a.add(q_seq, "q_seq", _I32, Nq).add(q_pos, "q_pos", _I32, Nq).add(ws, "ws", _WS)
    pq, pk, pv, pi, po, pl, pseq, ppos, pws = a.ptrs()
    rc = _lib.dsa_sparse_attn_prefill(layout.c(), pq, pk, ks, pv, vs, Hq, Dqk, Dv, pseq, ppos, Nq,
                                      pi, K, float(sm_scale), po, pl, pws, ws.numel(),
                                      _stream(stream))
    _check(rc, "dsa_sparse_attn_prefill")


def cache_write_workspace_size() -> int:
    return int(_lib.dsa_cache_write_workspace_size())


def cache_write(layout: PagedLayout, seq, pos, ws, kv_new=None, kv_pool=None, kidx_new=None,
                kidx_pool=None, stream=None):
    """Store row i of kv_new / kidx_new at position pos[i] of sequence seq[i] of
    kv_pool / kidx_pool, through the block table (include/dsa.h, dsa_cache_write).

    kv_new [N, row_elems] bf16 into kv_pool [NB, bs, stride >= row_elems];
    kidx_new [N, D_i] into kidx_pool [NB, bs, D_i] (bf16 or FP8 E4M3).
    """
    N = int(seq.shape[0])
    row_elems = int(kv_new.shape[-1]) if kv_new is not None else 0
    stride = int(_row_width(layout, kv_pool, "kv_pool")) if kv_pool is not None else 0
    D_i = int(kidx_new.shape[-1]) if kidx_new is not None else 0
    kdt = _elt_dtype(kidx_new) if kidx_new is not None else DSA_BF16
    ke = (kidx_new.element_size(),) if kidx_new is not None else _KEY
    a = _Args(layout).add(seq, "seq", _I32, N).add(pos, "pos", _I32, N)
    a.add(kv_new, "kv_new", _BF16, N * row_elems)
    a.add(kv_pool, "kv_pool", _BF16, _rows(layout, stride) if kv_new is not None else None)
    a.add(kidx_new, "kidx_new", _KEY, N * D_i)
    a.add(kidx_pool, "kidx_pool", ke,
          _rows(layout, D_i, kidx_pool) if kidx_new is not None else None)
    a.add(ws, "ws", _WS)
    pseq, ppos, pkv, pkp, pin, pip, pws = a.ptrs()
    rc = _lib.dsa_cache_write(layout.c(), pseq, ppos, N, pkv, row_elems, pkp, stride, pin, D_i, kdt,
                              pip, pws, ws.numel(), _stream(stream))
    _check(rc, "dsa_cache_write")


def index_bounds_update_workspace_size() -> int:
    return int(_lib.dsa_index_bounds_update_workspace_size())


def index_bounds_update(layout: PagedLayout, kidx_pool, kbound_pool, ws, seq=None, pos=None,
                        stream=None):
    """Recompute the key bounds of the pages holding rows (seq[i], pos[i]), or of
    every cached page when seq and pos are None (include/dsa.h,
    dsa_index_bounds_update).  kbound_pool [NB, 2, D_i] in the keys' dtype."""
    D_i = int(kidx_pool.shape[-1])
    N = int(seq.shape[0]) if seq is not None else 0
    ke = (kidx_pool.element_size(),)
    a = _Args(layout).add(seq, "seq", _I32, N).add(pos, "pos", _I32, N)
    a.add(kidx_pool, "kidx_pool", ke, _rows(layout, D_i, kidx_pool))
    a.add(kbound_pool, "kbound_pool", ke, layout.num_blocks * 2 * D_i).add(ws, "ws", _WS)
    pseq, ppos, pk, pb, pws = a.ptrs()
    rc = _lib.dsa_index_bounds_update(layout.c(), pseq, ppos, N, pk, D_i, _elt_dtype(kidx_pool),
                                      pb, pws, ws.numel(), _stream(stream))
    _check(rc, "dsa_index_bounds_update")


def index_score_bounded_workspace_size(B, H_i, D_i, ld, K) -> int:
    return int(_lib.dsa_index_score_bounded_workspace_size(B, H_i, D_i, ld, K))


def index_score_bounded(layout: PagedLayout, q_idx, w, kidx_pool, kbound_pool, K, scores, ws,
                        stream=None):
    """Decode indexer scores that leave out the tiles which cannot reach the
    top-K (include/dsa.h, dsa_index_score_bounded); dsa_topk over the row then
    selects exactly what it selects over dsa_index_score's row."""
    B, H_i, D_i = q_idx.shape
    ld = scores.shape[1]
    ke = (kidx_pool.element_size(),)
    a = _Args(layout).add(q_idx, "q_idx", _KEY).add(w, "w", _F32, B * H_i)
    a.add(kidx_pool, "kidx_pool", ke, _rows(layout, D_i, kidx_pool))
    a.add(kbound_pool, "kbound_pool", ke, layout.num_blocks * 2 * D_i)
    a.add(scores, "scores", _F32, B * ld).add(ws, "ws", _WS)
    pq, pw, pk, pb, ps, pws = a.ptrs()
    rc = _lib.dsa_index_score_bounded(layout.c(), pq, pw, pk, _elt_dtype(kidx_pool), H_i, D_i, pb,
                                      int(K), ps, ld, pws, ws.numel(), _stream(stream))
    _check(rc, "dsa_index_score_bounded")


def index_bounded_stats(ws, stream=None):
    """(tiles left out, tiles bounded) by the last dsa_index_score_bounded call on ws."""
    sk, tot = ctypes.c_uint64(0), ctypes.c_uint64(0)
    rc = _lib.dsa_index_bounded_stats(ctypes.c_void_p(ws.data_ptr()), _stream(stream),
                                      ctypes.byref(sk), ctypes.byref(tot))
    _check(rc, "dsa_index_bounded_stats")
    return int(sk.value), int(tot.value)


def decode_step_workspace_size(B, H_i, D_i, ld, Hq, Dqk, Dv, K) -> int:
    return int(_lib.dsa_decode_step_workspace_size(B, H_i, D_i, ld, Hq, Dqk, Dv, K))


def prefill_step_workspace_size(Nq, H_i, D_i, ld, Hq, Dqk, Dv, K) -> int:
    return int(_lib.dsa_prefill_step_workspace_size(Nq, H_i, D_i, ld, Hq, Dqk, Dv, K))


def decode_step(layout: PagedLayout, k_new, k_pool, kidx_new, kidx_pool, q_idx, w, q, K, sm_scale,
                scores, idx, out, lse, ws, v_new=None, v_pool=None, stream=None):
    """One incremental decode step (include/dsa.h, dsa_decode_step): append each
    sequence's new K/V and indexer-key rows at position seq_lens[b] - 1, then
    score, select and attend.  v_pool None: V is the first Dv dims of the K row."""
    B, Hq, Dqk = q.shape
    a = _Args(layout)
    H_i, D_i = q_idx.shape[1], q_idx.shape[2]
    Dv, K, ld = out.shape[2], int(K), scores.shape[1]
    vp = k_pool if v_pool is None else v_pool
    ks, vs = _row_width(layout, k_pool, "k_pool"), _row_width(layout, vp, "v_pool")
    ke = (q_idx.element_size(),)
    a.add(k_new, "k_new", _BF16, B * Dqk).add(k_pool, "k_pool", _BF16, _rows(layout, ks))
    a.add(v_new, "v_new", _BF16, B * Dv).add(vp, "v_pool", _BF16, _rows(layout, vs))
    a.add(kidx_new, "kidx_new", ke, B * D_i)
    a.add(kidx_pool, "kidx_pool", ke, _rows(layout, D_i, kidx_pool))
    a.add(q_idx, "q_idx", _KEY).add(w, "w", _F32, B * H_i).add(q, "q", _BF16)
    a.add(scores, "scores", _F32, B * ld).add(idx, "idx", _I32, B * K)
    a.add(out, "out", _BF16, B * Hq * Dv).add(lse, "lse", _F32, B * Hq).add(ws, "ws", _WS)
    (pkn, pkp, pvn, pvp, pin, pip, pqi, pw, pq, ps, pi, po, pl, pws) = a.ptrs()
    rc = _lib.dsa_decode_step(layout.c(), pkn, pkp, ks, pvn, pvp, vs, pin, pip,
                              _elt_dtype(kidx_pool), pqi, pw, H_i, D_i, pq, Hq, Dqk, Dv, K,
                              float(sm_scale), ps, ld, pi, po, pl, pws, ws.numel(),
                              _stream(stream))
    _check(rc, "dsa_decode_step")


def prefill_step(layout: PagedLayout, seq, q_pos, n_eligible, k_new, k_pool, kidx_new, kidx_pool,
                 q_idx, w, q, K, sm_scale, scores, idx, out, lse, ws, v_new=None, v_pool=None,
                 stream=None):
    """A prompt (or a chunk after an existing prefix) of sequence `seq` in one
    call (include/dsa.h, dsa_prefill_step): its rows are written at q_pos, then
    scored, selected and attended."""
    Nq, Hq, Dqk = q.shape
    a = _Args(layout).add(q_pos, "q_pos", _I32, Nq).add(n_eligible, "n_eligible", _I32, Nq)
    H_i, D_i = q_idx.shape[1], q_idx.shape[2]
    Dv, K, ld = out.shape[2], int(K), scores.shape[1]
    vp = k_pool if v_pool is None else v_pool
    ks, vs = _row_width(layout, k_pool, "k_pool"), _row_width(layout, vp, "v_pool")
    ke = (q_idx.element_size(),)
    a.add(k_new, "k_new", _BF16, Nq * Dqk).add(k_pool, "k_pool", _BF16, _rows(layout, ks))
    a.add(v_new, "v_new", _BF16, Nq * Dv).add(vp, "v_pool", _BF16, _rows(layout, vs))
    a.add(kidx_new, "kidx_new", ke, Nq * D_i)
    a.add(kidx_pool, "kidx_pool", ke, _rows(layout, D_i, kidx_pool))
    a.add(q_idx, "q_idx", _KEY).add(w, "w", _F32, Nq * H_i).add(q, "q", _BF16)
    a.add(scores, "scores", _F32, Nq * ld).add(idx, "idx", _I32, Nq * K)
    a.add(out, "out", _BF16, Nq * Hq * Dv).add(lse, "lse", _F32, Nq * Hq).add(ws, "ws", _WS)
    (ppos, pn, pkn, pkp, pvn, pvp, pin, pip, pqi, pw, pq, ps, pi, po, pl, pws) = a.ptrs()
    rc = _lib.dsa_prefill_step(layout.c(), int(seq), ppos, pn, Nq, pkn, pkp, ks, pvn, pvp, vs,
                               pin, pip, _elt_dtype(kidx_pool), pqi, pw, H_i, D_i, pq, Hq, Dqk, Dv,
                               K, float(sm_scale), ps, ld, pi, po, pl, pws, ws.numel(),
                               _stream(stream))
    _check(rc, "dsa_prefill_step")


def prefill_step_chunked_workspace_size(Nq, H_i, D_i, ld, Hq, Dqk, Dv, K, chunk=0) -> int:
    return int(_lib.dsa_prefill_step_chunked_workspace_size(Nq, H_i, D_i, ld, Hq, Dqk, Dv, K,
                                                            int(chunk)))


def prefill_step_chunked(layout: PagedLayout, seq, q_pos, n_eligible, k_new, k_pool, kidx_new,
                         kidx_pool, q_idx, w, q, K, sm_scale, ld, idx, out, lse, ws, chunk=0,
                         v_new=None, v_pool=None, stream=None):
    """dsa_prefill_step without the score matrix (include/dsa.h,
    dsa_prefill_step_chunked): queries scored and selected `chunk` at a time
    (0: automatic) through a scratch in the workspace."""
    Nq, Hq, Dqk = q.shape
    a = _Args(layout).add(q_pos, "q_pos", _I32, Nq).add(n_eligible, "n_eligible", _I32, Nq)
    H_i, D_i = q_idx.shape[1], q_idx.shape[2]
    Dv, K, ld = out.shape[2], int(K), int(ld)
    vp = k_pool if v_pool is None else v_pool
    ks, vs = _row_width(layout, k_pool, "k_pool"), _row_width(layout, vp, "v_pool")
    ke = (q_idx.element_size(),)
    a.add(k_new, "k_new", _BF16, Nq * Dqk).add(k_pool, "k_pool", _BF16, _rows(layout, ks))
    a.add(v_new, "v_new", _BF16, Nq * Dv).add(vp, "v_pool", _BF16, _rows(layout, vs))
    a.add(kidx_new, "kidx_new", ke, Nq * D_i)
    a.add(kidx_pool, "kidx_pool", ke, _rows(layout, D_i, kidx_pool))
    a.add(q_idx, "q_idx", _KEY).add(w, "w", _F32, Nq * H_i).add(q, "q", _BF16)
    a.add(idx, "idx", _I32, Nq * K).add(out, "out", _BF16, Nq * Hq * Dv)
    a.add(lse, "lse", _F32, Nq * Hq).add(ws, "ws", _WS)
    (ppos, pn, pkn, pkp, pvn, pvp, pin, pip, pqi, pw, pq, pi, po, pl, pws) = a.ptrs()
    rc = _lib.dsa_prefill_step_chunked(layout.c(), int(seq), ppos, pn, Nq, pkn, pkp, ks, pvn, pvp,
                                       vs, pin, pip, _elt_dtype(kidx_pool), pqi, pw, H_i, D_i, pq,
                                       Hq, Dqk, Dv, K, float(sm_scale), ld, int(chunk), pi, po, pl,
                                       pws, ws.numel(), _stream(stream))
    _check(rc, "dsa_prefill_step_chunked")


class HeadPart:
    """One tensor of new tokens' heads, normed and rotated on the way to `out`
    (include/dsa.h, dsa_head_part).

    x [N, heads, dim] bf16, any strides with the last dim contiguous (a slice
    of a projection's output).  out: [N, heads, dim] bf16 or FP8 E4M3, strided
    likewise, for head_norm_rope and cache_append(heads=...); a paged pool
    [num_blocks, block_size, heads * dim or wider], its heads packed, or
    [num_blocks, block_size, heads or more, dim or wider], a head in each slot,
    contiguous, for cache_append(cache); FP8 as float8_e4m3fn or as uint8 codes.
    norm: "none", "rms" or "layer" over the first norm_dim elements (default:
    all), weight / bias fp32 [norm_dim].
    rope_dim > 0 rotates elements [rope_offset, rope_offset + rope_dim) by
    position * inv_freq (fp32 [rope_dim / 2]); interleaved pairs
    (2 i, 2 i + 1), else (i, i + rope_dim / 2).  Shapes and types are checked
    here, once; the tensors are kept alive by the part.
    """

    def __init__(self, x, out, *, norm="none", norm_dim=None, eps=1e-6, weight=None, bias=None,
                 rope_offset=0, rope_dim=0, interleaved=False, inv_freq=None):
        if x.dim() != 3 or x.stride(2) != 1 and x.shape[2] > 1:
            raise ValueError("x: [N, heads, dim] with a contiguous last dim is required")
        if x.dtype != torch.bfloat16:
            raise TypeError(f"x: {x.dtype}; bfloat16 is required")
        if out.dtype not in (torch.bfloat16, torch.float8_e4m3fn, torch.uint8):
            raise TypeError(f"out: {out.dtype}; bfloat16, float8_e4m3fn or uint8 (E4M3 codes) "
                            "is required")
        if norm not in NORMS:
            raise ValueError(f"norm: {norm!r}; one of {', '.join(NORMS)}")
        n, heads, dim = x.shape
        norm_dim = dim if norm_dim is None else int(norm_dim)
        if norm == "none":
            norm_dim = 0
        for t, name, count in ((weight, "weight", norm_dim), (bias, "bias", norm_dim),
                               (inv_freq, "inv_freq", int(rope_dim) // 2)):
            if t is not None:
                if t.dtype != torch.float32:
                    raise TypeError(f"{name}: {t.dtype}; float32 is required")
                if not t.is_contiguous() or t.numel() < count:
                    raise ValueError(f"{name}: {count} contiguous elements are required")
        if rope_dim and inv_freq is None:
            raise ValueError("inv_freq: required when rope_dim > 0")
        self.x, self.out, self.weight, self.bias, self.inv_freq = x, out, weight, bias, inv_freq
        self.N = int(n)
        self._spec = (int(heads), int(dim), NORMS[norm], norm_dim, float(eps), int(rope_offset),
                      int(rope_dim), 1 if interleaved else 0)

    def _c(self, paged: bool) -> HeadPartC:
        heads, dim, norm, norm_dim, eps, roff, rdim, inter = self._spec
        x, out = self.x, self.out
        if paged:
            if out.dim() not in (3, 4) or not out.is_contiguous():
                raise ValueError("out: a contiguous pool [num_blocks, block_size, width] is required")
            ts, hs = self.row(), dim
            if out.dim() == 4:
                if out.shape[2] < heads or out.shape[3] < dim:
                    raise ValueError(f"out: a pool of {out.shape[2]} heads of {out.shape[3]}; "
                                     f"{heads} of {dim} are needed")
                hs = out.shape[3]
            elif ts < heads * dim:
                raise ValueError(f"out: pool rows of {ts} elements; {heads * dim} are needed")
        else:
            if tuple(out.shape) != (self.N, heads, dim) or out.stride(2) != 1 and dim > 1:
                raise ValueError(f"out: {tuple(out.shape)}; {(self.N, heads, dim)} with a "
                                 "contiguous last dim is required")
            # a dimension of one element may carry any stride
            ts = out.stride(0) if self.N > 1 else 0
            hs = out.stride(1) if heads > 1 else dim
        xts = x.stride(0) if self.N > 1 else 0
        xhs = x.stride(1) if heads > 1 else 0
        opt = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        return HeadPartC(x.data_ptr(), xts, xhs, out.data_ptr(), ts, hs,
                         _elt_dtype(out), heads, dim, norm, norm_dim, eps, opt(self.weight),
                         opt(self.bias), roff, rdim, inter, 0, opt(self.inv_freq))

    def row(self) -> int:
        """Elements of a row of `out` as a pool (from its shape: a page of one
        row may carry any stride)."""
        return math.prod(self.out.shape[2:])

    def tensors(self):
        return [(t, n) for t, n in ((self.x, "x"), (self.out, "out"), (self.weight, "weight"),
                                    (self.bias, "bias"), (self.inv_freq, "inv_freq"))
                if t is not None]


class HeadParts:
    """A list of 1..4 :class:`HeadPart` of the same tokens, with the C array the
    calls take.  A program whose buffers stay where they are builds it once."""

    def __init__(self, parts):
        self.parts = list(parts)
        if not 1 <= len(self.parts) <= MAX_HEAD_PARTS:
            raise ValueError(f"1 to {MAX_HEAD_PARTS} parts are taken")
        self.N = self.parts[0].N
        if any(p.N != self.N for p in self.parts):
            raise ValueError("the parts differ in their number of tokens")
        self.rotates = any(p._spec[6] for p in self.parts)
        self.n = len(self.parts)
        # rows of the smallest pool, for parts that go to paged pools
        self.pool_rows = min(p.out.numel() // max(1, p.row()) if p.out.dim() >= 3 else 0
                             for p in self.parts)
        self._arrays = {}
        self._device = None

    def __len__(self):
        return len(self.parts)

    def c(self, paged: bool):
        arr = self._arrays.get(paged)
        if arr is None:
            arr = (HeadPartC * len(self.parts))(*[p._c(paged) for p in self.parts])
            self._arrays[paged] = arr
        return arr

    def device(self) -> int:
        """Index of the GPU that holds every tensor of the parts."""
        if self._device is None:
            index = None
            for p in self.parts:
                for t, name in p.tensors():
                    if not t.is_cuda:
                        raise ValueError(f"{name}: a CUDA tensor is required")
                    if index is None:
                        index = t.device.index
                    if t.device.index != index:
                        raise ValueError(f"{name}: on {t.device}, other tensors on cuda:{index}")
            self._device = index
        return self._device


def _parts(parts) -> HeadParts:
    return parts if isinstance(parts, HeadParts) else HeadParts(parts)


# A call on a handful of tokens takes the GPU 3 us, so these two calls keep
# their host side short: plain integers to ctypes, one look at the device.
_get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _here(device: int, stream) -> int:
    """Raw handle of the stream to launch on, after a look that the tensors'
    device is the current one."""
    cur = _get_device()
    if device != cur:
        raise ValueError(f"tensors on cuda:{device}; the current device is cuda:{cur}")
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(cur)
    return torch.cuda.current_stream().cuda_stream


def _vec(t, name: str, dtype, numel: int, device: int):
    """Address of a contiguous operand on `device`, checked as _Args does, and
    its type (another type of the same size would be read as `dtype`)."""
    if t is None:
        return None
    if t.dtype != dtype:
        raise TypeError(f"{name}: {t.dtype}; {dtype} is required")
    if t.numel() < numel:
        raise ValueError(f"{name}: {t.numel()} elements; the call needs at least {numel}")
    if t.get_device() != device:
        raise ValueError(f"{name}: a CUDA tensor on cuda:{device} is required")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def head_norm_rope(parts, pos=None, stream=None):
    """Norm and rotate the heads of N tokens at positions pos [N] int32, one
    launch for up to four tensors (include/dsa.h, dsa_head_norm_rope).  parts:
    a :class:`HeadParts`, or a list of :class:`HeadPart`."""
    parts = _parts(parts)
    if pos is None and parts.rotates:
        raise ValueError("pos: required when a part rotates")
    arr = parts.c(False)
    dev = parts._device
    if dev is None:
        if pos is not None and not pos.is_cuda:   # sizes first, then residency, as everywhere
            _vec(pos, "pos", torch.int32, parts.N, -1)
        dev = parts.device()
    rc = _lib.dsa_head_norm_rope(arr, parts.n, _vec(pos, "pos", torch.int32, parts.N, dev), parts.N,
                                 _here(dev, stream))
    if rc:
        raise DsaError(rc, "dsa_head_norm_rope")


def cache_append_workspace_size() -> int:
    return int(_lib.dsa_cache_append_workspace_size())


def cache_append(layout: PagedLayout, seq, pos, cache, ws, heads=None, stream=None):
    """Store the new tokens' K (or latent), V and indexer-key rows in the paged
    pools, normed and rotated on the way, and with heads= their queries in the
    same launch (include/dsa.h, dsa_cache_append).  cache: :class:`HeadParts`
    (or a list of :class:`HeadPart`) whose outs are pools; seq, pos [N] int32,
    or both None: token i is position seq_lens[i] - 1 of sequence i."""
    cache = _parts(cache)
    N = cache.N
    arr = cache.c(True)
    if cache.pool_rows < layout.num_blocks * layout.block_size:
        raise ValueError(f"out: a pool of {cache.pool_rows} rows; the layout needs "
                         f"{layout.num_blocks * layout.block_size}")
    harr, nh = None, 0
    if heads is not None:
        heads = _parts(heads)
        if heads.N != N:
            raise ValueError(f"heads: {heads.N} tokens; the cache parts have {N}")
        harr, nh = heads.c(False), heads.n
    dev = cache._device
    if dev is None:
        for t, name, dtype, numel in ((seq, "seq", torch.int32, N), (pos, "pos", torch.int32, N),
                                      (ws, "ws", torch.uint8, 0)):
            if t is not None and not t.is_cuda:   # sizes first, then residency, as everywhere
                _vec(t, name, dtype, numel, -1)
        dev = cache.device()
    if nh and heads.device() != dev:
        raise ValueError("heads: on another device than the cache parts")
    if layout.block_table.get_device() != dev or layout.seq_lens.get_device() != dev:
        raise ValueError(f"layout: block_table and seq_lens must be CUDA tensors on cuda:{dev}")
    rc = _lib.dsa_cache_append(layout.c(), _vec(seq, "seq", torch.int32, N, dev), _vec(pos, "pos", torch.int32, N, dev),
                               N, arr, cache.n, harr, nh, _vec(ws, "ws", torch.uint8, 0, dev), ws.numel(),
                               _here(dev, stream))
    if rc:
        raise DsaError(rc, "dsa_cache_append")


def prefix_attn_decode_workspace_size(B, Hq, Dqk, Dv, prefix_len) -> int:
    return int(_lib.dsa_prefix_attn_decode_workspace_size(B, Hq, Dqk, Dv, int(prefix_len)))


def prefix_attn_decode(layout: PagedLayout, q, k_pool, v_pool, prefix_len, sm_scale, out, lse, ws,
                       stream=None):
    """Exact attention of one query per sequence over all its cached positions;
    the first prefix_len, shared by the batch, are read once (include/dsa.h,
    dsa_prefix_attn_decode).  prefix_len 0: dense decode attention.  q, out and
    the pools bfloat16, lse float32 or None.  One key head per pool row (the
    first Dqk and Dv elements of it): pools of several key heads take the C call
    once per head, at the head's offset."""
    B, Hq, Dqk = q.shape
    Dv = out.shape[2]
    if B != layout.batch:
        raise ValueError(f"q: {B} sequences; the layout has {layout.batch}")
    ks, vs = _row_width(layout, k_pool, "k_pool"), _row_width(layout, v_pool, "v_pool")
    rows = layout.num_blocks * layout.block_size
    dev = q.get_device()   # -1: the sizes are checked all the same, then q is refused
    pq = _vec(q, "q", torch.bfloat16, 0, dev)
    pk = _vec(k_pool, "k_pool", torch.bfloat16, rows * ks, dev)
    pv = pk if v_pool is k_pool else _vec(v_pool, "v_pool", torch.bfloat16, rows * vs, dev)
    po = _vec(out, "out", torch.bfloat16, B * Hq * Dv, dev)
    pl = _vec(lse, "lse", torch.float32, B * Hq, dev)
    pws = _vec(ws, "ws", torch.uint8, 0, dev)
    if dev < 0:
        raise ValueError("q: a CUDA tensor is required")
    if layout.block_table.get_device() != dev or layout.seq_lens.get_device() != dev:
        raise ValueError(f"layout: block_table and seq_lens must be CUDA tensors on cuda:{dev}")
    rc = _lib.dsa_prefix_attn_decode(layout.c(), pq, pk, ks, pv, vs, Hq, Dqk, Dv, prefix_len,
                                     sm_scale, po, pl, pws, ws.numel(), _here(dev, stream))
    if rc:
        raise DsaError(rc, "dsa_prefix_attn_decode")


# ------------------------------------------------------- prompt attention --
def _strided(t, name: str, dev: int):
    """(address, token stride, head stride) and shape of bf16 heads [N, heads, dim]."""
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name}: {t.dtype}; torch.bfloat16 is required")
    shape, st = t.shape, t.stride()
    if len(shape) != 3:
        raise ValueError(f"{name}: [tokens, heads, dim] is required, not {tuple(shape)}")
    n, heads, dim = shape
    if st[2] != 1 and dim > 1:
        raise ValueError(f"{name}: the elements of a head must be contiguous")
    if t.get_device() != dev:
        raise ValueError(f"{name}: a CUDA tensor on cuda:{dev} is required")
    # the stride of a dimension of one element is never used and may be anything
    return (t.data_ptr(), st[0] if n > 1 else 0, st[1] if heads > 1 else 0), n, heads, dim


def _on_gpu(dev: int, name: str, layout: Optional[PagedLayout] = None):
    if dev < 0:
        raise ValueError(f"{name}: a CUDA tensor is required")
    if layout is not None and (layout.block_table.get_device() != dev
                               or layout.seq_lens.get_device() != dev):
        raise ValueError(f"layout: block_table and seq_lens must be CUDA tensors on cuda:{dev}")


def prompt_attn_workspace_size(B, Nq, Hq, Hk, Dk, Dv) -> int:
    return int(_lib.dsa_prompt_attn_workspace_size(B, Nq, Hq, Hk, Dk, Dv))


def prompt_attn(q, k, v, sm_scale, out, lse, ws, cu_q=None, cu_k=None, stream=None):
    """Exact causal attention of packed prompts with grouped heads
    (include/dsa.h, dsa_prompt_attn): q [Nq, Hq, Dk], k [Nk, Hk, Dk],
    v [Nk, Hk, Dv] and out [Nq, Hq, Dv] bfloat16, strided; lse [Nq, Hq] float32
    or None.  cu_q, cu_k [B + 1] int32: where each sequence's tokens begin; only
    cu_q given: the keys are the same tokens; neither: one sequence."""
    dev = q.get_device()
    pq, Nq, Hq, Dk = _strided(q, "q", dev)
    pk, Nk, Hk, dk = _strided(k, "k", dev)
    pv, nv, hv, Dv = _strided(v, "v", dev)
    po, no, ho, do = _strided(out, "out", dev)
    if dk != Dk:
        raise ValueError(f"k: heads of {dk}; q has heads of {Dk}")
    if nv != Nk or hv != Hk:
        raise ValueError(f"v: {(nv, hv)} tokens and heads; k has {(Nk, Hk)}")
    if no != Nq or ho != Hq or do != Dv:
        raise ValueError(f"out: {(no, ho, do)}; the call writes {(Nq, Hq, Dv)}")
    if cu_q is None and cu_k is not None:
        raise ValueError("cu_q: required with cu_k")
    B = 1
    if cu_q is not None:
        if cu_k is None:
            if Nk != Nq:
                raise ValueError(f"cu_k: required, q has {Nq} tokens and k {Nk}")
            cu_k = cu_q
        B = cu_q.numel() - 1
        if B < 1:
            raise ValueError("cu_q: the beginning of each sequence and the end of the last are required")
    pc = (_vec(cu_q, "cu_q", torch.int32, B + 1, dev), _vec(cu_k, "cu_k", torch.int32, B + 1, dev))
    pl, pw = _vec(lse, "lse", torch.float32, Nq * Hq, dev), _vec(ws, "ws", torch.uint8, 0, dev)
    _on_gpu(dev, "q")
    rc = _lib.dsa_prompt_attn(*pq, *pk, *pv, *pc, B, Nq, Nk, Hq, Hk, Dk, Dv, sm_scale, *po, pl, pw,
                              ws.numel(), _here(dev, stream))
    if rc:
        raise DsaError(rc, "dsa_prompt_attn")


# ------------------------------------------------------------ 4-bit cache --
def cache4_row_bytes(Dk, Dv) -> int:
    """Bytes of a row of the 4-bit pool (one position of one key head)."""
    n = _row_bytes.get((Dk, Dv))
    if n is None:
        n = int(_lib.dsa_cache4_row_bytes(Dk, Dv))
        if n == 0:
            raise ValueError(f"head dims {Dk} / {Dv}: multiples of 16 up to 256 are taken")
        _row_bytes[(Dk, Dv)] = n
    return n


_row_bytes = {}  # of the dims met so far


def cache4_pool(num_blocks, heads, block_size, Dk, Dv, device=None) -> torch.Tensor:
    """A zero-filled 4-bit pool [num_blocks, heads, block_size, row bytes]."""
    return torch.zeros((num_blocks, heads, block_size, cache4_row_bytes(Dk, Dv)), dtype=torch.uint8,
                       device=device or "cuda")


def _pool4(layout: PagedLayout, pool, Dk: int, Dv: int, dev: int):
    """(address, heads) of a 4-bit pool, checked against the layout's pages."""
    shape, row = pool.shape, cache4_row_bytes(Dk, Dv)
    if len(shape) != 4 or shape[2] != layout.block_size or shape[3] != row:
        raise ValueError(f"pool: [num_blocks, heads, {layout.block_size}, {row}] is required, not {tuple(shape)}")
    if shape[0] < layout.num_blocks:
        raise ValueError(f"pool: {shape[0]} pages; the layout has {layout.num_blocks}")
    return _vec(pool, "pool", torch.uint8, 0, dev), shape[1]


def cache4_write_workspace_size() -> int:
    return int(_lib.dsa_cache4_write_workspace_size())


def cache4_write(layout: PagedLayout, seq, pos, k, v, pool, ws, k_scale=None, v_scale=None, k_out=None,
                 v_out=None, stream=None):
    """Store new tokens' K [N, Hk, Dk] and V [N, Hk, Dv] (bf16, strided) in the
    4-bit pool (include/dsa.h, dsa_cache4_write).  seq, pos [N] int32, or both
    None: token i is position seq_lens[i] - 1 of sequence i.  k_scale, v_scale
    [Hk] float32 or None; k_out, v_out: the values that the cache keeps, bf16."""
    dev = k.get_device()
    pk, N, Hk, Dk = _strided(k, "k", dev)
    pv, nv, hv, Dv = _strided(v, "v", dev)
    if nv != N or hv != Hk:
        raise ValueError(f"v: {(nv, hv)} tokens and heads; k has {(N, Hk)}")
    pp, heads = _pool4(layout, pool, Dk, Dv, dev)
    if heads != Hk:
        raise ValueError(f"pool: {heads} heads; k has {Hk}")
    args = (_vec(k_scale, "k_scale", torch.float32, Hk, dev), _vec(v_scale, "v_scale", torch.float32, Hk, dev),
            pp, _vec(k_out, "k_out", torch.bfloat16, N * Hk * Dk, dev),
            _vec(v_out, "v_out", torch.bfloat16, N * Hk * Dv, dev), _vec(ws, "ws", torch.uint8, 0, dev))
    ps, po = _vec(seq, "seq", torch.int32, N, dev), _vec(pos, "pos", torch.int32, N, dev)
    _on_gpu(dev, "k", layout)
    rc = _lib.dsa_cache4_write(layout.c(), ps, po, N, *pk, *pv, Hk, Dk, Dv, *args,
                               ws.numel(), _here(dev, stream))
    if rc:
        raise DsaError(rc, "dsa_cache4_write")


def cache4_read_workspace_size() -> int:
    return int(_lib.dsa_cache4_read_workspace_size())


def cache4_read(layout: PagedLayout, seq, pos, pool, k_out, v_out, ws, k_scale=None, v_scale=None,
                stream=None):
    """The values of N positions of the 4-bit pool as bf16 heads k_out
    [N, Hk, Dk] and v_out [N, Hk, Dv] (include/dsa.h, dsa_cache4_read)."""
    dev = k_out.get_device()
    sk, sv = k_out.shape, v_out.shape
    if len(sk) != 3 or len(sv) != 3 or sk[0] != sv[0] or sk[1] != sv[1]:
        raise ValueError("k_out, v_out: [tokens, heads, dim] of the same tokens and heads are required")
    (N, Hk, Dk), Dv = sk, sv[2]
    pp, heads = _pool4(layout, pool, Dk, Dv, dev)
    if heads != Hk:
        raise ValueError(f"pool: {heads} heads; k_out has {Hk}")
    ps, po = _vec(seq, "seq", torch.int32, N, dev), _vec(pos, "pos", torch.int32, N, dev)
    args = (_vec(k_scale, "k_scale", torch.float32, Hk, dev), _vec(v_scale, "v_scale", torch.float32, Hk, dev),
            pp, _vec(k_out, "k_out", torch.bfloat16, 0, dev), _vec(v_out, "v_out", torch.bfloat16, 0, dev),
            _vec(ws, "ws", torch.uint8, 0, dev))
    _on_gpu(dev, "k_out", layout)
    rc = _lib.dsa_cache4_read(layout.c(), ps, po, N, Hk, Dk, Dv, *args, ws.numel(), _here(dev, stream))
    if rc:
        raise DsaError(rc, "dsa_cache4_read")


def cache4_attn_decode_workspace_size(B, Hq, Hk, Dk, Dv) -> int:
    return int(_lib.dsa_cache4_attn_decode_workspace_size(B, Hq, Hk, Dk, Dv))


def cache4_attn_decode(layout: PagedLayout, q, pool, sm_scale, out, lse, ws, k_scale=None, v_scale=None,
                       stream=None):
    """Exact attention of one query per sequence, q [B, Hq, Dk], over all its
    positions in the 4-bit pool (include/dsa.h, dsa_cache4_attn_decode); Hq a
    multiple of the pool's heads, out [B, Hq, Dv] bfloat16, lse float32 or
    None."""
    dev = q.get_device()
    sq, so = q.shape, out.shape
    if len(sq) != 3 or len(so) != 3 or sq[0] != so[0] or sq[1] != so[1]:
        raise ValueError("q, out: [sequences, heads, dim] of the same sequences and heads are required")
    (B, Hq, Dk), Dv = sq, so[2]
    if B != layout.batch:
        raise ValueError(f"q: {B} sequences; the layout has {layout.batch}")
    pp, Hk = _pool4(layout, pool, Dk, Dv, dev)
    pq, po = _vec(q, "q", torch.bfloat16, 0, dev), _vec(out, "out", torch.bfloat16, 0, dev)
    pl, pw = _vec(lse, "lse", torch.float32, B * Hq, dev), _vec(ws, "ws", torch.uint8, 0, dev)
    ks, vs = _vec(k_scale, "k_scale", torch.float32, Hk, dev), _vec(v_scale, "v_scale", torch.float32, Hk, dev)
    _on_gpu(dev, "q", layout)
    rc = _lib.dsa_cache4_attn_decode(layout.c(), pq, pp, Hq, Hk, Dk, Dv, ks, vs, sm_scale, po, pl, pw,
                                     ws.numel(), _here(dev, stream))
    if rc:
        raise DsaError(rc, "dsa_cache4_attn_decode")


def get_status(ws, clear: bool = True, stream=None) -> int:
    v = ctypes.c_int32(0)
    (pws,) = _Args().add(ws, "ws", _WS).ptrs()
    _check(_lib.dsa_get_status(pws, _stream(stream), ctypes.byref(v), int(clear)),
           "dsa_get_status")
    return int(v.value)


class Pipeline:
    """The three stages of one decode or prefill step with preallocated buffers.

    kind="decode": one query per sequence at position L_b - 1 (q [B, Hq, Dqk]).
    kind="prefill": Nq queries of sequence `prefill_seq` at positions q_pos (the
    indexer then shares key tiles across queries); prefill_seq=None scores
    queries of any sequences given by q_seq.
    Buffers (scores, idx, out, lse, workspaces) are allocated once through torch.
    """

    def __init__(self, layout: PagedLayout, *, kind: str, Nq: int, Hq: int, Dqk: int, Dv: int,
                 H_i: int, D_i: int, K: int, ld: Optional[int] = None, device="cuda",
                 prefill_seq: Optional[int] = 0):
        self.layout, self.kind, self.K = layout, kind, int(K)
        self.prefill_seq = prefill_seq
        self.Nq, self.Hq, self.Dqk, self.Dv = int(Nq), int(Hq), int(Dqk), int(Dv)
        # default row stride: the longest row rounded up to 4 scores, so that
        # every row starts on a 16-byte boundary (top-K then loads it with
        # 16-byte copies)
        self.ld = int(ld if ld is not None else (max(layout.max_seq_len, 1) + 3) // 4 * 4)
        self.scores = torch.empty((self.Nq, self.ld), dtype=torch.float32, device=device)
        self.idx = torch.empty((self.Nq, self.K), dtype=torch.int32, device=device)
        self.out = torch.empty((self.Nq, Hq, Dv), dtype=torch.bfloat16, device=device)
        self.lse = torch.empty((self.Nq, Hq), dtype=torch.float32, device=device)
        self.ws_index = workspace(index_score_workspace_size(self.Nq, H_i, D_i, self.ld), device)
        self.ws_topk = workspace(topk_workspace_size(self.Nq, self.ld, self.K), device)
        if kind == "decode":
            n = sparse_attn_decode_workspace_size(self.Nq, Hq, Dqk, Dv, self.K)
        else:
            n = sparse_attn_prefill_workspace_size(self.Nq, Hq, Dqk, Dv, self.K)
        self.ws_attn = workspace(n, device)

    def run(self, q, q_idx, w, kidx_pool, k_pool, v_pool, sm_scale, n_eligible=None, q_seq=None,
            q_pos=None, stream=None):
        if n_eligible is None:
            if self.kind != "decode":
                raise ValueError("prefill needs n_eligible (q_pos + 1)")
            n_eligible = self.layout.seq_lens
        if self.kind == "decode" or self.prefill_seq is None:
            index_score(self.layout, q_idx, w, kidx_pool, self.scores, self.ws_index, q_seq=q_seq,
                        q_pos=q_pos, stream=stream)
        else:
            index_score_prefill(self.layout, self.prefill_seq, q_idx, w, kidx_pool, self.scores,
                                self.ws_index, q_pos=q_pos, stream=stream)
        topk(self.scores, n_eligible, self.K, self.idx, self.ws_topk, stream=stream)
        if self.kind == "decode":
            sparse_attn_decode(self.layout, q, k_pool, v_pool, self.idx, sm_scale, self.out,
                               self.lse, self.ws_attn, stream=stream)
        else:
            sparse_attn_prefill(self.layout, q, k_pool, v_pool, self.idx, sm_scale, self.out,
                                self.lse, self.ws_attn, q_seq=q_seq, q_pos=q_pos, stream=stream)
        return self.out

    def status(self) -> int:
        return (get_status(self.ws_index) | get_status(self.ws_topk) | get_status(self.ws_attn))
