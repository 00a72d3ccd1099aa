"""Python binding of libstep5sa: the Step-5 sparse-indexer attention on GB300 (sm_103a).

Thin ctypes marshalling over the C ABI declared in ``include/step5_sparse_attn.h``:
each function takes torch tensors that already live on the GPU, passes their device
pointers and the current CUDA stream, and raises ``Step5Error`` on a non-OK status.
Every step of the computation runs in the library's kernels; there is no other path.
If the library has not been built, the first call raises.

Steps (TensorFold PR #903, "Step-5-Preview on one 256 GB Mac", CSA-indexer commit):
  step5_region_summarize  -- e4m3 summary of each completed 8-token region
  step5_index_score_topk  -- sum_h relu(e4m3(q_h) . summary) * w_h, top-k by (-score, id)
  step5_sparse_attn       -- attention over the picked regions plus the row's own region
  step5_sparse_attn_gated -- the same, followed by the per-head sigmoid output gate
  step5_indexer_front     -- decode front end: q/k norms, k/z cache write, summary on completion

The paged KV cache, in bf16 or 8 bits (``PagedCache``):
  step5_paged_plan        -- a step's pages, block tables, rows and regions, made on the GPU
  step5_kv_append, step5_kv_append_e4m3 -- rotate and append the rows' keys and values
  step5_paged_attn, step5_paged_attn_e4m3 -- causal (or sliding-window) attention over the pages
  step5_sparse_attn_paged, step5_sparse_attn_e4m3 -- step (4) over the pages
"""
from __future__ import annotations

import ctypes
import math
import os
from dataclasses import dataclass
from typing import Optional

import torch

from ._build import LIB, build  # noqa: F401

__all__ = [
    "Step5Error", "Geometry", "STEP5_GEOMETRY", "library_path", "load",
    "step5_region_summarize", "step5_index_score_topk", "step5_sparse_attn", "step5_sparse_attn_gated",
    "step5_indexer_front",
    "step5_index_score_topk_noalloc",
    "step5_index_score_topk_shard", "step5_merge_topk", "step5_sparse_attn_shard", "step5_attn_combine",
    "step5_merge_attend_shard",
    "RowsLayout", "step5_rows_layout_for", "HostRows", "step5_decode_step_host", "step5_set_host_copies",
    "step5_workspace_bytes", "step5_workspace_init", "step5_device_status",
    "step5_set_select_path", "step5_set_wait_polls", "step5_set_attention_path", "step5_select_path_for", "step5_set_prologue_overlap", "step5_set_check_only", "step5_decode_step", "step5_status_string", "step5_convert_bf16_to_e4m3",
    "Workspace", "decode_step",
    "Pages", "PagedCache", "PagedWorkspace", "step5_kv_append", "step5_kv_append_e4m3", "step5_paged_attn_e4m3",
    "step5_sparse_attn_e4m3", "step5_paged_workspace_bytes", "decode_step_paged",
    "step5_paged_attn", "step5_sparse_attn_paged", "PagedTable", "PagedRows", "step5_paged_plan",
]

STATUS = {0: "STEP5_OK", 1: "STEP5_ERR_INVALID_ARGUMENT", 2: "STEP5_ERR_UNSUPPORTED",
          3: "STEP5_ERR_WORKSPACE", 4: "STEP5_ERR_CUDA", 5: "STEP5_ERR_TIMEOUT"}
DEV_RANGE, DEV_TIMEOUT = 1, 2


class Step5Error(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str = ""):
        self.status = status
        super().__init__(f"{fn}: {STATUS.get(status, status)}" + (f" ({detail})" if detail else ""))


class Geometry(ctypes.Structure):
    _fields_ = [("num_q_heads", ctypes.c_int32), ("num_kv_groups", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("idx_heads", ctypes.c_int32),
                ("idx_dim", ctypes.c_int32), ("rope_dims", ctypes.c_int32),
                ("region_tokens", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("softmax_scale", ctypes.c_float)]

    @classmethod
    def step5(cls, **over) -> "Geometry":
        vals = dict(num_q_heads=32, num_kv_groups=4, head_dim=128, idx_heads=16, idx_dim=64,
                    rope_dims=32, region_tokens=8, top_k=512, softmax_scale=1.0 / math.sqrt(128.0))
        vals.update(over)
        return cls(**vals)

    @classmethod
    def of(cls, g) -> "Geometry":
        if isinstance(g, Geometry):
            return g
        return cls(g.num_q_heads, g.num_kv_groups, g.head_dim, g.idx_heads, g.idx_dim,
                   g.rope_dims, g.region_tokens, g.top_k, g.softmax_scale)


STEP5_GEOMETRY = Geometry.step5()

_lib = None


def library_path() -> str:
    return LIB


def load():
    """Loads libstep5sa.so (raises if it is missing: build it with ``build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB):
        raise RuntimeError(f"{LIB} is not built; run block_sparse_attention_step5_gb300.build() "
                           "(nvcc, sm_103a) first")
    lib = ctypes.CDLL(LIB)
    P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    G = ctypes.POINTER(Geometry)
    PG = ctypes.POINTER(Pages)
    sigs = {
        "step5_region_summarize": (i32, [G, i32, i32, i32, i32, P, P, P, P, P, P, P, P, P]),
        "step5_index_score_topk": (i32, [G, i32, i32, i32, i32, P, P, P, P, P, P, P, P, P, P, P,
                                         P, sz, P]),
        "step5_sparse_attn": (i32, [G, i32, i32, i32, P, P, P, P, P, P, P, P, P, sz, P]),
        "step5_sparse_attn_gated": (i32, [G, i32, i32, i32, P, P, P, P, P, P, P, P, P, P, sz, P]),
        "step5_indexer_front": (i32, [G, i32, i32, i32, i32, P, P, P, P, P, P, ctypes.c_float, P, P, P, P,
                                      P, P, P, P, P]),
        "step5_decode_step": (i32, [G, i32, i32, i32, i32, i32, P, P, P, P, P, P, P, P, P, P, P, P, P, P,
                                    P, P, P, P, sz, P]),
        "step5_index_score_topk_noalloc": (i32, [G, i32, i32, i32, i32, P, P, P, P, P, P, P, P, P,
                                                 P, P, P]),
        "step5_index_score_topk_shard": (i32, [G, i32, i32, i32, i32, i32, P, P, P, P, P, P, P, P, P,
                                               P, P, sz, P]),
        "step5_merge_topk": (i32, [G, i32, i32, P, P, P, P, P, P, P]),
        "step5_sparse_attn_shard": (i32, [G, i32, i32, i32, i32, P, P, P, P, P, P, P, P, P, sz, P]),
        "step5_attn_combine": (i32, [G, i32, i32, P, P, P, P]),
        "step5_merge_attend_shard": (i32, [G, i32, i32, i32, i32, i32, P, P, P, P, P, P, P, P, P, P, P, P, sz, P]),
        "step5_rows_layout_for": (i32, [G, i32, i32, ctypes.POINTER(RowsLayout)]),
        "step5_decode_step_host": (i32, [G, i32, i32, i32, i32, i32, P, P, P, P, P, P, P, P, P, P, P, P, P,
                                         P, sz, P]),
        "step5_kv_append": (i32, [G, PG, i32, i32, i32, i32, P, i64, P, i64, P, i64, P, P, P, P, P, P, P, P, P]),
        "step5_kv_append_e4m3": (i32, [G, PG, i32, i32, i32, i32, P, i64, P, i64, P, i64, P, P, P, P, P, P, P, P, P,
                                       P, P]),
        "step5_paged_attn_e4m3": (i32, [G, PG, i32, i32, i32, P, P, P, P, P, P, P, P, P, P, P, sz, P]),
        "step5_sparse_attn_e4m3": (i32, [G, PG, i32, i32, P, P, P, P, P, P, P, P, P, P, P, P, P, sz, P]),
        "step5_paged_attn": (i32, [G, PG, i32, i32, i32, P, i64, P, P, P, P, P, P, P, P, sz, P]),
        "step5_sparse_attn_paged": (i32, [G, PG, i32, i32, P, i64, P, P, P, P, P, P, P, P, P, P, sz, P]),
        "step5_paged_plan": (i32, [G, PG, i32, i32, P, P, P, P, P, P, P, P, P, P, P, P, P, P]),
        "step5_paged_workspace_bytes": (sz, [G]),
        "step5_workspace_bytes": (sz, [G, i32, i32]),
        "step5_workspace_init": (i32, [P, sz, P]),
        "step5_device_status": (i32, [ctypes.POINTER(ctypes.c_uint32), P]),
        "step5_set_select_path": (i32, [i32]),
        "step5_set_wait_polls": (ctypes.c_uint32, [ctypes.c_uint32]),
        "step5_set_attention_path": (i32, [i32]),
        "step5_set_prologue_overlap": (i32, [i32]),
        "step5_set_host_copies": (i32, [i32]),
        "step5_set_check_only": (i32, [i32]),
        "step5_select_path_for": (i32, [G, i32, i32, i32]),
        "step5_status_string": (ctypes.c_char_p, [i32]),
        "step5_convert_bf16_to_e4m3": (i32, [P, P, i64, P]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors passed to libstep5sa must be on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors passed to libstep5sa must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn: str, status: int):
    if status != 0:
        raise Step5Error(fn, status)


def _run(call):
    """Makes a call that has been checked and laid out: the C function's name and its arguments."""
    fn, args = call
    st = getattr(load(), fn)(*args)
    if st:
        raise Step5Error(fn, st)


def step5_status_string(status: int) -> str:
    return load().step5_status_string(status).decode()


def step5_set_select_path(mode: int) -> int:
    """0 = automatic, 1 = one block per (row, group), 2 = histogram split path, 3 =
    tensor-core scoring then one selecting block per (row, group)."""
    return load().step5_set_select_path(mode)


def step5_set_attention_path(mode: int) -> int:
    """Step (4) without a split: 0 = automatic, 1 = warp-level MMA kernel, 2 = tcgen05
    kernel; returns the previous value."""
    return load().step5_set_attention_path(mode)


def step5_set_wait_polls(polls: int) -> int:
    """Poll limit of the split selection path's waits on other blocks (0 = default);
    returns the previous limit."""
    return int(load().step5_set_wait_polls(polls))


def step5_set_prologue_overlap(enable: int) -> int:
    """1 = the scoring kernel reads its non-summary inputs before waiting for the launch
    before it (which must not write them); 0 = every read waits.  Returns the previous."""
    return load().step5_set_prologue_overlap(enable)


def step5_set_check_only(enable: int) -> int:
    """1: this thread's calls of a paged step (see the header) only check their arguments; 0 (default): they
    run.  Returns the previous value."""
    return load().step5_set_check_only(int(enable))


def step5_set_host_copies(always: int) -> int:
    """1: step5_decode_step_host always copies its host buffers; 0 (default): in place
    when they are device-addressable page-locked memory.  Returns the previous value."""
    return load().step5_set_host_copies(int(always))


def step5_select_path_for(geom, N: int, r_cap: int, B: int = None) -> int:
    """1 (fused), 2 (split) or 3 (tensor-core scoring, then selection) for N rows of B
    sequences (default: one row per sequence) and r_cap."""
    return load().step5_select_path_for(ctypes.byref(Geometry.of(geom)), N, N if B is None else B, r_cap)


def step5_workspace_bytes(geom, N: int, r_cap: int) -> int:
    return load().step5_workspace_bytes(ctypes.byref(Geometry.of(geom)), N, r_cap)


def step5_workspace_init(workspace: torch.Tensor, stream=None):
    _check("step5_workspace_init", load().step5_workspace_init(
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def step5_device_status(stream=None) -> int:
    """Reads and clears the device status word (synchronises the stream)."""
    v = ctypes.c_uint32(0)
    st = load().step5_device_status(ctypes.byref(v), _stream(stream))
    if st not in (0, 5):
        _check("step5_device_status", st)
    return v.value


def step5_convert_bf16_to_e4m3(x: torch.Tensor, out: torch.Tensor, stream=None):
    assert x.dtype == torch.bfloat16 and out.dtype == torch.uint8 and out.numel() == x.numel()
    _check("step5_convert_bf16_to_e4m3", load().step5_convert_bf16_to_e4m3(
        _ptr(x), _ptr(out), x.numel(), _stream(stream)))


def step5_region_summarize(geom, idx_k, idx_z, cos, sin, region_begin, region_end,
                           summaries, summaries_f32=None, max_regions_per_seq=None, stream=None):
    """idx_k/idx_z [B][G][t_cap][64] bf16, cos/sin [t_cap][rope/2] bf16 (or None),
    region_begin/end [B] int32, summaries [B][G][r_cap][64] uint8 (written)."""
    _run(_summarize_call(geom, idx_k, idx_z, cos, sin, region_begin, region_end, summaries, summaries_f32,
                         max_regions_per_seq, stream))


def _summarize_call(geom, idx_k, idx_z, cos, sin, region_begin, region_end, summaries, summaries_f32, max_regions_per_seq,
                    stream):
    B, G, t_cap, _ = idx_k.shape
    r_cap = summaries.shape[2]
    if max_regions_per_seq is None:
        max_regions_per_seq = r_cap
    return "step5_region_summarize", (
        ctypes.byref(Geometry.of(geom)), B, t_cap, r_cap, int(max_regions_per_seq), _ptr(idx_k), _ptr(idx_z), _ptr(cos), _ptr(sin),
        _ptr(region_begin), _ptr(region_end), _ptr(summaries), _ptr(summaries_f32), _stream(stream))


def step5_index_score_topk(geom, idx_q, w, row_seq, row_pos, cos, sin, summaries, sel_ids,
                           sel_count, workspace, t_cap, scores=None, sel_scores=None, stream=None):
    """idx_q [N][idx_heads][64] bf16, w [N][idx_heads] fp32, row_seq/row_pos [N] int32,
    summaries [B][G][r_cap][64] uint8; writes sel_ids [N][G][top_k], sel_count [N][G]."""
    _run(_score_call(geom, idx_q, w, row_seq, row_pos, cos, sin, summaries, sel_ids, sel_count, workspace, t_cap, scores,
                     sel_scores, stream))


def _score_call(geom, idx_q, w, row_seq, row_pos, cos, sin, summaries, sel_ids, sel_count, workspace, t_cap, scores, sel_scores,
                stream):
    N = idx_q.shape[0]
    B, _, r_cap, _ = summaries.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return "step5_index_score_topk", (
        ctypes.byref(Geometry.of(geom)), N, B, int(t_cap), r_cap, _ptr(idx_q), _ptr(w), _ptr(row_seq), _ptr(row_pos), _ptr(cos),
        _ptr(sin), _ptr(summaries), _ptr(sel_ids), _ptr(sel_count), _ptr(scores), _ptr(sel_scores), _ptr(workspace), ws_bytes,
        _stream(stream))


def step5_index_score_topk_noalloc(geom, idx_q, w, row_seq, row_pos, cos, sin, summaries, sel_ids,
                                   sel_count, t_cap, scores=None, sel_scores=None, stream=None):
    """step5_index_score_topk with the library's fixed static scratch (about 6.1 MiB: 4 MiB
    for this call's own scratch after the ~2.1 MiB any workspace keeps for step (4))
    instead of a caller workspace, for callers that cannot allocate device memory (see
    the header for the size limit and the sharing rules)."""
    N = idx_q.shape[0]
    B, _, r_cap, _ = summaries.shape
    _check("step5_index_score_topk_noalloc", load().step5_index_score_topk_noalloc(
        ctypes.byref(Geometry.of(geom)), N, B, int(t_cap), r_cap, _ptr(idx_q), _ptr(w),
        _ptr(row_seq), _ptr(row_pos), _ptr(cos), _ptr(sin), _ptr(summaries), _ptr(sel_ids),
        _ptr(sel_count), _ptr(scores), _ptr(sel_scores), _stream(stream)))


def step5_indexer_front(geom, q_pre, k_pre, z_pre, q_norm_w, k_norm_w, k_norm_b, eps, row_seq, row_pos,
                        cos, sin, idx_q_out, idx_k, idx_z, summaries, stream=None):
    """The indexer's decode front end: q RMSNorm (1 + w) into idx_q_out, k LayerNorm and z
    written at each row's position of the caches, and the summary of a region the row's
    token completes (see the header)."""
    N = q_pre.shape[0]
    B, _, t_cap, _ = idx_k.shape
    r_cap = summaries.shape[2]
    _check("step5_indexer_front", load().step5_indexer_front(
        ctypes.byref(Geometry.of(geom)), N, B, t_cap, r_cap, _ptr(q_pre), _ptr(k_pre), _ptr(z_pre),
        _ptr(q_norm_w), _ptr(k_norm_w), _ptr(k_norm_b), float(eps), _ptr(row_seq), _ptr(row_pos),
        _ptr(cos), _ptr(sin), _ptr(idx_q_out), _ptr(idx_k), _ptr(idx_z), _ptr(summaries), _stream(stream)))


def step5_sparse_attn_gated(geom, q, k_cache, v_cache, row_seq, row_pos, sel_ids, sel_count, gate,
                            out, workspace, stream=None):
    """step5_sparse_attn followed by the per-head sigmoid output gate: gate [N][Hq] bf16
    logits; every dim of head h of row n is scaled by sigmoid(gate[n][h]) before the
    output's rounding."""
    N = q.shape[0]
    B, _, t_cap, _ = k_cache.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("step5_sparse_attn_gated", load().step5_sparse_attn_gated(
        ctypes.byref(Geometry.of(geom)), N, B, t_cap, _ptr(q), _ptr(k_cache), _ptr(v_cache),
        _ptr(row_seq), _ptr(row_pos), _ptr(sel_ids), _ptr(sel_count), _ptr(gate), _ptr(out),
        _ptr(workspace), ws_bytes, _stream(stream)))


def step5_sparse_attn(geom, q, k_cache, v_cache, row_seq, row_pos, sel_ids, sel_count, out,
                      workspace, stream=None):
    """q [N][Hq][128] bf16, k/v cache [B][G][t_cap][128] bf16 -> out [N][Hq][128] bf16."""
    N = q.shape[0]
    B, _, t_cap, _ = k_cache.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("step5_sparse_attn", load().step5_sparse_attn(
        ctypes.byref(Geometry.of(geom)), N, B, t_cap, _ptr(q), _ptr(k_cache), _ptr(v_cache),
        _ptr(row_seq), _ptr(row_pos), _ptr(sel_ids), _ptr(sel_count), _ptr(out), _ptr(workspace),
        ws_bytes, _stream(stream)))


def step5_index_score_topk_shard(geom, idx_q, w, row_seq, row_pos, cos, sin, summaries, region_lo,
                                 sel_ids, sel_count, sel_scores, workspace, t_cap, stream=None):
    """Scoring and top-k of one sequence shard: summaries [B][G][r_cap_local][64] hold
    regions region_lo .. region_lo + r_cap_local - 1; writes the shard's pick with the
    rows' region ids, sel_scores required."""
    N = idx_q.shape[0]
    B, _, r_cap, _ = summaries.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("step5_index_score_topk_shard", load().step5_index_score_topk_shard(
        ctypes.byref(Geometry.of(geom)), N, B, int(t_cap), r_cap, int(region_lo), _ptr(idx_q), _ptr(w),
        _ptr(row_seq), _ptr(row_pos), _ptr(cos), _ptr(sin), _ptr(summaries), _ptr(sel_ids),
        _ptr(sel_count), _ptr(sel_scores), _ptr(workspace), ws_bytes, _stream(stream)))


def step5_merge_topk(geom, shard_ids, shard_scores, shard_counts, sel_ids, sel_count, sel_scores=None,
                     stream=None):
    """The rows' pick from S shards' picks: shard_ids / shard_scores [S][N][G][top_k],
    shard_counts [S][N][G] -> sel_ids [N][G][top_k], sel_count [N][G] (+ sel_scores)."""
    S, N = shard_ids.shape[0], shard_ids.shape[1]
    _check("step5_merge_topk", load().step5_merge_topk(
        ctypes.byref(Geometry.of(geom)), S, N, _ptr(shard_ids), _ptr(shard_scores), _ptr(shard_counts),
        _ptr(sel_ids), _ptr(sel_count), _ptr(sel_scores), _stream(stream)))


def step5_sparse_attn_shard(geom, q, k_cache, v_cache, token_lo, row_seq, row_pos, sel_ids, sel_count,
                            states, workspace, stream=None):
    """Attention of one sequence shard: k/v cache [B][G][t_cap_local][128] hold tokens
    token_lo .. token_lo + t_cap_local - 1; writes states [N][Hq][130] fp32 (m, l, o)."""
    N = q.shape[0]
    B, _, t_cap, _ = k_cache.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("step5_sparse_attn_shard", load().step5_sparse_attn_shard(
        ctypes.byref(Geometry.of(geom)), N, B, t_cap, int(token_lo), _ptr(q), _ptr(k_cache), _ptr(v_cache),
        _ptr(row_seq), _ptr(row_pos), _ptr(sel_ids), _ptr(sel_count), _ptr(states), _ptr(workspace),
        ws_bytes, _stream(stream)))


def step5_merge_attend_shard(geom, shard_ids, shard_scores, shard_counts, q, k_cache, v_cache, token_lo, row_seq,
                             row_pos, sel_ids, sel_count, states, workspace, stream=None):
    """The merge of S shards' picks [S][N][G][K] into sel_ids/sel_count, then this shard's
    attention states [N][Hq][130], in one call (see the header)."""
    S, N = shard_ids.shape[0], shard_ids.shape[1]
    B, _, t_cap, _ = k_cache.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("step5_merge_attend_shard", load().step5_merge_attend_shard(
        ctypes.byref(Geometry.of(geom)), S, N, B, t_cap, int(token_lo), _ptr(shard_ids), _ptr(shard_scores),
        _ptr(shard_counts), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(row_seq), _ptr(row_pos), _ptr(sel_ids),
        _ptr(sel_count), _ptr(states), _ptr(workspace), ws_bytes, _stream(stream)))


def step5_attn_combine(geom, states, out, gate=None, stream=None):
    """The output from S shards' states [S][N][Hq][130] -> out [N][Hq][128] bf16 (with the
    per-head sigmoid gate [N][Hq] when given)."""
    S, N = states.shape[0], states.shape[1]
    _check("step5_attn_combine", load().step5_attn_combine(
        ctypes.byref(Geometry.of(geom)), S, N, _ptr(states), _ptr(gate), _ptr(out), _stream(stream)))


def step5_decode_step(geom, t: dict, ws, sel_ids, sel_count, out, max_regions_per_seq, stream=None):
    """The whole step in one C-ABI call (summaries of [sum_begin, sum_end), score +
    select, attention), over the tensors of ``t`` (keys as produced by the synthetic
    workload module).  Same results as the three calls."""
    B, G, t_cap, _ = t["idx_k"].shape
    r_cap = t["summaries"].shape[2]
    N = t["idx_q"].shape[0]
    ws_t = None if ws is None else (ws.tensor if isinstance(ws, Workspace) else ws)
    ws_bytes = 0 if ws_t is None else ws_t.numel() * ws_t.element_size()
    _check("step5_decode_step", load().step5_decode_step(
        ctypes.byref(Geometry.of(geom)), N, B, t_cap, r_cap, int(max_regions_per_seq),
        _ptr(t["idx_k"]), _ptr(t["idx_z"]), _ptr(t["cos"]), _ptr(t["sin"]), _ptr(t["sum_begin"]),
        _ptr(t["sum_end"]), _ptr(t["summaries"]), _ptr(t["idx_q"]), _ptr(t["w"]), _ptr(t["row_seq"]),
        _ptr(t["row_pos"]), _ptr(t["q"]), _ptr(t["k_cache"]), _ptr(t["v_cache"]), _ptr(sel_ids),
        _ptr(sel_count), _ptr(out), _ptr(ws_t), ws_bytes, _stream(stream)))


class RowsLayout(ctypes.Structure):
    """Byte offsets of a step's per-row inputs packed in one buffer (step5_rows_layout_for)."""
    _fields_ = [(n, ctypes.c_size_t) for n in
                ("q", "idx_q", "w", "row_seq", "row_pos", "region_begin", "region_end", "total")]


def step5_rows_layout_for(geom, N: int, B: int) -> RowsLayout:
    lay = RowsLayout()
    _check("step5_rows_layout_for", load().step5_rows_layout_for(ctypes.byref(Geometry.of(geom)), N, B,
                                                                 ctypes.byref(lay)))
    return lay


class HostRows:
    """A decode step's per-row inputs packed in one page-locked host buffer (filled by the
    caller through ``view``) and its device copy, plus the page-locked output; the buffers
    that step5_decode_step_host takes."""

    def __init__(self, geom, N: int, B: int, device="cuda"):
        g = Geometry.of(geom)
        self.N, self.B = N, B
        self.layout = step5_rows_layout_for(geom, N, B)
        self.host = torch.zeros(self.layout.total, dtype=torch.uint8, pin_memory=True)
        self.dev = torch.zeros(self.layout.total, dtype=torch.uint8, device=device)
        self.out_host = torch.zeros((N, g.num_q_heads, g.head_dim), dtype=torch.bfloat16, pin_memory=True)
        self.out_dev = torch.zeros((N, g.num_q_heads, g.head_dim), dtype=torch.bfloat16, device=device)
        self._shapes = {"q": ((N, g.num_q_heads, g.head_dim), torch.bfloat16),
                        "idx_q": ((N, g.idx_heads, g.idx_dim), torch.bfloat16),
                        "w": ((N, g.idx_heads), torch.float32), "row_seq": ((N,), torch.int32),
                        "row_pos": ((N,), torch.int32), "region_begin": ((B,), torch.int32),
                        "region_end": ((B,), torch.int32)}

    def view(self, name: str, on_device: bool = False) -> torch.Tensor:
        """The array ``name`` of the packed buffer (host, or its device copy)."""
        shape, dtype = self._shapes[name]
        off = getattr(self.layout, name)
        nbytes = math.prod(shape) * torch.tensor([], dtype=dtype).element_size()
        buf = self.dev if on_device else self.host
        return buf[off:off + nbytes].view(dtype).view(shape)

    @property
    def h2d_bytes(self) -> int:
        return int(self.layout.total)

    @property
    def d2h_bytes(self) -> int:
        return self.out_host.numel() * self.out_host.element_size()


def _hptr(t: torch.Tensor):
    if t.is_cuda or not t.is_contiguous():
        raise ValueError("host buffers passed to libstep5sa must be contiguous CPU tensors")
    return ctypes.c_void_p(t.data_ptr())


def step5_decode_step_host(geom, t: dict, ws, rows: HostRows, sel_ids, sel_count, max_regions_per_seq,
                           stream=None):
    """The whole step from host inputs to host output in one C-ABI call: the step runs
    over rows.host's arrays (in place when the device can address them, else copied to
    rows.dev) and the device caches, summaries and tables of ``t``; the output lands in
    rows.out_host (valid after the stream reaches the end of the call's work)."""
    B, G, t_cap, _ = t["idx_k"].shape
    r_cap = t["summaries"].shape[2]
    ws_t = None if ws is None else (ws.tensor if isinstance(ws, Workspace) else ws)
    ws_bytes = 0 if ws_t is None else ws_t.numel() * ws_t.element_size()
    _check("step5_decode_step_host", load().step5_decode_step_host(
        ctypes.byref(Geometry.of(geom)), rows.N, B, t_cap, r_cap, int(max_regions_per_seq),
        _ptr(t["idx_k"]), _ptr(t["idx_z"]), _ptr(t["cos"]), _ptr(t["sin"]), _ptr(t["summaries"]),
        _ptr(t["k_cache"]), _ptr(t["v_cache"]), _hptr(rows.host), _ptr(rows.dev), _hptr(rows.out_host),
        _ptr(rows.out_dev), _ptr(sel_ids), _ptr(sel_count), _ptr(ws_t), ws_bytes, _stream(stream)))


@dataclass
class Workspace:
    """Device workspace for N rows and r_cap summary slots, zeroed once on creation."""
    tensor: torch.Tensor

    @classmethod
    def create(cls, geom, N: int, r_cap: int, device="cuda") -> "Workspace":
        nbytes = step5_workspace_bytes(geom, N, r_cap)
        if nbytes == 0:
            raise Step5Error("step5_workspace_bytes", 2, "unsupported geometry")
        t = torch.empty(nbytes, dtype=torch.uint8, device=device)
        step5_workspace_init(t)
        return cls(t)


def decode_step(geom, t: dict, ws: Workspace, sel_ids, sel_count, out, max_regions_per_seq,
                summarize: bool = True, stream=None):
    """One pass of the whole path over the tensors of ``t`` (keys as produced by the
    synthetic workload module): summarise [sum_begin, sum_end), score + select, attend."""
    if summarize:
        step5_region_summarize(geom, t["idx_k"], t["idx_z"], t["cos"], t["sin"], t["sum_begin"],
                               t["sum_end"], t["summaries"],
                               max_regions_per_seq=max_regions_per_seq, stream=stream)
    # the launch just before the scoring call is the summary kernel (or, without it, the
    # previous step's attention), which writes none of the scoring inputs but summaries
    prev = step5_set_prologue_overlap(1 if summarize else 0)
    try:
        step5_index_score_topk(geom, t["idx_q"], t["w"], t["row_seq"], t["row_pos"], t["cos"],
                               t["sin"], t["summaries"], sel_ids, sel_count, ws.tensor,
                               t_cap=t["idx_k"].shape[2], stream=stream)
    finally:
        step5_set_prologue_overlap(prev)
    step5_sparse_attn(geom, t["q"], t["k_cache"], t["v_cache"], t["row_seq"], t["row_pos"],
                      sel_ids, sel_count, out, ws.tensor, stream=stream)


class Pages(ctypes.Structure):
    """Shape of a paged pool (step5_pages)."""
    _fields_ = [("num_pages", ctypes.c_int32), ("page_tokens", ctypes.c_int32), ("table_len", ctypes.c_int32)]


class PagedCache:
    """A paged KV cache: pools ``k``, ``v`` [num_pages][G][page_tokens][128] (bf16, or uint8
    e4m3 codes with fp32 ``k_scales``, ``v_scales`` [num_pages][G][page_tokens / 8]) and the
    int32 ``block_table`` [B][table_len] of page numbers.  ``block_table`` None: sequence b owns
    page b, so that contiguous caches [B][G][t_cap][128] are a PagedCache as they are.  The
    tensors belong to the caller, who may change the table's entries between calls, or assign
    another tensor to an attribute (checked again then); what follows from them is read-only."""

    _TENSORS = ("k", "v", "block_table", "k_scales", "v_scales")
    _FOLLOWS = ("e4m3", "B", "pages", "groups", "head_dim", "device", "_index", "_shape", "_pages", "_pools")

    def __init__(self, k: torch.Tensor, v: torch.Tensor, block_table: Optional[torch.Tensor] = None,
                 k_scales: Optional[torch.Tensor] = None, v_scales: Optional[torch.Tensor] = None):
        self._lay_out(k, v, block_table, k_scales, v_scales)

    def __setattr__(self, name, value):
        if name in self._TENSORS:
            self._lay_out(*(value if n == name else getattr(self, n) for n in self._TENSORS))
        elif name in self._FOLLOWS:
            raise AttributeError(f"{name} of a PagedCache follows from its tensors")
        else:
            super().__setattr__(name, value)

    def _lay_out(self, k, v, block_table, k_scales, v_scales):
        """Checks the tensors, and lays out the C calls' arguments, which stay the same as long as the tensors do."""
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype:
            raise ValueError("k and v must be pools [num_pages][G][page_tokens][128] of one shape and type")
        if k.dtype not in (torch.bfloat16, torch.uint8):
            raise ValueError("pools are bf16 or e4m3 codes (uint8)")
        e4m3 = k.dtype == torch.uint8
        pages, groups, tokens, head_dim = k.shape
        want = (pages, groups, tokens // 8)
        for s in (k_scales, v_scales):
            if e4m3 != (s is not None):
                raise ValueError("e4m3 pools come with k_scales and v_scales, bf16 pools without")
            if s is not None and (tuple(s.shape) != want or s.dtype != torch.float32):
                raise ValueError(f"scales must be fp32 {want}")
        if block_table is not None and (block_table.dim() != 2 or block_table.dtype != torch.int32):
            raise ValueError("block_table must be int32 [B][table_len]")
        tensors = (k, v, block_table, k_scales, v_scales)
        for t in tensors:
            if t is not None and t.device != k.device:
                raise ValueError(f"the cache's tensors are on {k.device} and {t.device}")
        if not all(t is None or t.is_contiguous() for t in tensors):
            raise ValueError("the cache's tensors must be contiguous")
        shape = Pages(pages, tokens, 1 if block_table is None else block_table.shape[1])
        pools = (k, v, k_scales, v_scales, block_table) if e4m3 else (k, v, block_table)
        self.__dict__.update(zip(self._TENSORS, tensors))
        self.__dict__.update(e4m3=e4m3, B=pages if block_table is None else block_table.shape[0], groups=groups,
                             head_dim=head_dim, device=k.device, _index=k.device.index if k.is_cuda else -1,
                             _shape=shape, _pages=ctypes.byref(shape),
                             _pools=tuple(None if t is None else t.data_ptr() for t in pools))

    @property
    def pages(self) -> Pages:
        return Pages.from_buffer_copy(self._shape)

    @classmethod
    def create(cls, geom, num_pages: int, page_tokens: int, block_table: torch.Tensor, e4m3: bool = True,
               device="cuda") -> "PagedCache":
        """An empty cache (codes 0, scales 1)."""
        g = Geometry.of(geom)
        shape = (num_pages, g.num_kv_groups, page_tokens, g.head_dim)
        k, v = (torch.zeros(shape, dtype=torch.uint8 if e4m3 else torch.bfloat16, device=device) for _ in range(2))
        if not e4m3:
            return cls(k, v, block_table)
        ks, vs = (torch.ones((num_pages, g.num_kv_groups, page_tokens // 8), dtype=torch.float32, device=device)
                  for _ in range(2))
        return cls(k, v, block_table, ks, vs)


def step5_paged_workspace_bytes(geom) -> int:
    return load().step5_paged_workspace_bytes(ctypes.byref(Geometry.of(geom)))


@dataclass
class PagedWorkspace:
    """Device workspace of the attention calls over pages (it may hold anything)."""
    tensor: torch.Tensor

    @classmethod
    def create(cls, geom, device="cuda") -> "PagedWorkspace":
        nbytes = step5_paged_workspace_bytes(geom)
        if nbytes == 0:
            raise Step5Error("step5_paged_workspace_bytes", 2, "unsupported geometry")
        return cls(torch.empty(nbytes, dtype=torch.uint8, device=device))


def _raise_for(what: str, t, dtype, shape, dev: int):
    """Says what is wrong with a tensor argument that _arg or _rows has turned down."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{what} must be a tensor, got {type(t).__name__}")
    if not t.is_cuda:
        raise ValueError(f"{what}: tensors passed to libstep5sa must be on the GPU")
    if t.get_device() != dev:
        raise ValueError(f"{what} is on {t.device}, the current device is cuda:{dev}")
    if t.dtype != dtype or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must be {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    raise ValueError(f"{what}: tensors passed to libstep5sa must be contiguous (of q, k and v the heads of each row)")


def _arg(what: str, t, dtype, shape, dev: int) -> int:
    """Address of a dense tensor of this type and shape on the current device."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _raise_for(what, t, dtype, shape, dev)


def _rows(what: str, t, heads: int, dim: int, dev: int, N: int):
    """Address and row stride of a bf16 [N][heads][dim] tensor whose rows may lie apart."""
    shape = (N, heads, dim)
    try:
        if t.dtype is torch.bfloat16 and t.shape == shape and t.get_device() == dev:
            row, head, one = t.stride()
            if one == 1 and (head == dim or heads == 1):
                return t.data_ptr(), (row if N > 1 else heads * dim)
    except AttributeError:
        pass
    _raise_for(what, t, torch.bfloat16, shape, dev)


# the current stream's handle without a Stream object around it (1 us of a 7 us call), and the current device without
# looking whether CUDA is up (a tensor of the cache is there), where torch offers that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _device_and_stream(cache: "PagedCache", geom, stream):
    """Current device and the stream's handle, after checking that the cache is there and fits the geometry."""
    dev = _current_device() if cache._index >= 0 else torch.cuda.current_device()
    if cache._index != dev:
        raise ValueError(f"the cache is on {cache.device}, the current device is cuda:{dev}")
    if cache.groups != geom.num_kv_groups or cache.head_dim != geom.head_dim:
        raise ValueError("the cache's groups and head dim are not the geometry's")
    if stream is not None:
        return dev, stream.cuda_stream
    return dev, (_raw_stream(dev) if _raw_stream else torch.cuda.current_stream(dev).cuda_stream)


def _append_call(fn: str, e4m3: bool, geom, k, v, cache: PagedCache, row_seq, row_pos, cos, sin, q, q_out, stream):
    g = Geometry.of(geom)
    dev, st = _device_and_stream(cache, g, stream)
    if cache.e4m3 != e4m3:
        raise ValueError(f"{fn} does not write this kind of pool")
    G, D, N = cache.groups, cache.head_dim, k.shape[0]
    kp, ks = _rows("k", k, G, D, dev, N)
    vp, vs = _rows("v", v, G, D, dev, N)
    qp, qs, qo = None, 0, None
    if q is not None or q_out is not None:
        Hq = g.num_q_heads
        qp, qs = _rows("q", q, Hq, D, dev, N)
        qo = _arg("q_out", q_out, torch.bfloat16, (N, Hq, D), dev)
    cp, sp, t_cap, half = None, None, 1, 0
    if cos is not None or sin is not None:
        table = cos.shape if isinstance(cos, torch.Tensor) and cos.dim() == 2 else ()
        cp = _arg("cos", cos, torch.bfloat16, table, dev)
        sp = _arg("sin", sin, torch.bfloat16, table, dev)
        t_cap, half = table
    rows = (N,)
    return fn, (g, cache._pages, N, cache.B, 2 * half, t_cap, qp, qs, kp, ks, vp, vs,
                _arg("row_seq", row_seq, torch.int32, rows, dev), _arg("row_pos", row_pos, torch.int32, rows, dev), cp, sp, qo,
                *cache._pools, st)


def step5_kv_append(geom, k, v, cache: PagedCache, row_seq, row_pos, cos=None, sin=None, q=None, q_out=None,
                    stream=None):
    """Rotates the rows' k [N][G][128] (cos/sin [t_cap][rot / 2] bf16; None: no rotation) and
    writes it and v into the bf16 cache at (row_seq, row_pos) [N] int32; with q
    [N][Hq][128], its rotation into q_out.  q, k and v may be slices of one [N][heads][128]
    tensor (rows apart, heads together)."""
    _run(_append_call("step5_kv_append", False, geom, k, v, cache, row_seq, row_pos, cos, sin, q, q_out, stream))


def step5_kv_append_e4m3(geom, k, v, cache: PagedCache, row_seq, row_pos, cos=None, sin=None, q=None, q_out=None,
                         stream=None):
    """step5_kv_append into an e4m3 cache: codes and the power-of-two scale of each region
    and group.  A sequence's rows stand together at ascending positions (see the header)."""
    _run(_append_call("step5_kv_append_e4m3", True, geom, k, v, cache, row_seq, row_pos, cos, sin, q, q_out, stream))


def _attend_call(fn: str, e4m3: bool, geom, q, cache: PagedCache, row_seq, row_pos, out, ws, gate, stream, window=None,
                 sel_ids=None, sel_count=None):
    g = Geometry.of(geom)
    dev, st = _device_and_stream(cache, g, stream)
    if cache.e4m3 != e4m3:
        raise ValueError(f"{fn} reads {'e4m3' if e4m3 else 'bf16'} pools")
    N, Hq = q.shape[0], g.num_q_heads
    shape = (N, Hq, g.head_dim)
    w = ws.tensor if isinstance(ws, PagedWorkspace) else ws
    if w is not None and (w.get_device() != dev or not w.is_contiguous()):
        _raise_for("workspace", w, w.dtype, w.shape, dev)
    if window is None:
        before = ()
        after = (_arg("sel_ids", sel_ids, torch.int32, (N, g.num_kv_groups, g.top_k), dev),
                 _arg("sel_count", sel_count, torch.int32, (N, g.num_kv_groups), dev))
    else:
        before, after = (window,), ()
    rows = (_arg("q", q, torch.bfloat16, shape, dev),) if e4m3 else _rows("q", q, Hq, g.head_dim, dev, N)
    return fn, (g, cache._pages, N, cache.B, *before, *rows, *cache._pools, _arg("row_seq", row_seq, torch.int32, (N,), dev),
                _arg("row_pos", row_pos, torch.int32, (N,), dev), *after,
                None if gate is None else _arg("gate", gate, torch.bfloat16, (N, Hq), dev),
                _arg("out", out, torch.bfloat16, shape, dev), None if w is None else w.data_ptr(), 0 if w is None else w.nbytes, st)


def _window(window) -> int:
    return max(-1, min(int(window), 2 ** 31 - 1))  # (within the C call's 32 bits)


def step5_paged_attn_e4m3(geom, q, cache: PagedCache, row_seq, row_pos, out, workspace, window: int = 0, gate=None,
                          stream=None):
    """Causal attention of rows q [N][Hq][128] bf16 at (row_seq, row_pos) over the e4m3
    cache's tokens max(0, pos - window + 1) .. pos (window 0: all) -> out, with the per-head
    sigmoid gate [N][Hq] when given."""
    _run(_attend_call("step5_paged_attn_e4m3", True, geom, q, cache, row_seq, row_pos, out, workspace, gate, stream,
                      window=_window(window)))


def step5_paged_attn(geom, q, cache: PagedCache, row_seq, row_pos, out, workspace, window: int = 0, gate=None,
                     stream=None):
    """step5_paged_attn_e4m3 over the bf16 cache.  q may be a slice of one [N][heads][128]
    tensor (rows apart, heads together)."""
    _run(_attend_call("step5_paged_attn", False, geom, q, cache, row_seq, row_pos, out, workspace, gate, stream,
                      window=_window(window)))


def step5_sparse_attn_e4m3(geom, q, cache: PagedCache, row_seq, row_pos, sel_ids, sel_count, out, workspace,
                           gate=None, stream=None):
    """step5_sparse_attn over the e4m3 cache: the picked regions sel_ids [N][G][top_k],
    sel_count [N][G] and the row's own region."""
    _run(_attend_call("step5_sparse_attn_e4m3", True, geom, q, cache, row_seq, row_pos, out, workspace, gate, stream,
                      sel_ids=sel_ids, sel_count=sel_count))


def step5_sparse_attn_paged(geom, q, cache: PagedCache, row_seq, row_pos, sel_ids, sel_count, out, workspace,
                            gate=None, stream=None):
    """step5_sparse_attn over the bf16 cache's pages, as step5_sparse_attn_e4m3 over the e4m3
    ones.  q as in step5_paged_attn."""
    _run(_attend_call("step5_sparse_attn_paged", False, geom, q, cache, row_seq, row_pos, out, workspace, gate, stream,
                      sel_ids=sel_ids, sel_count=sel_count))


class _Int32s:
    """A handle of int32 GPU tensors, checked and laid out for the C call once, and again when one is assigned."""

    def __setattr__(self, name, value):
        if name in self._TENSORS:
            self._lay_out(*(value if n == name else getattr(self, n) for n in self._TENSORS))
        elif name in self._FOLLOWS:
            raise AttributeError(f"{name} of a {type(self).__name__} follows from its tensors")
        else:
            super().__setattr__(name, value)

    def _keep(self, tensors, shapes, **follows):
        for name, t, shape in zip(self._TENSORS, tensors, shapes):
            if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous int32 tensor {shape}")
            if t.device != tensors[0].device:
                raise ValueError(f"the tensors are on {tensors[0].device} and {t.device}")
        d = tensors[0].device
        self.__dict__.update(zip(self._TENSORS, tensors))
        self.__dict__.update(follows, device=d, _index=d.index if d.type == "cuda" else -1,
                             _args=tuple(t.data_ptr() for t in tensors))


def _length(t, dims: int) -> tuple:
    if not isinstance(t, torch.Tensor) or t.dim() != dims:
        raise ValueError(f"a tensor of {dims} dimension{'s' if dims > 1 else ''} is needed")
    return tuple(t.shape)


class PagedTable(_Int32s):
    """The pages of a cache's sequences, all int32 on the GPU: the block table [B][table_len] (the tensor
    that the PagedCache has), the pages that each sequence holds [B], and the stack of free pages: free_pages
    [num_pages], of which the first free_count [1] are free, the last of them its top."""

    _TENSORS = ("block_table", "held", "free_pages", "free_count")
    _FOLLOWS = ("B", "page_tokens", "device", "_index", "_args", "_shape")

    def __init__(self, block_table, held, free_pages, free_count, page_tokens: int):
        self.__dict__["page_tokens"] = int(page_tokens)
        self._lay_out(block_table, held, free_pages, free_count)

    def _lay_out(self, *tensors):
        (B, table_len), (num_pages,) = _length(tensors[0], 2), _length(tensors[2], 1)
        self._keep(tensors, ((B, table_len), (B,), (num_pages,), (1,)), B=B,
                   _shape=Pages(num_pages, self.page_tokens, table_len))

    @classmethod
    def create(cls, num_pages: int, page_tokens: int, table_len: int, B: int, device="cuda") -> "PagedTable":
        """Every page free, no sequence holding any."""
        zeros = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=device)
        return cls(zeros(B, table_len), zeros(B), torch.arange(num_pages - 1, -1, -1, dtype=torch.int32, device=device),
                   zeros(1) + num_pages, page_tokens)


class PagedRows(_Int32s):
    """What step5_paged_plan writes of a step, all int32: of each row its sequence and position [N] (-1:
    padding), of each sequence its first row [B + 1], its tokens after the step, those granted, and the regions
    [region_begin, region_end) that the step completes [B]."""

    _TENSORS = ("row_seq", "row_pos", "row_start", "ends", "granted", "region_begin", "region_end")
    _FOLLOWS = ("B", "N", "device", "_index", "_args")

    def __init__(self, row_seq, row_pos, row_start, ends, granted, region_begin, region_end):
        self._lay_out(row_seq, row_pos, row_start, ends, granted, region_begin, region_end)

    def _lay_out(self, *tensors):
        (N,), (B,) = _length(tensors[0], 1), _length(tensors[3], 1)
        self._keep(tensors, ((N,), (N,), (B + 1,), (B,), (B,), (B,), (B,)), N=N, B=B)

    @classmethod
    def create(cls, B: int, N: int, device="cuda") -> "PagedRows":
        empty = lambda n: torch.empty(n, dtype=torch.int32, device=device)
        return cls(empty(N), empty(N), empty(B + 1), *(empty(B) for _ in range(4)))


def step5_paged_plan(table: PagedTable, rows: PagedRows, lengths, new_tokens, stream=None, geom=STEP5_GEOMETRY):
    """Plans a step of sequences that have ``lengths`` [B] tokens in the cache and get ``new_tokens`` [B] (int32):
    pages move between the table and its free ones, and ``rows`` is filled in (see the header).  lengths may be
    rows.ends, so that a captured step goes on from the one before."""
    dev = _current_device() if table._index >= 0 else torch.cuda.current_device()
    if table._index != dev or rows._index != dev:
        raise ValueError(f"the table is on {table.device}, the rows on {rows.device}, the current device is cuda:{dev}")
    B = table.B
    if rows.B != B:
        raise ValueError(f"the table has {B} sequences, the rows {rows.B}")
    if stream is not None:
        st = stream.cuda_stream
    else:
        st = _raw_stream(dev) if _raw_stream else torch.cuda.current_stream(dev).cuda_stream
    st = load().step5_paged_plan(Geometry.of(geom), table._shape, rows.N, B, _arg("lengths", lengths, torch.int32, (B,), dev),
                                 _arg("new_tokens", new_tokens, torch.int32, (B,), dev), *table._args, *rows._args, st)
    if st:
        raise Step5Error("step5_paged_plan", st)


def _check_indexers(g, t: dict, rows: dict):
    """That the indexer's tensors have the step's rows and sequences: the calls take these from different ones of them."""
    N, B, G, D = t["q"].shape[0], rows["sum_begin"].shape[0], g.num_kv_groups, g.idx_dim
    length = lambda name: t[name].shape[2] if isinstance(t[name], torch.Tensor) and t[name].dim() == 4 else -1
    t_cap, r_cap = length("idx_k"), length("summaries")
    bf16, i32 = torch.bfloat16, torch.int32
    for name, dtype, want in (("sum_begin", i32, (B,)), ("sum_end", i32, (B,)), ("idx_k", bf16, (B, G, t_cap, D)),
                              ("idx_z", bf16, (B, G, t_cap, D)), ("summaries", torch.uint8, (B, G, r_cap, D)),
                              ("idx_q", bf16, (N, g.idx_heads, D)), ("w", torch.float32, (N, g.idx_heads))):
        x = (rows if name in rows else t)[name]
        if not isinstance(x, torch.Tensor) or x.dtype != dtype or tuple(x.shape) != want:
            raise ValueError(f"{name} must be {dtype} {want}, of the step's {N} rows and {B} sequences")
    for name in ("cos", "sin"):
        x = t[name]
        if x is not None and (x.dtype != bf16 or x.dim() != 2 or x.shape[0] < t_cap or x.shape[1] != g.rope_dims // 2):
            raise ValueError(f"{name} of the indexer must be {bf16} {(t_cap, g.rope_dims // 2)}, or longer")


def decode_step_paged(geom, t: dict, cache: PagedCache, ws: Workspace, paged_ws: PagedWorkspace, k, v, sel_ids,
                      sel_count, q_rot, out, max_regions_per_seq, cos=None, sin=None, gate=None, stream=None,
                      plan=None):
    """One pass of the whole path over a paged cache, e4m3 or bf16: the rows' k and v appended (and
    t["q"] rotated into q_rot by cos/sin), then summarise, score + select over the indexer
    tensors of ``t`` as decode_step does, and attend over the picked regions of the cache.  With ``plan``,
    (table, rows, lengths, new_tokens) as step5_paged_plan takes them, the step is planned first, and its
    rows and regions take the place of t's row_seq, row_pos, sum_begin and sum_end; no page moves if the plan or a
    call behind it refuses an argument.  Rows that it pads have no picks, and their q_rot and out are left as they are."""
    rows = t
    if plan is not None:
        table, p = plan[:2]
        # (refused before any page moves)
        if p.N != t["q"].shape[0]:
            raise ValueError(f"the plan has {p.N} rows, q {t['q'].shape[0]}")
        if (cache.block_table is None or table._args[0] != cache.block_table.data_ptr() or table.B != cache.B
                or bytes(table._shape) != bytes(cache._shape)):
            raise ValueError("the plan's table must be the cache's, all its sequences")
        rows = {"row_seq": p.row_seq, "row_pos": p.row_pos, "sum_begin": p.region_begin, "sum_end": p.region_end}
    _check_indexers(Geometry.of(geom), t, rows)
    append, attend = (("step5_kv_append_e4m3", "step5_sparse_attn_e4m3") if cache.e4m3 else
                      ("step5_kv_append", "step5_sparse_attn_paged"))
    seq, pos = rows["row_seq"], rows["row_pos"]
    calls = (_append_call(append, cache.e4m3, geom, k, v, cache, seq, pos, cos, sin, t["q"], q_rot, stream),
             _summarize_call(geom, t["idx_k"], t["idx_z"], t["cos"], t["sin"], rows["sum_begin"], rows["sum_end"], t["summaries"],
                             None, max_regions_per_seq, stream),
             _score_call(geom, t["idx_q"], t["w"], seq, pos, t["cos"], t["sin"], t["summaries"], sel_ids, sel_count, ws.tensor,
                         t["idx_k"].shape[2], None, None, stream),
             _attend_call(attend, cache.e4m3, geom, q_rot, cache, seq, pos, out, paged_ws, gate, stream, sel_ids=sel_ids,
                          sel_count=sel_count))
    if plan is not None:  # (the other calls' checks first: 11 us of the host, once a step)
        prev = step5_set_check_only(1)
        try:
            for call in calls:
                _run(call)
        finally:
            step5_set_check_only(prev)
        step5_paged_plan(*plan, stream=stream, geom=geom)
    for call in calls:
        _run(call)
