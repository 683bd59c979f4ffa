"""Python face of the C ABI: the same entry points as include/dsa.h, taking torch tensors.

Argument marshalling only (pointers, sizes, strides, dtype codes, the current stream); outputs and
workspaces that the caller does not pass are allocated with torch on the inputs' device.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple, Optional, Tuple

import torch

from . import _native as N

__all__ = ["dsa_index_score", "dsa_topk", "dsa_topk_noalloc", "dsa_topk_pairs", "dsa_topk_merge",
           "dsa_sparse_attn_partial", "dsa_attn_combine", "dsa_sparse_attn", "DsaCall", "dsa_decode", "dsa_prefill",
           "dsa_workspace_size", "dsa_launch_count", "dsa_get_device_error", "ld_scores_for",
           "dsa_quantize_mxfp8", "dsa_quantize_fp8_rows", "dsa_quantize_fp8_tiles",
           "dsa_block_plan", "BlockPlan", "dsa_rope", "dsa_rope_append", "dsa_tree_attn"]


# The current stream's handle and the current device without building torch objects (a serving step makes
# several short calls, and the host's share of each is most of its time).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


# What a call allocates belongs to the stream that it runs on.  torch's allocator hands a freed block to later work of
# the stream that it was allocated on, without waiting for any other stream: scratch from the current stream's pool
# would be given away while the kernels on the caller's `stream` still use it, and an output's block may still be read
# by pending work of the current stream.

def _side(stream, device):
    """`stream`, where it is given and is not the device's current one; None otherwise."""
    return None if stream is None or stream.cuda_stream == _raw_stream(device.index) else stream


def _scratch(side, shape, dtype, device, zero=False):
    with contextlib.nullcontext() if side is None else torch.cuda.stream(side):
        return (torch.zeros if zero else torch.empty)(shape, dtype=dtype, device=device)


def _hand_back(t, device):
    """The caller's current stream reads `t` too: its block waits for that stream before it is used again."""
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _output(side, shape, dtype, device):
    return torch.empty(shape, dtype=dtype, device=device) if side is None else _hand_back(_scratch(side, shape, dtype, device), device)


def _zeros(stream, n, device):
    """A zero-filled workspace of n bytes: filled on the stream that the call runs on."""
    return _scratch(_side(stream, device), n, torch.uint8, device, zero=True)


class Owned:
    """Buffers that an object keeps for its calls (outputs, a workspace that was zero-filled), made on the current
    stream.  `follow` puts the first call on any other stream behind them, and holds their blocks back until that
    stream's work is done, should the object be dropped before it."""

    def __init__(self, *tensors):
        self._tensors = [t for t in tensors if t is not None]
        self._device = self._tensors[0].device
        current = torch.cuda.current_stream(self._device)
        self._known = {current.cuda_stream}
        self._captured = torch.cuda.is_current_stream_capturing()
        self._made = torch.cuda.Event()
        self._made.record(current)

    def follow(self, stream):
        if (_raw_stream(self._device.index) if stream is None else stream.cuda_stream) in self._known:
            return
        if stream is None:
            stream = torch.cuda.current_stream(self._device)
        with torch.cuda.stream(stream):
            capturing = torch.cuda.is_current_stream_capturing()
        if capturing or self._captured:
            return  # a graph cannot wait for what is outside of it: the capture's own forks and joins order it
        stream.wait_event(self._made)
        for t in self._tensors:
            t.record_stream(stream)
        self._known.add(stream.cuda_stream)


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _idx_dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return N.DSA_BF16
    if t.dtype == torch.uint8:
        return N.DSA_MXFP8_E4M3
    raise TypeError(f"indexer tensors must be bfloat16 or uint8 (E4M3 codes), got {t.dtype}")


def _kv_dtype(t: torch.Tensor, scale: Optional[torch.Tensor] = None) -> int:
    """bf16 rows; E4M3 rows with one scale per row (kv_scale without a last tile axis), or with
    one scale per 128-element tile (kv_scale [..., ceil(D_qk / 128)] beside the rows' axes)."""
    if t.dtype == torch.bfloat16:
        return N.DSA_BF16
    if t.dtype == torch.uint8:
        if scale is not None and scale.dim() == t.dim():
            return N.DSA_FP8_E4M3_T128
        return N.DSA_FP8_E4M3
    raise TypeError(f"kv must be bfloat16 or uint8 (E4M3 codes), got {t.dtype}")


def _seq_stride(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.stride(0) * t.element_size()


def ld_scores_for(L: int) -> int:
    return max(4, (L + 3) // 4 * 4)


def dsa_index_score(q_idx, w, k_idx, *, q_idx_sf=None, k_idx_sf=None, q_per_seq=1, q_pos0=-1,
                    n_valid=None, scores=None, stream=None) -> torch.Tensor:
    """Indexer scores [T, ld] fp32 (entries s >= n_t unspecified).  q_idx [T, H_idx, d],
    k_idx [n_seq, L, d] (rows packed), sf tensors for MXFP8."""
    T, H_idx, d = q_idx.shape
    L = k_idx.shape[1]
    if scores is None:
        scores = _output(_side(stream, q_idx.device), (T, ld_scores_for(L)), torch.float32, q_idx.device)
    st = N.lib.dsa_index_score(_p(q_idx), _p(q_idx_sf), _p(w), _p(k_idx), _p(k_idx_sf),
                               _seq_stride(k_idx), _seq_stride(k_idx_sf), T, q_per_seq, q_pos0,
                               _p(n_valid), L, H_idx, d, _idx_dtype(q_idx), _p(scores),
                               scores.stride(0), _stream(stream))
    N.check(st, "dsa_index_score")
    return scores


def dsa_topk(scores, K, *, L, q_per_seq=1, q_pos0=-1, n_valid=None, idx=None, ws=None, stream=None) -> torch.Tensor:
    """Top-K positions [T, K] int32 (ascending, -1 padded).  `ws`, if given, is a zero-filled
    uint8 tensor of at least dsa_topk_workspace_size bytes that later calls may reuse."""
    T = scores.shape[0]
    if idx is None:
        idx = _output(_side(stream, scores.device), (T, K), torch.int32, scores.device)
    ws_bytes = N.lib.dsa_topk_workspace_size(T, L, K)
    if ws is None:
        ws = _zeros(stream, max(ws_bytes, 16), scores.device) if ws_bytes else None
    else:
        ws_bytes = ws.numel()
    st = N.lib.dsa_topk(_p(scores), scores.stride(0), T, q_per_seq, q_pos0, _p(n_valid), L, K, _p(idx),
                        _p(ws), ws_bytes, _stream(stream))
    N.check(st, "dsa_topk")
    return idx


def dsa_topk_noalloc(scores, K, *, L, q_per_seq=1, q_pos0=-1, n_valid=None, idx=None, stream=None) -> torch.Tensor:
    """dsa_topk without a workspace: the library's own fixed scratch serves as the exchange area
    (at most 16 queries per call; calls that overlap on the GPU race, see dsa.h)."""
    T = scores.shape[0]
    if idx is None:
        idx = _output(_side(stream, scores.device), (T, K), torch.int32, scores.device)
    st = N.lib.dsa_topk_noalloc(_p(scores), scores.stride(0), T, q_per_seq, q_pos0, _p(n_valid), L, K,
                                _p(idx), _stream(stream))
    N.check(st, "dsa_topk_noalloc")
    return idx


def dsa_sparse_attn(q, kv, idx, *, sm_scale, kv_v=None, kv_scale=None, D_v=None, q_per_seq=1,
                    out=None, lse=None, ws=None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention over the rows named by idx.  q [T, H, D_qk] bf16; kv [n_seq, L, row] (bf16 or E4M3
    codes, row pitch from its stride); kv_v optional [n_seq, L, D_v] bf16; kv_scale [n_seq, L]."""
    T, H, D_qk = q.shape
    L = kv.shape[1]
    K = idx.shape[1]
    if D_v is None:
        D_v = kv_v.shape[-1] if kv_v is not None else (512 if D_qk == 576 else D_qk)
    if out is None:
        out = _output(_side(stream, q.device), (T, H, D_v), torch.bfloat16, q.device)
    if lse is None:
        lse = _output(_side(stream, q.device), (T, H), torch.float32, q.device)
    need = N.lib.dsa_sparse_attn_workspace_size(T, H, K, D_v)
    if ws is None and need:
        ws = _zeros(stream, need, q.device)
    st = N.lib.dsa_sparse_attn(_p(q), _p(kv), _p(kv_v), _p(kv_scale), kv.stride(1) * kv.element_size(),
                               _seq_stride(kv), 0 if kv_v is None else kv_v.stride(1) * 2, _seq_stride(kv_v),
                               _p(idx), T, q_per_seq, L, K, H, D_qk, D_v, float(sm_scale), _kv_dtype(kv, kv_scale),
                               _p(out), _p(lse), _p(ws), 0 if ws is None else ws.numel(), _stream(stream))
    N.check(st, "dsa_sparse_attn")
    return out, lse


def dsa_topk_pairs(scores, K, *, L, pos_offset, cand_pos, cand_scores, q_per_seq=1, q_pos0=-1, n_valid=None,
                   ws=None, stream=None):
    """One context slice's Top-K as (score, global position) pairs written into the [T, >= K]
    views cand_pos (int32) / cand_scores (fp32), which may be column slices of a wider buffer."""
    T = scores.shape[0]
    ws_bytes = N.lib.dsa_topk_workspace_size(T, L, K)
    if ws is None:
        ws = _zeros(stream, max(ws_bytes, 16), scores.device)
    st = N.lib.dsa_topk_pairs(_p(scores), scores.stride(0), T, q_per_seq, q_pos0, _p(n_valid), L, K,
                              int(pos_offset), _p(cand_pos), _p(cand_scores), cand_pos.stride(0), _p(ws),
                              ws.numel(), _stream(stream))
    N.check(st, "dsa_topk_pairs")
    return cand_pos, cand_scores


def dsa_topk_merge(cand_scores, cand_pos, K, *, idx=None, stream=None) -> torch.Tensor:
    """The K best (score, position) pairs of each query's candidates (-1 positions are empty), in
    candidate order, -1 padded.  Candidates as [T, n] (one part per query row) or as [G, T, n]
    (G parts, e.g. gathered from G devices), contiguous in the last axis."""
    if cand_pos.dim() == 2:
        T, n = cand_pos.shape
        parts, ld, pst = 1, cand_pos.stride(0), 0
    else:
        parts, T, n = cand_pos.shape
        ld, pst = cand_pos.stride(1), cand_pos.stride(0)
    if idx is None:
        idx = _output(_side(stream, cand_pos.device), (T, K), torch.int32, cand_pos.device)
    st = N.lib.dsa_topk_merge(_p(cand_scores), _p(cand_pos), T, parts, n, ld, pst, K, _p(idx), _stream(stream))
    N.check(st, "dsa_topk_merge")
    return idx


def dsa_sparse_attn_partial(q, kv, idx, *, sm_scale, pos_lo, kv_v=None, kv_scale=None, D_v=None, q_per_seq=1,
                            o_part=None, lse_part=None, ws=None, stream=None):
    """Attention of one context slice (cache rows = positions pos_lo .. pos_lo + L - 1) over the
    entries of idx it holds: fp32 normalised output [T, H, D_v] and its log-sum-exp [T, H]."""
    T, H, D_qk = q.shape
    L = kv.shape[1]
    K = idx.shape[1]
    if D_v is None:
        D_v = kv_v.shape[-1] if kv_v is not None else (512 if D_qk == 576 else D_qk)
    if o_part is None:
        o_part = _output(_side(stream, q.device), (T, H, D_v), torch.float32, q.device)
    if lse_part is None:
        lse_part = _output(_side(stream, q.device), (T, H), torch.float32, q.device)
    need = N.lib.dsa_sparse_attn_workspace_size(T, H, K, D_v)
    if ws is None and need:
        ws = _zeros(stream, need, q.device)
    st = N.lib.dsa_sparse_attn_partial(
        _p(q), _p(kv), _p(kv_v), _p(kv_scale), kv.stride(1) * kv.element_size(), _seq_stride(kv),
        0 if kv_v is None else kv_v.stride(1) * 2, _seq_stride(kv_v), _p(idx), T, q_per_seq, L, K, H, D_qk, D_v,
        float(sm_scale), _kv_dtype(kv, kv_scale), int(pos_lo), _p(o_part), _p(lse_part), _p(ws),
        0 if ws is None else ws.numel(), _stream(stream))
    N.check(st, "dsa_sparse_attn_partial")
    return o_part, lse_part


def dsa_attn_combine(o_parts, lse_parts, *, out=None, lse=None, stream=None):
    """Merge of G partial outputs o_parts [G, T, H, D_v] fp32 / lse_parts [G, T, H] into the bf16
    output [T, H, D_v] and its log-sum-exp [T, H]."""
    G, T, H, D_v = o_parts.shape
    if out is None:
        out = _output(_side(stream, o_parts.device), (T, H, D_v), torch.bfloat16, o_parts.device)
    if lse is None:
        lse = _output(_side(stream, o_parts.device), (T, H), torch.float32, o_parts.device)
    st = N.lib.dsa_attn_combine(_p(o_parts), _p(lse_parts), G, o_parts.stride(0), lse_parts.stride(0), T, H, D_v,
                                _p(out), _p(lse), _stream(stream))
    N.check(st, "dsa_attn_combine")
    return out, lse


class DsaCall:
    """One configured fused call (dsa_decode or dsa_prefill) with its outputs and workspace
    allocated once; calling it enqueues the chain on the current (or given) stream."""

    def __init__(self, *, q_idx, w, k_idx, q, kv, K, sm_scale, q_idx_sf=None, k_idx_sf=None,
                 kv_scale=None, kv_v=None, D_v=None, q_per_seq=1, q_pos0=-1, n_valid=None,
                 out=None, lse=None, idx_out=None, keep_idx=True, ws=None,
                 block_table=None, block_size=0, L=None):
        """Caches are [n_seq, L, ...] per sequence, or, with `block_table` (int32 [n_seq,
        max_blocks]) and `block_size`, pools of rows ([rows, ...]; kv_scale [rows]) shared by all
        sequences, with the positions per sequence `L` given explicitly."""
        T, H_idx, d_idx = q_idx.shape
        _, H, D_qk = q.shape
        paged = block_table is not None
        if paged:
            if L is None or block_size <= 0:
                raise ValueError("paged caches need L and block_size")
        else:
            L = k_idx.shape[1]
        if D_v is None:
            D_v = kv_v.shape[-1] if kv_v is not None else (512 if D_qk == 576 else D_qk)
        dev = q.device
        self.prefill = q_pos0 >= 0
        self.out = out if out is not None else torch.empty(T, H, D_v, dtype=torch.bfloat16, device=dev)
        self.lse = lse if lse is not None else torch.empty(T, H, dtype=torch.float32, device=dev)
        if idx_out is None and keep_idx:
            idx_out = torch.empty(T, K, dtype=torch.int32, device=dev)
        self.idx = idx_out
        a = N.DsaArgs()
        a.T, a.q_per_seq, a.q_pos0, a.L, a.K = T, q_per_seq, q_pos0, L, K
        a.H_idx, a.d_idx, a.H, a.D_qk, a.D_v = H_idx, d_idx, H, D_qk, D_v
        a.sm_scale = float(sm_scale)
        a.idx_dtype, a.kv_dtype = _idx_dtype(q_idx), _kv_dtype(kv, kv_scale)
        ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        a.n_valid = ptr(n_valid)
        a.q_idx, a.q_idx_sf, a.w = ptr(q_idx), ptr(q_idx_sf), ptr(w)
        a.k_idx, a.k_idx_sf = ptr(k_idx), ptr(k_idx_sf)
        a.q, a.kv, a.kv_v, a.kv_scale = ptr(q), ptr(kv), ptr(kv_v), ptr(kv_scale)
        if paged:
            a.k_seq_stride = a.k_sf_seq_stride = a.kv_seq_stride = a.v_seq_stride = 0
            a.kv_row_stride = kv.stride(0) * kv.element_size()
            a.v_row_stride = 0 if kv_v is None else kv_v.stride(0) * kv_v.element_size()
            a.block_table = ptr(block_table)
            a.block_size = int(block_size)
            a.max_blocks = block_table.shape[1]
            a.num_blocks = k_idx.shape[0] // int(block_size)
        else:
            a.k_seq_stride, a.k_sf_seq_stride = _seq_stride(k_idx), _seq_stride(k_idx_sf)
            a.kv_row_stride = kv.stride(1) * kv.element_size()
            a.kv_seq_stride = _seq_stride(kv)
            a.v_row_stride = 0 if kv_v is None else kv_v.stride(1) * kv_v.element_size()
            a.v_seq_stride = _seq_stride(kv_v)
            a.block_table = None
        a.out, a.lse, a.idx_out = ptr(self.out), ptr(self.lse), ptr(self.idx)
        self.args = a
        # keep every tensor the struct points at alive as long as the call object
        self._keep = (q_idx, w, k_idx, q, kv, q_idx_sf, k_idx_sf, kv_scale, kv_v, n_valid, block_table)
        need = dsa_workspace_size(a, self.prefill)
        if ws is None:
            ws = torch.zeros(max(need, 16), dtype=torch.uint8, device=dev)
        elif ws.numel() < need:
            raise ValueError(f"workspace has {ws.numel()} bytes, needs {need}")
        self.ws = ws
        self._fn = N.lib.dsa_prefill if self.prefill else N.lib.dsa_decode
        self.launches = dsa_launch_count(a, self.prefill)  # kernels per call
        self._owned = Owned(self.out, self.lse, self.idx, self.ws)

    def __call__(self, stream=None):
        self._owned.follow(stream)
        st = self._fn(ctypes.byref(self.args), _p(self.ws), self.ws.numel(), _stream(stream))
        N.check(st, "dsa_prefill" if self.prefill else "dsa_decode")
        return self.out, self.lse, self.idx


def dsa_workspace_size(args: N.DsaArgs, prefill: bool) -> int:
    n = ctypes.c_size_t(0)
    N.check(N.lib.dsa_workspace_size(ctypes.byref(args), int(bool(prefill)), ctypes.byref(n)),
            "dsa_workspace_size")
    return n.value


def dsa_quantize_mxfp8(x, *, codes=None, sf=None, dst_rows=None, stream=None):
    """bf16 rows x [rows, d] -> (E4M3 codes, E8M0 exponents per 32).  With `dst_rows` (int64
    [rows]) input row r is written to row dst_rows[r] of the given `codes` [*, d] / `sf`
    [*, d/32] (a cache append); without it new [rows, d] / [rows, d/32] tensors are returned."""
    rows, d = x.shape
    if codes is None:
        codes = _output(_side(stream, x.device), (rows, d), torch.uint8, x.device)
    if sf is None:
        sf = _output(_side(stream, x.device), (rows, d // 32), torch.uint8, x.device)
    N.check(N.lib.dsa_quantize_mxfp8(_p(x), x.stride(0), rows, d, _p(codes), _p(sf), _p(dst_rows),
                                     _stream(stream)), "dsa_quantize_mxfp8")
    return codes, sf


def dsa_quantize_fp8_rows(x, *, codes=None, scales=None, dst_rows=None, stream=None):
    """bf16 rows x [rows, width] -> (E4M3 codes, one fp32 scale per row); `dst_rows` as in
    dsa_quantize_mxfp8 (codes [*, >= width] with any row pitch, scales [*])."""
    rows, width = x.shape
    if codes is None:
        codes = _output(_side(stream, x.device), (rows, width), torch.uint8, x.device)
    if scales is None:
        scales = _output(_side(stream, x.device), rows, torch.float32, x.device)
    N.check(N.lib.dsa_quantize_fp8_rows(_p(x), x.stride(0), rows, width, _p(codes), codes.stride(0),
                                        _p(scales), _p(dst_rows), _stream(stream)),
            "dsa_quantize_fp8_rows")
    return codes, scales


def dsa_quantize_fp8_tiles(x, *, tile=128, codes=None, scales=None, dst_rows=None, stream=None):
    """bf16 rows x [rows, width] -> (E4M3 codes, fp32 scales [rows, ceil(width / tile)]): one
    scale per `tile` consecutive elements of a row; `dst_rows` as in dsa_quantize_mxfp8."""
    rows, width = x.shape
    nt = -(-width // tile)
    if codes is None:
        codes = _output(_side(stream, x.device), (rows, width), torch.uint8, x.device)
    if scales is None:
        scales = _output(_side(stream, x.device), (rows, nt), torch.float32, x.device)
    N.check(N.lib.dsa_quantize_fp8_tiles(_p(x), x.stride(0), rows, width, tile, _p(codes), codes.stride(0),
                                         _p(scales), _p(dst_rows), _stream(stream)), "dsa_quantize_fp8_tiles")
    return codes, scales


# The serving-step operators below check their tensors (device, dtype, layout) and run on the
# tensors' own device and its current stream, whichever device is current, or on the `stream` given: then
# the inputs have to be ready on that stream and to live until its work is done, and the outputs are ready
# when it is.

def _check(what, device, name, t, dtype, dims=None, dense=True):
    if t is None:
        return
    if t.device != device:
        raise ValueError(f"{what}: {name} is on {t.device}, the call on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{what}: {name} must be {dtype}, got {t.dtype}")
    if dims is not None and t.dim() != dims:
        raise ValueError(f"{what}: {name} must have {dims} axes, got shape {tuple(t.shape)}")
    if dense and not t.is_contiguous():
        raise ValueError(f"{what}: {name} must be contiguous")


def _cuda_device(what, t) -> torch.device:
    if not t.is_cuda:
        raise ValueError(f"{what}: tensors must be on a CUDA device, got {t.device}")
    return t.device


def _run(what, fn, device, stream, *args):
    i = device.index
    if stream is None:
        handle = _raw_stream(i)
    elif stream.device != device:
        raise ValueError(f"{what}: the stream is on {stream.device}, the tensors on {device}")
    else:
        handle = stream.cuda_stream
    if _current_device() == i:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            st = fn(*args, handle)
    if st != N.DSA_OK:
        N.check(st, what)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


class BlockPlan(NamedTuple):
    """What dsa_block_plan gives (see dsa.h): per row `dst_rows` int64, `pos` and `seq` int32 (-1: no
    token); `row_start` int32 [n_seq + 1]; `n_placed` int32 [n_seq]; `taken` int32 [1]."""
    dst_rows: torch.Tensor
    pos: torch.Tensor
    seq: torch.Tensor
    row_start: torch.Tensor
    n_placed: torch.Tensor
    taken: torch.Tensor


def dsa_block_plan(n_ctx, n_new, free_blocks, block_table, *, block_size, num_blocks, rows=None, q_per_seq=0,
                   n_free=None, out: Optional[BlockPlan] = None, stream=None) -> BlockPlan:
    """Blocks, block-table entries and destination rows of a step that appends n_new[s] tokens to
    sequences of n_ctx[s] (int32 [n_seq]).  New blocks come from the front of `free_blocks` (int32; the
    first n_free[0] of them when given); `block_table` int32 [n_seq, max_blocks] is updated in place.
    Rows are packed (`rows` given, at least the tokens of the step), or padded to q_per_seq per
    sequence (`rows` defaults to n_seq * q_per_seq)."""
    what = "dsa_block_plan"
    dev = _cuda_device(what, n_ctx)
    i32 = torch.int32
    _check(what, dev, "n_ctx", n_ctx, i32, 1)
    _check(what, dev, "n_new", n_new, i32, 1)
    _check(what, dev, "free_blocks", free_blocks, i32, 1)
    _check(what, dev, "n_free", n_free, i32)
    _check(what, dev, "block_table", block_table, i32, 2)
    n_seq = n_ctx.shape[0]
    if n_new.shape[0] != n_seq or block_table.shape[0] != n_seq or (n_free is not None and n_free.numel() < 1):
        raise ValueError(f"{what}: n_ctx, n_new and block_table must agree on the number of sequences")
    if rows is None:
        if q_per_seq <= 0:
            raise ValueError(f"{what}: packed rows need their number (rows)")
        rows = n_seq * q_per_seq
    if out is None:
        # (six allocations take 9 us of the host, six views of one 12.5: most of it when they are freed)
        side = _side(stream, dev)
        out = BlockPlan(_output(side, rows, torch.int64, dev), _output(side, rows, i32, dev), _output(side, rows, i32, dev),
                        _output(side, n_seq + 1, i32, dev), _output(side, n_seq, i32, dev), _output(side, 1, i32, dev))
    else:
        for name, t, n, kind in (("dst_rows", out.dst_rows, rows, torch.int64), ("pos", out.pos, rows, i32),
                                 ("seq", out.seq, rows, i32), ("row_start", out.row_start, n_seq + 1, i32),
                                 ("n_placed", out.n_placed, n_seq, i32), ("taken", out.taken, 1, i32)):
            _check(what, dev, name, t, kind, 1)
            if t.shape[0] < n:
                raise ValueError(f"{what}: {name} has {t.shape[0]} entries, needs {n}")
    _run(what, N.lib.dsa_block_plan, dev, stream, n_ctx.data_ptr(), n_new.data_ptr(), n_seq, int(q_per_seq),
         int(block_size), free_blocks.data_ptr(), _ptr(n_free), free_blocks.shape[0], int(num_blocks),
         block_table.data_ptr(), block_table.shape[1], int(rows), out.dst_rows.data_ptr(), out.pos.data_ptr(),
         out.seq.data_ptr(), out.row_start.data_ptr(), out.n_placed.data_ptr(), out.taken.data_ptr())
    return out


_ROPE_STYLE = {"half": N.DSA_ROPE_HALF, "pairs": N.DSA_ROPE_PAIRS}


def _rope_args(what, dev, x, pos, inv_freq, rot_off, rot_dim, sections, pair_axis, style):
    shape = x.shape
    one = pos.dim() == 1
    _check(what, dev, "pos", pos, torch.int32, 1 if one else 2)
    _check(what, dev, "inv_freq", inv_freq, torch.float32, 1)
    if rot_dim is None:
        rot_dim = shape[-1] - rot_off
    n_axes = 1 if one else pos.shape[1]
    if pos.shape[0] != shape[0] or 2 * inv_freq.shape[0] != rot_dim:
        raise ValueError(f"{what}: pos must have one row per row of x, inv_freq rot_dim / 2 entries")
    if pair_axis is None and sections is not None:
        if len(sections) != n_axes:
            raise ValueError(f"{what}: {len(sections)} sections for {n_axes} axes")
        if min(sections) < 0:
            raise ValueError(f"{what}: sections are numbers of pairs, got {tuple(sections)}")
        pair_axis = b"".join(bytes([a]) * int(n) for a, n in enumerate(sections))
    elif pair_axis is not None:
        pair_axis = bytes(pair_axis)
    if pair_axis is not None and 2 * len(pair_axis) != rot_dim:
        raise ValueError(f"{what}: {len(pair_axis)} pairs have an axis, rot_dim / 2 = {rot_dim // 2} need one")
    if style not in _ROPE_STYLE:
        raise ValueError(f"{what}: style must be one of {tuple(_ROPE_STYLE)}, got {style!r}")
    return rot_dim, n_axes, pair_axis, _ROPE_STYLE[style]


def dsa_rope(x, pos, inv_freq, *, rot_off=0, rot_dim=None, sections=None, pair_axis=None, style="half",
             inverse=False, out=None, stream=None) -> torch.Tensor:
    """Rotary positions on columns [rot_off, rot_off + rot_dim) (default: to the last one) of bf16 x
    [rows, heads, width] or [rows, width].  pos int32 [rows] or [rows, n_axes]; inv_freq fp32
    [rot_dim / 2]; with several axes `sections` (pairs per axis, in order) or `pair_axis` (the axis
    of each pair) says which axis turns a pair.  `out` may be x itself (in place) or any strided
    tensor of x's shape that does not overlap it; `inverse` turns back (the gradient)."""
    what = "dsa_rope"
    dev = _cuda_device(what, x)
    _check(what, dev, "x", x, torch.bfloat16, None, dense=False)
    shape, xs = x.shape, x.stride()
    if len(shape) not in (2, 3) or (shape[-1] > 1 and xs[-1] != 1):
        raise ValueError(f"{what}: x must be [rows, heads, width] or [rows, width] with dense columns")
    rot_dim, n_axes, pair_axis, code = _rope_args(what, dev, x, pos, inv_freq, rot_off, rot_dim, sections, pair_axis, style)
    if out is None:
        out = _output(_side(stream, dev), shape, torch.bfloat16, dev)
        os = out.stride()
    else:
        _check(what, dev, "out", out, torch.bfloat16, len(shape), dense=False)
        os = out.stride()
        if out.shape != shape or (shape[-1] > 1 and os[-1] != 1):
            raise ValueError(f"{what}: out must have x's shape and dense columns")
    rows, width = shape[0], shape[-1]
    heads = shape[1] if len(shape) == 3 else 1
    if rows == 0 or heads == 0:
        return out
    xh, oh = (xs[1], os[1]) if heads > 1 else (width, width)
    _run(what, N.lib.dsa_rope, dev, stream, x.data_ptr(), xs[0], xh, rows, heads, width, int(rot_off), int(rot_dim),
         pos.data_ptr(), n_axes, pair_axis, inv_freq.data_ptr(), code, int(bool(inverse)), out.data_ptr(), os[0], oh)
    return out


def dsa_rope_append(x, pos, inv_freq, dst, *, scale=None, dst_rows=None, rot_off, rot_dim=None, sections=None,
                    pair_axis=None, style="half", stream=None) -> None:
    """bf16 rows x [rows, width], turned as in dsa_rope, encoded and written to rows dst_rows (int64
    [rows]; negative: dropped; None: row r) of the cache rows dst [*, >= width]: bf16, or uint8 E4M3
    codes with `scale` fp32 [*] (per row), fp32 [*, ceil(width / 128)] (per 128 columns) or uint8
    [*, width / 32] (MXFP8 exponents)."""
    what = "dsa_rope_append"
    dev = _cuda_device(what, x)
    _check(what, dev, "x", x, torch.bfloat16, 2, dense=False)
    (rows, width), (x_row, x_col) = x.shape, x.stride()
    if width > 1 and x_col != 1:
        raise ValueError(f"{what}: x must have dense columns")
    rot_dim, n_axes, pair_axis, code = _rope_args(what, dev, x, pos, inv_freq, rot_off, rot_dim, sections, pair_axis, style)
    if dst.dtype == torch.bfloat16:
        kind, want = N.DSA_BF16, None
    elif scale is None:
        raise ValueError(f"{what}: E4M3 rows need their scales")
    elif scale.dtype == torch.uint8:
        kind, want = N.DSA_MXFP8_E4M3, (width // 32,)
    elif scale.dim() == 1:
        kind, want = N.DSA_FP8_E4M3, ()
    else:
        kind, want = N.DSA_FP8_E4M3_T128, (-(-width // 128),)
    _check(what, dev, "dst", dst, torch.bfloat16 if kind == N.DSA_BF16 else torch.uint8, 2, dense=False)
    (n_dst, dst_width), (dst_row, dst_col) = dst.shape, dst.stride()
    if dst_width < width or dst_col != 1 or (n_dst > 1 and dst_row < width):
        raise ValueError(f"{what}: dst rows must hold {width} dense columns")
    if want is not None:
        _check(what, dev, "scale", scale, torch.uint8 if kind == N.DSA_MXFP8_E4M3 else torch.float32)
        if scale.shape[1:] != want or scale.shape[0] < n_dst:
            raise ValueError(f"{what}: scale must be [{n_dst}{''.join(f', {n}' for n in want)}], got {tuple(scale.shape)}")
    _check(what, dev, "dst_rows", dst_rows, torch.int64, 1)
    if dst_rows is not None and dst_rows.shape[0] != rows:
        raise ValueError(f"{what}: dst_rows must have one entry per row of x")
    if rows == 0:
        return
    _run(what, N.lib.dsa_rope_append, dev, stream, x.data_ptr(), x_row, rows, width, int(rot_off), int(rot_dim),
         pos.data_ptr(), n_axes, pair_axis, inv_freq.data_ptr(), code, kind, dst.data_ptr(),
         (dst_row if n_dst > 1 else width) * (2 if kind == N.DSA_BF16 else 1), n_dst,
         None if kind == N.DSA_BF16 else scale.data_ptr(), _ptr(dst_rows))


def dsa_tree_attn(q, kv, n_ctx, *, sm_scale, q_per_seq, n_new=None, tree_mask=None, kv_scale=None, block_table=None,
                  block_size=0, L=None, out=None, lse=None, ws=None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of drafted tokens over the visible latent cache (see dsa.h): (out [T, H, 512] bf16,
    lse [T, H] fp32).  q bf16 [n_seq * q_per_seq, H, 576]; kv [n_seq, L, 576] bf16 or uint8 E4M3
    codes (kv_scale [n_seq, L] or [n_seq, L, 5]), or with `block_table` (int32 [n_seq, max_blocks]) and
    `block_size` a pool [rows, 576] (kv_scale [rows] or [rows, 5]) with `L` positions per sequence at
    most.  n_ctx, n_new int32 [n_seq]; tree_mask int32 or uint32 [T, ceil(q_per_seq / 32)] bits, None
    for a chain.  `ws` (uint8) is scratch that later calls on the same stream may reuse."""
    what = "dsa_tree_attn"
    dev = _cuda_device(what, q)
    _check(what, dev, "q", q, torch.bfloat16, 3)
    _check(what, dev, "n_ctx", n_ctx, torch.int32, 1)
    _check(what, dev, "n_new", n_new, torch.int32, 1)
    T, H, D = q.shape
    n_seq = n_ctx.shape[0]
    if q_per_seq < 1 or T != n_seq * q_per_seq or (n_new is not None and n_new.shape[0] != n_seq):
        raise ValueError(f"{what}: {T} queries are not q_per_seq = {q_per_seq} nodes of {n_seq} sequences")
    if tree_mask is not None:
        _check(what, dev, "tree_mask", tree_mask, torch.uint32 if tree_mask.dtype == torch.uint32 else torch.int32, 2)
        if tree_mask.shape[0] != T or tree_mask.shape[1] != (q_per_seq + 31) // 32:
            raise ValueError(f"{what}: tree_mask must be [{T}, {(q_per_seq + 31) // 32}], got {tuple(tree_mask.shape)}")
    paged = block_table is not None
    axes = 2 if paged else 3
    bf16 = kv.dtype == torch.bfloat16
    _check(what, dev, "kv", kv, torch.bfloat16 if bf16 else torch.uint8, axes, dense=False)
    shape, strides = kv.shape, kv.stride()
    if shape[-1] < D or strides[-1] != 1:
        raise ValueError(f"{what}: kv rows must hold {D} dense columns")
    a = N.DsaTreeArgs()
    a.kv_dtype = N.DSA_BF16
    if not bf16:
        if kv_scale is None:
            raise ValueError(f"{what}: E4M3 rows need their scales")
        a.kv_dtype = N.DSA_FP8_E4M3_T128 if kv_scale.dim() == axes else N.DSA_FP8_E4M3
        _check(what, dev, "kv_scale", kv_scale, torch.float32)
        want = tuple(shape[:-1]) + ((-(-D // 128),) if kv_scale.dim() == axes else ())
        if tuple(kv_scale.shape) != want:
            raise ValueError(f"{what}: kv_scale must be {list(want)}, got {tuple(kv_scale.shape)}")
        a.kv_scale = kv_scale.data_ptr()
    elem = 2 if bf16 else 1
    if paged:
        _check(what, dev, "block_table", block_table, torch.int32, 2)
        if L is None or block_size <= 0 or block_table.shape[0] != n_seq:
            raise ValueError(f"{what}: paged caches need L, block_size and one row of block_table per sequence")
        a.block_table, a.block_size, a.max_blocks = block_table.data_ptr(), int(block_size), block_table.shape[1]
        a.num_blocks = shape[0] // int(block_size)
        a.kv_row_stride = strides[0] * elem
    else:
        if shape[0] != n_seq or (L is not None and L != shape[1]):
            raise ValueError(f"{what}: kv must be [{n_seq}, L, {D}], got {tuple(shape)}")
        L = shape[1]
        a.kv_row_stride, a.kv_seq_stride = strides[1] * elem, strides[0] * elem
    side = _side(stream, dev)
    if out is None:
        out = _output(side, (T, H, 512), torch.bfloat16, dev)
    else:
        _check(what, dev, "out", out, torch.bfloat16, 3)
        if tuple(out.shape) != (T, H, 512):
            raise ValueError(f"{what}: out must be [{T}, {H}, 512]")
    if lse is None:
        lse = _output(side, (T, H), torch.float32, dev)
    else:
        _check(what, dev, "lse", lse, torch.float32, 2)
        if tuple(lse.shape) != (T, H):
            raise ValueError(f"{what}: lse must be [{T}, {H}]")
    a.n_seq, a.q_per_seq, a.L, a.H, a.D_qk, a.D_v, a.sm_scale = n_seq, int(q_per_seq), int(L), H, D, 512, float(sm_scale)
    a.n_ctx, a.n_new, a.tree_mask = n_ctx.data_ptr(), _ptr(n_new), _ptr(tree_mask)
    a.q, a.kv, a.out, a.lse = q.data_ptr(), kv.data_ptr(), out.data_ptr(), lse.data_ptr()
    need = ctypes.c_size_t(0)
    N.check(N.lib.dsa_tree_attn_workspace_size(ctypes.byref(a), ctypes.byref(need)), what)
    if ws is None:
        ws = _scratch(side, need.value, torch.uint8, dev) if need.value else None
    else:
        _check(what, dev, "ws", ws, torch.uint8, 1)
    _run(what, N.lib.dsa_tree_attn, dev, stream, ctypes.byref(a), _ptr(ws), 0 if ws is None else ws.numel())
    return out, lse


def dsa_launch_count(args: N.DsaArgs, prefill: bool) -> int:
    """Kernels one dsa_decode / dsa_prefill call with `args` launches."""
    n = ctypes.c_int(0)
    N.check(N.lib.dsa_launch_count(ctypes.byref(args), int(bool(prefill)), ctypes.byref(n)),
            "dsa_launch_count")
    return n.value


def dsa_decode(**kw):
    """Fused indexer -> Top-K -> sparse attention for a decode batch; returns (out, lse, idx)."""
    return DsaCall(**kw)()


def dsa_prefill(**kw):
    """Fused chain for a causal chunk (q_pos0 >= 0); returns (out, lse, idx)."""
    if kw.get("q_pos0", -1) < 0:
        raise ValueError("dsa_prefill needs q_pos0 >= 0")
    return DsaCall(**kw)()


def dsa_set_attn_kernel(kernel: int) -> None:
    """Select the attention kernel for the 576/512 latent row (N.DSA_ATTN_AUTO or
    N.DSA_ATTN_TCGEN05; process-wide, for calls made afterwards)."""
    N.check(N.lib.dsa_set_attn_kernel(int(kernel)), "dsa_set_attn_kernel")


def dsa_get_device_error(stream=None) -> int:
    code = ctypes.c_int(0)
    N.check(N.lib.dsa_get_device_error(ctypes.byref(code), _stream(stream)), "dsa_get_device_error")
    return code.value


def dsa_selftest_wait_timeout(stream=None) -> None:
    """Enqueue the failure-path self-test: a kernel whose bounded wait runs out (about one second)
    and records the wait-timeout device error code; read it with dsa_get_device_error."""
    N.check(N.lib.dsa_selftest_wait_timeout(_stream(stream)), "dsa_selftest_wait_timeout")
