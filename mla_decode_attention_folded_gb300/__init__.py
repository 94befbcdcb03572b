"""Folded, KV-balanced FP8 MLA decode for GB300 (sm_103a).

A thin Python binding over the C ABI of ``include/mlafold.h``: it marshals
PyTorch device tensors into pointers and calls the library; every step of the
decode runs in the library's CUDA kernels. PyTorch only owns the memory and
the stream.

The API follows the pages (drafter-attention page, ``folded_decode``;
balanced-MLA page, ``BalancedMla.require`` / ``plan`` / ``decode``):

* ``FoldedMla(R, k, H, max_pages, num_pages, device)`` allocates the plan
  buffers (``counts`` zeros, ``work`` -1) and the split-KV workspace up front,
  so nothing is allocated later (and a CUDA graph can capture the calls);
* ``.plan(seq_lens)`` plans the step's splits on the device, once per step;
* ``.decode(q, kv, block_table, seq_lens, bmm1_scale, bmm2_scale)`` runs the
  split-KV decode and the LSE reduction: BF16 ``out [R, k*H, 512]`` and the
  base-2 ``lse [R, k*H]``, in the stock token-major-then-head order.

Around the decode (additions of this library): ``kv_append(...)`` writes new
tokens into the paged cache (RMS norm, rotation, E4M3), ``query_absorb(...)``
makes the decode's queries (W_UK, rotation, E4M3), ``rope_table(rows)`` makes the
table of angles both read; ``PrefixMla(...)`` decodes a batch whose requests
share a prefix, reading the prefix's keys once for all of them.

Before the cache: ``prompt_attention(...)`` over whole packed prompts, or chunks of
them, in the expanded form. To bound the cache: ``kv_weigh(...)`` adds up the attention
weight of every cached key after a decode, ``kv_evict(...)`` keeps the keys of most
weight.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib
from ._lib import (AppendShape, CacheShape, FAULT_PAGE_RANGE, FAULT_ROPE_RANGE, FAULT_WAIT_TIMEOUT,
                   FAULT_WORK_ITEM, MlaError, MlaShape, POLICY_BALANCED, POLICY_UNIFORM,
                   PromptShape, QueryShape)

__all__ = ["MlaShape", "MlaError", "POLICY_BALANCED", "POLICY_UNIFORM", "make_shape",
           "plan_list_len", "workspace_bytes", "plan_splits", "folded_decode",
           "split_combine", "uv_combine", "lse_merge", "folded_decode_noalloc",
           "folded_decode_wait_test", "tier_plan", "row_copy", "balanced_tiers", "TIERS", "MOVE",
           "FoldedMla", "TieredMla", "fold_factor", "FAULT_WAIT_TIMEOUT", "FAULT_PAGE_RANGE",
           "FAULT_WORK_ITEM", "FAULT_ROPE_RANGE", "library_path", "rope_table", "kv_append",
           "query_absorb", "query_absorb_wait_test", "prefix_workspace_bytes", "prefix_plan",
           "prefix_decode", "prefix_decode_wait_test", "PrefixMla", "kv_weigh", "kv_weigh_wait_test",
           "kv_evict", "kv_evict_workspace_bytes", "prompt_attention", "prompt_attention_wait_test",
           "prompt_workspace_bytes"]

PAGE = 64


def library_path() -> str:
    return _lib.LIB_PATH


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:      # the current stream's handle, without a Stream object around it
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def make_shape(R: int, k: int, H: int, max_pages: int, num_pages: int, num_ctas: int,
               min_split_tokens: int = 256, max_splits: int = 64,
               policy: int = POLICY_BALANCED, groups: int = 1) -> MlaShape:
    return MlaShape(R, k, H, PAGE, max_pages, num_pages, num_ctas, min_split_tokens,
                    max_splits, policy, groups)


def fold_factor(k: int, H: int, max_heads: int = 128) -> int:
    """Tokens folded into one decode row when a row may hold at most
    `max_heads` heads: the largest divisor f of k with f * H <= max_heads
    (1 when even one token's heads exceed it). The drafter-attention page's
    `fold_plan` rule for the LSE-returning kernel (its example: k = 4 at 64
    heads folds pairs). Use groups = k // f row groups per request."""
    best = 1
    for f in range(1, k + 1):
        if k % f == 0 and f * H <= max_heads:
            best = f
    return best


def plan_list_len(shape: MlaShape) -> int:
    return _lib.check("mla_plan_list_len", _lib.load().mla_plan_list_len(ctypes.byref(shape)))


def workspace_bytes(shape: MlaShape) -> int:
    out = ctypes.c_size_t(0)
    _lib.check("mla_workspace_bytes", _lib.load().mla_workspace_bytes(ctypes.byref(shape),
                                                                      ctypes.byref(out)))
    return out.value


def plan_splits(shape: MlaShape, seq_lens, counts, work, stream=None) -> None:
    _lib.check("mla_plan_splits", _lib.load().mla_plan_splits(
        ctypes.byref(shape), _ptr(seq_lens), _ptr(counts), _ptr(work), work.numel(),
        _stream(stream)))


def folded_decode(shape: MlaShape, q, kv, block_table, seq_lens, bmm1_scale: float,
                  bmm2_scale: float, counts, work, workspace, out, lse, status=None,
                  stream=None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _lib.check("mla_folded_decode", _lib.load().mla_folded_decode(
        ctypes.byref(shape), _ptr(q), _ptr(kv), _ptr(block_table), _ptr(seq_lens),
        float(bmm1_scale), float(bmm2_scale), _ptr(counts), _ptr(work), work.numel(),
        _ptr(workspace), ws_bytes, _ptr(out), _ptr(lse), _ptr(status), _stream(stream)))


def folded_decode_wait_test(shape: MlaShape, q, kv, block_table, seq_lens, bmm1_scale: float,
                            bmm2_scale: float, counts, work, workspace, out, lse, status,
                            wait_limit_ns: int, stream=None) -> None:
    """Failure-detection test hook: the decode with every pipeline wait bounded
    by wait_limit_ns and CTA 0's first KV copy withheld, so that a wait runs
    out and MLA_FAULT_WAIT_TIMEOUT is set in `status` (see include/mlafold.h)."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _lib.check("mla_folded_decode_wait_test", _lib.load().mla_folded_decode_wait_test(
        ctypes.byref(shape), _ptr(q), _ptr(kv), _ptr(block_table), _ptr(seq_lens),
        float(bmm1_scale), float(bmm2_scale), _ptr(counts), _ptr(work), work.numel(),
        _ptr(workspace), ws_bytes, _ptr(out), _ptr(lse), _ptr(status), int(wait_limit_ns),
        _stream(stream)))


def split_combine(shape: MlaShape, counts, work, workspace, bmm2_scale: float, out, lse,
                  stream=None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _lib.check("mla_split_combine", _lib.load().mla_split_combine(
        ctypes.byref(shape), _ptr(counts), _ptr(work), work.numel(), _ptr(workspace), ws_bytes,
        float(bmm2_scale), _ptr(out), _ptr(lse), _stream(stream)))


def uv_combine(shape: MlaShape, counts, work, workspace, bmm2_scale: float, out, w_uv, y,
               status=None, stream=None) -> None:
    """The split reduction fused with the W_UV up-projection: y [R*k, H, 128]
    BF16 from the decode's workspace partials and one-split rows `out`, with
    w_uv [H, 128, 512] BF16 (W_UV[h] transposed, latent-contiguous)."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _lib.check("mla_uv_combine", _lib.load().mla_uv_combine(
        ctypes.byref(shape), _ptr(counts), _ptr(work), work.numel(), _ptr(workspace), ws_bytes,
        float(bmm2_scale), _ptr(out), _ptr(w_uv), _ptr(y), _ptr(status), _stream(stream)))


def lse_merge(parts_out, parts_lse, out, lse, stream=None) -> None:
    """Merge S partial results over disjoint key sets: parts_out [S, rows, 512]
    BF16 and parts_lse [S, rows] FP32 log2 -> out [rows, 512], lse [rows]
    (the decode-context-parallel combine; see include/mlafold.h)."""
    S, rows = parts_lse.shape[0], parts_lse.numel() // parts_lse.shape[0]
    _lib.check("mla_lse_merge", _lib.load().mla_lse_merge(
        S, rows, _ptr(parts_out), _ptr(parts_lse), _ptr(out), _ptr(lse), _stream(stream)))


def folded_decode_noalloc(shape: MlaShape, q, kv, block_table, seq_lens, bmm1_scale: float,
                          bmm2_scale: float, counts, work, out, lse, status=None,
                          stream=None) -> None:
    """Decode plus LSE reduction with the library's own fixed device scratch
    (no workspace argument, no allocation): for callers that may not allocate
    device memory. Shapes whose workspace exceeds the library's 64 MiB scratch
    raise MlaError(MLA_ERR_SCRATCH_LIMIT). Calls that overlap on the GPU share
    that scratch and race."""
    _lib.check("mla_folded_decode_noalloc", _lib.load().mla_folded_decode_noalloc(
        ctypes.byref(shape), _ptr(q), _ptr(kv), _ptr(block_table), _ptr(seq_lens),
        float(bmm1_scale), float(bmm2_scale), _ptr(counts), _ptr(work), work.numel(), _ptr(out),
        _ptr(lse), _ptr(status), _stream(stream)))


# The tiered launch's constants. The pages name TIERS and MOVE without values
# (drafter-attention page, `balanced_tiers`, `_balanced_tables`); these are
# this library's: tiers of 8, 16 and 32 rows, and a row moves when it is longer
# than one pair's share of the batch's keys.
TIERS = (8, 16, 32)
MOVE = (1, 1)


def balanced_tiers(rows: int, sms: int, tiers=TIERS) -> tuple:
    """Tier sizes for `rows` decode rows on `sms` SMs (drafter-attention page,
    `balanced_tiers`): none when rows * 4 <= sms, else the sizes of `tiers` in
    order while their sum stays at most rows // 2."""
    if rows * 4 <= sms:
        return ()
    out: list = []
    for size in tiers:
        if sum(out) + size > rows // 2:
            break
        out.append(size)
    return tuple(out)


def tier_plan(rows: int, split_rows: int, pairs: int, move, seq_lens, rest_lens, tier_rows,
              tier_lens, stream=None) -> None:
    """Which rows move into the tiers (see mla_tier_plan in include/mlafold.h)."""
    _lib.check("mla_tier_plan", _lib.load().mla_tier_plan(
        rows, split_rows, pairs, int(move[0]), int(move[1]), _ptr(seq_lens), _ptr(rest_lens),
        _ptr(tier_rows), _ptr(tier_lens), _stream(stream)))


def row_copy(src, dst, index, targets: int, bound: int, gather: bool, stream=None) -> None:
    """Whole-row gather (dst[i] = src[index[i]]) or scatter (dst[index[i]] =
    src[i]) of the rows whose index lies in [0, bound); rows are the leading
    dimension of src and dst (see mla_row_copy in include/mlafold.h)."""
    row_bytes = src[0].numel() * src.element_size()
    if dst[0].numel() * dst.element_size() != row_bytes:
        raise ValueError("src and dst rows differ in size")
    _lib.check("mla_row_copy", _lib.load().mla_row_copy(
        _ptr(src), _ptr(dst), _ptr(index), int(targets), int(bound), int(row_bytes),
        1 if gather else 0, _stream(stream)))


class FoldedMla:
    """Plan buffers and split-KV workspace of one decode shape. `groups` row
    groups per request (a divisor of k): 1 folds all k tokens into one decode
    row, k is the stock unfolded layout, `k // fold_factor(k, H)` the partial
    fold of the pages' `fold_plan`; out and lse keep the same layout.

    Everything is allocated here, before any capture; ``plan`` and ``decode``
    only launch kernels (balanced-MLA page, ``BalancedMla.require``: prepared
    before capture, one shared scratch)."""

    def __init__(self, R: int, k: int, H: int, max_pages: int, num_pages: int,
                 device=None, num_ctas: int | None = None, min_split_tokens: int = 256,
                 max_splits: int = 64, policy: int = POLICY_BALANCED, groups: int = 1):
        self.device = torch.device(device if device is not None else "cuda")
        if num_ctas is None:
            num_ctas = torch.cuda.get_device_properties(self.device).multi_processor_count
        self.shape = make_shape(R, k, H, max_pages, num_pages, num_ctas, min_split_tokens,
                                max_splits, policy, groups)
        self.R, self.k, self.H, self.M = R, k, H, k * H
        self.groups = groups
        i32 = dict(dtype=torch.int32, device=self.device)
        self.counts = torch.zeros(R * groups, **i32)
        self.work = torch.full((plan_list_len(self.shape),), -1, **i32)
        self.workspace = torch.empty(max(workspace_bytes(self.shape), 256), dtype=torch.uint8,
                                     device=self.device)
        self.status = torch.zeros(1, **i32)

    def plan(self, seq_lens, stream=None) -> None:
        plan_splits(self.shape, seq_lens, self.counts, self.work, stream)

    def decode(self, q, kv, block_table, seq_lens, bmm1_scale: float, bmm2_scale: float,
               out=None, lse=None, stream=None, return_lse: bool = True):
        """out [R, M, 512] BF16 and, with return_lse, the base-2 lse [R, M]
        (else None: the no-LSE route, nothing written for it)."""
        if out is None:
            out = torch.empty((self.R, self.M, 512), dtype=torch.bfloat16, device=self.device)
        if lse is None and return_lse:
            lse = torch.empty((self.R, self.M), dtype=torch.float32, device=self.device)
        if not return_lse:
            lse = None
        folded_decode(self.shape, q, kv, block_table, seq_lens, bmm1_scale, bmm2_scale,
                      self.counts, self.work, self.workspace, out, lse, self.status, stream)
        split_combine(self.shape, self.counts, self.work, self.workspace, bmm2_scale, out, lse,
                      stream)
        return out, lse

    def decode_uv(self, q, kv, block_table, seq_lens, bmm1_scale: float, bmm2_scale: float,
                  w_uv, y=None, out=None, stream=None):
        """The decode followed by the split reduction fused with W_UV:
        y [R*k, H, 128] BF16 (w_uv [H, 128, 512] BF16, latent-contiguous).
        `out` receives the one-split requests' rows only; no LSE is written."""
        if out is None:
            out = torch.empty((self.R, self.M, 512), dtype=torch.bfloat16, device=self.device)
        if y is None:
            y = torch.empty((self.R * self.k, self.H, 128), dtype=torch.bfloat16,
                            device=self.device)
        folded_decode(self.shape, q, kv, block_table, seq_lens, bmm1_scale, bmm2_scale,
                      self.counts, self.work, self.workspace, out, None, self.status, stream)
        uv_combine(self.shape, self.counts, self.work, self.workspace, bmm2_scale, out, w_uv, y,
                   self.status, stream)
        return y


class TieredMla:
    """The pages' tiered launch (drafter-attention page, `balanced_decode`),
    built from this library's kernels for comparison with the single
    persistent decode of `FoldedMla`: the longest decode rows move out of one
    unsplit launch into tiers of TIERS rows, each tier a decode launch of its
    own with split rows, on streams of decreasing priority (the unsplit launch
    on the highest, then the tiers from the coarsest split to the finest).

    One folded decode row per request (groups = 1). Split counts: the unsplit
    launch gives every row one split; a tier of m rows gets this library's
    uniform split count for m rows (the pages' stock kernel gives sms // (2m)
    splits: CTA pairs per row split; here the plan's concurrent items per row).
    Every buffer is allocated here, before any capture."""

    def __init__(self, R: int, k: int, H: int, max_pages: int, num_pages: int, device=None,
                 sms: int | None = None, tiers=None, move=MOVE):
        self.device = torch.device(device if device is not None else "cuda")
        if sms is None:
            sms = torch.cuda.get_device_properties(self.device).multi_processor_count
        self.R, self.k, self.H, self.M, self.max_pages = R, k, H, k * H, max_pages
        self.tiers = balanced_tiers(R, sms) if tiers is None else tuple(tiers)
        self.split_rows = sum(self.tiers)
        if self.split_rows > R:
            raise ValueError("the tiers hold more rows than the batch")
        self.pairs = max(1, sms // 2)
        self.move = tuple(move)
        self.unsplit = FoldedMla(R, k, H, max_pages, num_pages, self.device, num_ctas=sms,
                                 max_splits=1, policy=POLICY_UNIFORM)
        self.engines = [FoldedMla(m, k, H, max_pages, num_pages, self.device, num_ctas=sms,
                                  policy=POLICY_UNIFORM) for m in self.tiers]
        n = max(self.split_rows, 1)
        i32 = dict(dtype=torch.int32, device=self.device)
        self.rest = torch.zeros(R, **i32)
        self.tier_rows = torch.full((n,), R, **i32)
        self.tier_lens = torch.zeros(n, **i32)
        self.q_s = torch.empty((n * k, H, 576), dtype=torch.uint8, device=self.device)
        self.bt_s = torch.zeros((n, max_pages), **i32)
        self.out_s = torch.empty((n, self.M, 512), dtype=torch.bfloat16, device=self.device)
        self.lse_s = torch.empty((n, self.M), dtype=torch.float32, device=self.device)
        low, high = torch.cuda.Stream.priority_range()
        self.streams = [torch.cuda.Stream(self.device, priority=min(low, high + i))
                        for i in range(len(self.tiers) + 1)]

    def decode(self, q, kv, block_table, seq_lens, bmm1_scale: float, bmm2_scale: float,
               out=None, lse=None, return_lse: bool = True):
        """out [R, M, 512] BF16 and the base-2 lse [R, M] (None without
        return_lse), as FoldedMla.decode returns them."""
        if out is None:
            out = torch.empty((self.R, self.M, 512), dtype=torch.bfloat16, device=self.device)
        if lse is None and return_lse:
            lse = torch.empty((self.R, self.M), dtype=torch.float32, device=self.device)
        if not return_lse:
            lse = None
        main = torch.cuda.current_stream(self.device)
        R, k, n = self.R, self.k, self.split_rows
        tier_plan(R, n, self.pairs, self.move, seq_lens, self.rest, self.tier_rows,
                  self.tier_lens, main)
        first = self.streams[0]
        first.wait_stream(main)
        self.unsplit.plan(self.rest, first)
        self.unsplit.decode(q, kv, block_table, self.rest, bmm1_scale, bmm2_scale, out=out,
                            lse=lse, stream=first, return_lse=return_lse)
        if n:
            row_copy(q.view(R, -1), self.q_s.view(n, -1), self.tier_rows, n, R, True, main)
            row_copy(block_table, self.bt_s, self.tier_rows, n, R, True, main)
            launches, start = [], 0
            for m, eng in zip(self.tiers, self.engines):
                launches.append((start, m, eng))
                start += m
            for stream, (b, m, eng) in zip(self.streams[1:], reversed(launches)):
                stream.wait_stream(main)
                lens = self.tier_lens[b:b + m]
                eng.plan(lens, stream)
                eng.decode(self.q_s[b * k:(b + m) * k], kv, self.bt_s[b:b + m], lens, bmm1_scale,
                           bmm2_scale, out=self.out_s[b:b + m],
                           lse=self.lse_s[b:b + m] if return_lse else None, stream=stream,
                           return_lse=return_lse)
        for stream in self.streams:
            main.wait_stream(stream)
        if n:
            row_copy(self.out_s, out, self.tier_rows, n, R, False, main)
            if lse is not None:
                row_copy(self.lse_s, lse, self.tier_rows, n, R, False, main)
        return out, lse


# ---------------------------------------------------------------- around the decode
_E4M3 = (torch.uint8, torch.float8_e4m3fn)
_BF16, _F32, _I32 = (torch.bfloat16,), (torch.float32,), (torch.int32,)


def _check(dev: int, name: str, t, dtypes, shape) -> None:
    """`t` is a contiguous tensor of this shape and one of these types on CUDA
    device `dev`; the library sees only its pointer."""
    if isinstance(t, torch.Tensor) and t.get_device() == dev and t.dtype in dtypes and \
            t.shape == shape and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        raise ValueError(f"{name} is not a tensor on cuda:{dev}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has type {t.dtype}, not {dtypes[0]}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {shape}")
    raise ValueError(f"{name} is not contiguous")


def _device(name: str, t, dims: int) -> int:
    """The CUDA device of `t`, a tensor of so many dims."""
    if not isinstance(t, torch.Tensor) or t.get_device() < 0:
        raise ValueError(f"{name} is not a CUDA tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {dims} dims")
    return t.get_device()


def _empty(size, dtype, device, stream):
    """An output for a launch on `stream`, from that stream's memory pool."""
    if stream is None:
        return torch.empty(size, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(size, dtype=dtype, device=device)


def rope_table(rows: int, base: float = 10000.0, device=None) -> torch.Tensor:
    """[rows, 64] FP32: the cosines, then the sines, of position * base^(-2i/64)
    for the 32 planes of the 64 rope dims (angles in 64 bits). Models that scale
    their angles fill a table of this layout themselves."""
    device = torch.device("cuda" if device is None else device)
    inv = base ** (-torch.arange(0, 64, 2, dtype=torch.float64, device=device) / 64)
    angle = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def kv_append(kv_new, kv, block_table, starts, rope, kv_scale: float, norm_weight=None,
              norm_eps: float = 1e-6, cu_tokens=None, rope_starts=None, interleaved: bool = True,
              status=None, stream=None) -> None:
    """Append new tokens to the paged cache kv [pages, 64, 576] (E4M3 codes,
    written in place): kv_new [tokens, 576] BF16 (rows may be strided), latent
    dims normed with norm_weight [512] BF16 (None: no norm), rope dims rotated
    at position rope_starts[r] + i (None: starts), divided by kv_scale. Token i
    of request r goes to cache index starts[r] + i through block_table[r]; a
    request with a negative start is skipped. cu_tokens [R + 1] gives ragged
    requests their rows; without it each has tokens / R. See mla_kv_append in
    include/mlafold.h."""
    dev = _device("kv", kv, 3)
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return kv_append(kv_new, kv, block_table, starts, rope, kv_scale, norm_weight,
                             norm_eps, cu_tokens, rope_starts, interleaved, status, stream)
    _device("block_table", block_table, 2)
    _device("rope", rope, 2)
    R, max_pages = block_table.shape
    pages, rope_rows = kv.shape[0], rope.shape[0]
    _check(dev, "kv", kv, _E4M3, (pages, PAGE, 576))
    _check(dev, "block_table", block_table, _I32, (R, max_pages))
    _check(dev, "starts", starts, _I32, (R,))
    _check(dev, "rope", rope, _F32, (rope_rows, 64))
    if _device("kv_new", kv_new, 2) != dev or kv_new.shape[1] != 576 or \
            kv_new.dtype != torch.bfloat16 or kv_new.stride(1) != 1:
        raise ValueError("kv_new is not [tokens, 576] BF16 with contiguous rows on kv's device")
    if norm_weight is not None:
        _check(dev, "norm_weight", norm_weight, _BF16, (512,))
    if cu_tokens is not None:
        _check(dev, "cu_tokens", cu_tokens, _I32, (R + 1,))
    if rope_starts is not None:
        _check(dev, "rope_starts", rope_starts, _I32, (R,))
    if status is not None:
        _check(dev, "status", status, _I32, (1,))
    tokens = kv_new.shape[0]
    shape = AppendShape(R, tokens, PAGE, max_pages, pages, rope_rows, 1 if interleaved else 0,
                        kv_new.stride(0) if tokens > 1 else 576)
    _lib.check("mla_kv_append", _lib.load().mla_kv_append(
        ctypes.byref(shape), _ptr(kv_new), _ptr(norm_weight), float(norm_eps), _ptr(rope),
        _ptr(cu_tokens), _ptr(starts), _ptr(rope_starts), _ptr(block_table), float(kv_scale),
        _ptr(kv), _ptr(status), _stream(stream)))


def query_absorb(q, w_uk, rope, rope_starts, q_scale: float, out=None, interleaved: bool = True,
                 status=None, stream=None):
    """The decode's queries [R*k, H, 576] (E4M3 codes): q [R*k, H, 192] BF16
    (128 nope, 64 rope dims; tokens and heads may be strided), the nope part
    times w_uk [H, 128, 512] BF16 per head, the rope part rotated at position
    rope_starts[r] + i of token i of request r, divided by q_scale. See
    mla_query_absorb in include/mlafold.h."""
    dev = _device("q", q, 3)
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return query_absorb(q, w_uk, rope, rope_starts, q_scale, out, interleaved, status,
                                stream)
    if q.shape[2] != 192 or q.dtype != torch.bfloat16 or q.stride(2) != 1:
        raise ValueError("q is not [R*k, H, 192] BF16 with contiguous dims")
    _device("rope", rope, 2)
    _device("rope_starts", rope_starts, 1)
    T, H, _ = q.shape
    R, rope_rows = rope_starts.shape[0], rope.shape[0]
    if R < 1 or T < R or T % R:
        raise ValueError(f"{T} tokens are not a positive multiple of {R} requests")
    _check(dev, "rope_starts", rope_starts, _I32, (R,))
    _check(dev, "w_uk", w_uk, _BF16, (H, 128, 512))
    _check(dev, "rope", rope, _F32, (rope_rows, 64))
    if status is not None:
        _check(dev, "status", status, _I32, (1,))
    if out is None:
        out = _empty((T, H, 576), torch.uint8, q.device, stream)
    else:
        _check(dev, "out", out, _E4M3, (T, H, 576))
    shape = QueryShape(R, T // R, H, rope_rows, 1 if interleaved else 0,
                       q.stride(0) if T > 1 else H * 192, q.stride(1) if H > 1 else 192)
    _lib.check("mla_query_absorb", _lib.load().mla_query_absorb(
        ctypes.byref(shape), _ptr(q), _ptr(w_uk), _ptr(rope), _ptr(rope_starts), float(q_scale),
        _ptr(out), _ptr(status), _stream(stream)))
    return out


def query_absorb_wait_test(q, w_uk, rope, rope_starts, q_scale: float, out, status,
                           wait_limit_ns: int, withhold: bool = True, interleaved: bool = True,
                           stream=None) -> None:
    """Failure-detection test hook: query_absorb with every pipeline wait bounded by
    wait_limit_ns and, with `withhold`, CTA 0's first weights never loaded, so that a
    wait runs out and MLA_FAULT_WAIT_TIMEOUT is set in `status` (see include/mlafold.h)."""
    T, H, _ = q.shape
    R = rope_starts.shape[0]
    shape = QueryShape(R, T // R, H, rope.shape[0], 1 if interleaved else 0,
                       q.stride(0) if T > 1 else H * 192, q.stride(1) if H > 1 else 192)
    _lib.check("mla_query_absorb_wait_test", _lib.load().mla_query_absorb_wait_test(
        ctypes.byref(shape), _ptr(q), _ptr(w_uk), _ptr(rope), _ptr(rope_starts), float(q_scale),
        _ptr(out), _ptr(status), 1 if withhold else 0, int(wait_limit_ns), _stream(stream)))


def prefix_workspace_bytes(shape: MlaShape) -> int:
    out = ctypes.c_size_t(0)
    _lib.check("mla_prefix_workspace_bytes", _lib.load().mla_prefix_workspace_bytes(
        ctypes.byref(shape), ctypes.byref(out)))
    return out.value


def prefix_plan(shape: MlaShape, seq_lens, plan, stream=None) -> None:
    """The line of work of the requests' own keys: plan [R + 1] int32 (see
    mla_prefix_plan in include/mlafold.h)."""
    _lib.check("mla_prefix_plan", _lib.load().mla_prefix_plan(
        ctypes.byref(shape), _ptr(seq_lens), _ptr(plan), plan.numel(), _stream(stream)))


def prefix_decode(shape: MlaShape, q, kv, prefix_table, prefix_len, block_table, seq_lens,
                  bmm1_scale: float, bmm2_scale: float, plan, workspace, out, lse, status=None,
                  stream=None) -> None:
    """The shared-prefix decode over the plan of prefix_plan for the requests'
    own lengths; it notes in the plan's first word whether that serves them (see
    mla_prefix_decode in include/mlafold.h)."""
    _lib.check("mla_prefix_decode", _lib.load().mla_prefix_decode(
        ctypes.byref(shape), prefix_table.numel(), _ptr(q), _ptr(kv), _ptr(prefix_table),
        _ptr(prefix_len), _ptr(block_table), _ptr(seq_lens), float(bmm1_scale), float(bmm2_scale),
        _ptr(plan), plan.numel(), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _ptr(out), _ptr(lse), _ptr(status), _stream(stream)))


def prefix_decode_wait_test(shape: MlaShape, q, kv, prefix_table, prefix_len, block_table, seq_lens,
                            bmm1_scale: float, bmm2_scale: float, plan, workspace, out, lse, status,
                            wait_limit_ns: int, stream=None) -> None:
    """Failure-detection test hook: the shared-prefix decode with every pipeline wait
    bounded by wait_limit_ns and CTA 0's first queries withheld, so that a wait runs out
    and MLA_FAULT_WAIT_TIMEOUT is set in `status` (see include/mlafold.h)."""
    _lib.check("mla_prefix_decode_wait_test", _lib.load().mla_prefix_decode_wait_test(
        ctypes.byref(shape), prefix_table.numel(), _ptr(q), _ptr(kv), _ptr(prefix_table),
        _ptr(prefix_len), _ptr(block_table), _ptr(seq_lens), float(bmm1_scale), float(bmm2_scale),
        _ptr(plan), plan.numel(), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _ptr(out), _ptr(lse), _ptr(status), int(wait_limit_ns), _stream(stream)))


class PrefixMla:
    """Decode of a batch of R requests that share a prefix of up to
    prefix_pages pages: plan and workspace of one shape, allocated here and
    reused by every call. ``plan(seq_lens)`` plans the requests' own keys once
    per step (the first ``decode`` does so itself where none was planned);
    ``decode`` attends over the prefix and them. Calls on one object share its
    buffers: they must run in stream order (``status`` is cleared on the stream
    that is current when the object is made)."""

    def __init__(self, R: int, k: int, H: int, max_pages: int, prefix_pages: int, num_pages: int,
                 device=None, num_ctas: int | None = None):
        self.device = torch.device(device if device is not None else "cuda")
        if num_ctas is None:
            num_ctas = torch.cuda.get_device_properties(self.device).multi_processor_count
        self.shape = make_shape(R, k, H, max_pages, num_pages, num_ctas)
        self.R, self.k, self.H, self.M = R, k, H, k * H
        self.max_pages, self.prefix_pages, self.num_pages = max_pages, prefix_pages, num_pages
        self.workspace = torch.empty(prefix_workspace_bytes(self.shape), dtype=torch.uint8,
                                     device=self.device)
        # Not filled: a fill on this stream could come after a plan on another.
        self.places = torch.empty(R + 1, dtype=torch.int32, device=self.device)
        self.planned = False
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)

    def plan(self, seq_lens, stream=None) -> None:
        """Plan the requests' own keys: seq_lens [R] int32."""
        dev = self.places.get_device()
        if dev != torch.cuda.current_device():
            with torch.cuda.device(dev):
                return self.plan(seq_lens, stream)
        _check(dev, "seq_lens", seq_lens, _I32, (self.R,))
        prefix_plan(self.shape, seq_lens, self.places, stream)
        self.planned = True

    def decode(self, q, kv, prefix_table, prefix_len, block_table, seq_lens, bmm1_scale: float,
               bmm2_scale: float, out=None, lse=None, stream=None, return_lse: bool = True):
        """out [R, k*H, 512] BF16 and the base-2 lse [R, k*H] (None without
        return_lse) of queries q [R*k, H, 576] over the prefix (prefix_table
        [prefix_pages] and prefix_len [1], int32) and each request's own keys
        (block_table [R, max_pages], seq_lens [R]). All keys of seq_lens are attended
        to; lengths that need more tiles than the planned ones only take longer."""
        dev = self.places.get_device()
        if dev != torch.cuda.current_device():
            with torch.cuda.device(dev):
                return self.decode(q, kv, prefix_table, prefix_len, block_table, seq_lens,
                                   bmm1_scale, bmm2_scale, out, lse, stream, return_lse)
        R, M = self.R, self.M
        _check(dev, "q", q, _E4M3, (R * self.k, self.H, 576))
        _check(dev, "kv", kv, _E4M3, (self.num_pages, PAGE, 576))
        _check(dev, "prefix_table", prefix_table, _I32, (self.prefix_pages,))
        _check(dev, "prefix_len", prefix_len, _I32, (1,))
        _check(dev, "block_table", block_table, _I32, (R, self.max_pages))
        _check(dev, "seq_lens", seq_lens, _I32, (R,))
        if out is None:
            out = _empty((R, M, 512), torch.bfloat16, q.device, stream)
        else:
            _check(dev, "out", out, _BF16, (R, M, 512))
        if not return_lse:
            lse = None
        elif lse is None:
            lse = _empty((R, M), torch.float32, q.device, stream)
        else:
            _check(dev, "lse", lse, _F32, (R, M))
        if not self.planned:
            self.plan(seq_lens, stream)
        prefix_decode(self.shape, q, kv, prefix_table, prefix_len, block_table, seq_lens,
                      bmm1_scale, bmm2_scale, self.places, self.workspace, out, lse, self.status,
                      stream)
        return out, lse


# ---------------------------------------------------------------- bounding the cache
def kv_weigh(q, kv, block_table, seq_lens, lse, bmm1_scale: float, weights, starts,
             decay: float = 1.0, positions=None, rope_starts=None, status=None, stream=None) -> None:
    """Add to weights [R, max_pages * 64] FP32 (in place) what every cached key got
    from the k*H query rows of its request in a decode with these queries q
    [R*k, H, 576], keys and base-2 lse [R, k*H]: earlier weights times decay, plus
    the sum of 2^(score - lse). Keys at slots from starts[r] on are new: they begin
    with this step's weight, and positions [R, max_pages * 64] int32 (or None) gets
    theirs, counted from rope_starts[r] (None: starts). A request with a negative
    start is skipped. See mla_kv_weigh in include/mlafold.h."""
    dev = _device("kv", kv, 3)
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return kv_weigh(q, kv, block_table, seq_lens, lse, bmm1_scale, weights, starts, decay,
                            positions, rope_starts, status, stream)
    shape = _weigh_shape(dev, q, kv, block_table, seq_lens, lse, weights, starts, positions,
                         rope_starts, status)
    _lib.check("mla_kv_weigh", _lib.load().mla_kv_weigh(
        ctypes.byref(shape), q.data_ptr(), kv.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
        lse.data_ptr(), float(bmm1_scale), float(decay), starts.data_ptr(), _ptr(rope_starts),
        weights.data_ptr(), _ptr(positions), _ptr(status), _stream_on(dev, stream)))


def _weigh_shape(dev, q, kv, block_table, seq_lens, lse, weights, starts, positions, rope_starts,
                 status) -> CacheShape:
    _device("block_table", block_table, 2)
    _device("q", q, 3)
    (R, max_pages), (T, H, _), pages = block_table.shape, q.shape, kv.shape[0]
    if R < 1 or T < R or T % R:
        raise ValueError(f"{T} tokens are not a positive multiple of {R} requests")
    k, slots = T // R, max_pages * PAGE
    _check(dev, "q", q, _E4M3, (T, H, 576))
    _check(dev, "kv", kv, _E4M3, (pages, PAGE, 576))
    _check(dev, "block_table", block_table, _I32, (R, max_pages))
    _check(dev, "seq_lens", seq_lens, _I32, (R,))
    _check(dev, "lse", lse, _F32, (R, k * H))
    _check(dev, "weights", weights, _F32, (R, slots))
    _check(dev, "starts", starts, _I32, (R,))
    if positions is not None:
        _check(dev, "positions", positions, _I32, (R, slots))
    if rope_starts is not None:
        _check(dev, "rope_starts", rope_starts, _I32, (R,))
    if status is not None:
        _check(dev, "status", status, _I32, (1,))
    return CacheShape(R, k, H, PAGE, max_pages, pages)


def kv_weigh_wait_test(q, kv, block_table, seq_lens, lse, bmm1_scale: float, weights, starts, status,
                       wait_limit_ns: int, decay: float = 1.0, positions=None, rope_starts=None,
                       stream=None) -> None:
    """Failure-detection test hook: kv_weigh with every pipeline wait bounded by
    wait_limit_ns and CTA 0's first keys withheld, so that a wait runs out and
    MLA_FAULT_WAIT_TIMEOUT is set in `status` (see include/mlafold.h)."""
    shape = _weigh_shape(_device("kv", kv, 3), q, kv, block_table, seq_lens, lse, weights, starts,
                         positions, rope_starts, status)
    _lib.check("mla_kv_weigh_wait_test", _lib.load().mla_kv_weigh_wait_test(
        ctypes.byref(shape), _ptr(q), _ptr(kv), _ptr(block_table), _ptr(seq_lens), _ptr(lse),
        float(bmm1_scale), float(decay), _ptr(starts), _ptr(rope_starts), _ptr(weights),
        _ptr(positions), _ptr(status), int(wait_limit_ns), _stream(stream)))


@functools.lru_cache(maxsize=64)
def kv_evict_workspace_bytes(R: int, max_pages: int, num_pages: int = 1) -> int:
    out = ctypes.c_size_t(0)
    _lib.check("mla_kv_evict_workspace_bytes", _lib.load().mla_kv_evict_workspace_bytes(
        ctypes.byref(CacheShape(R, 1, 1, PAGE, max_pages, num_pages)), ctypes.byref(out)))
    return out.value


def kv_evict(kv, block_table, seq_lens, weights, keep, positions=None, recent: int = 0,
             sinks: int = 0, weights_out=None, positions_out=None, lens_out=None, workspace=None,
             status=None, stream=None):
    """Keep at most keep[r] keys of every request of the paged cache kv
    [pages, 64, 576]: those of positions below `sinks`, the `recent` newest, then
    those of most weight (ties: the lower slot). Kept keys behind the new length
    move into slots of dropped ones, with their weights and positions
    [R, max_pages * 64] (positions None: a key's position is its slot; else the caller
    has set those of keys that no kv_weigh call counted as new, a prompt's). Returns
    the new lengths [R] int32. weights_out and positions_out may be the inputs, which
    is the default; lens_out may be seq_lens; other overlaps of an output with what it is
    made from are refused, and any of lens_out with keep. `workspace`: uint8, at least
    kv_evict_workspace_bytes (None: allocated for the call). See mla_kv_evict in
    include/mlafold.h."""
    dev = _device("kv", kv, 3)
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return kv_evict(kv, block_table, seq_lens, weights, keep, positions, recent, sinks,
                            weights_out, positions_out, lens_out, workspace, status, stream)
    _device("block_table", block_table, 2)
    (R, max_pages), pages = block_table.shape, kv.shape[0]
    slots = (R, max_pages * PAGE)
    _check(dev, "kv", kv, _E4M3, (pages, PAGE, 576))
    _check(dev, "block_table", block_table, _I32, (R, max_pages))
    _check(dev, "seq_lens", seq_lens, _I32, (R,))
    _check(dev, "weights", weights, _F32, slots)
    _check(dev, "keep", keep, _I32, (R,))
    if weights_out is None:
        weights_out = weights
    else:
        _check(dev, "weights_out", weights_out, _F32, slots)
        _apart("weights_out", weights_out, weights)
    if positions is not None:
        _check(dev, "positions", positions, _I32, slots)
        if positions_out is None:
            positions_out = positions
        else:
            _check(dev, "positions_out", positions_out, _I32, slots)
            _apart("positions_out", positions_out, positions)
    elif positions_out is not None:
        raise ValueError("positions_out without positions")
    if status is not None:
        _check(dev, "status", status, _I32, (1,))
    recent, sinks = int(recent), int(sinks)
    if not (-2 ** 31 <= recent < 2 ** 31 and -2 ** 31 <= sinks < 2 ** 31):
        raise ValueError(f"recent {recent} or sinks {sinks} is no int32")
    if lens_out is None:
        lens_out = _empty((R,), torch.int32, kv.device, stream)
    else:
        _check(dev, "lens_out", lens_out, _I32, (R,))
        _apart("lens_out", lens_out, seq_lens)
        _apart("lens_out", lens_out, keep, same=False)
    if workspace is None:
        workspace = _empty((kv_evict_workspace_bytes(R, max_pages),), torch.uint8, kv.device, stream)
    else:
        _check(dev, "workspace", workspace, (torch.uint8,), workspace.shape)
    _lib.check("mla_kv_evict", _lib.load().mla_kv_evict(
        ctypes.byref(CacheShape(R, 1, 1, PAGE, max_pages, pages)), kv.data_ptr(),
        block_table.data_ptr(), seq_lens.data_ptr(), weights.data_ptr(), _ptr(positions),
        keep.data_ptr(), recent, sinks, weights_out.data_ptr(), _ptr(positions_out),
        lens_out.data_ptr(), workspace.data_ptr(), workspace.numel(), _ptr(status),
        _stream_on(dev, stream)))
    return lens_out


def _stream_on(dev: int, stream) -> int:
    """The stream's handle; None: the current one of device `dev`."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def _apart(name: str, t, other, same: bool = True) -> None:
    """`t` is `other` itself (where `same`), or shares no memory with it (both contiguous)."""
    a, b = t.data_ptr(), other.data_ptr()
    if not (same and a == b) and a < b + other.numel() * other.element_size() and \
            b < a + t.numel() * t.element_size():
        raise ValueError(f"{name} overlaps its input")


# ---------------------------------------------------------------- the prompt
def prompt_workspace_bytes(R: int, num_ctas: int | None = None, device=None) -> int:
    """Bytes of the workspace of prompt_attention for R requests (num_ctas None: the
    device's SM count, as the call takes it)."""
    if num_ctas is None:
        num_ctas = torch.cuda.get_device_properties(
            torch.device("cuda" if device is None else device)).multi_processor_count
    return _prompt_bytes(R, num_ctas)


@functools.lru_cache(maxsize=64)
def _prompt_bytes(R: int, num_ctas: int) -> int:
    shape = PromptShape(R, 1, 1, 1, 1, 1, num_ctas, 192, 192, 128, 128, 128, 128, 64)
    out = ctypes.c_size_t(0)
    _lib.check("mla_prompt_workspace_bytes", _lib.load().mla_prompt_workspace_bytes(
        ctypes.byref(shape), ctypes.byref(out)))
    return out.value


def prompt_attention(q, k_nope, k_rope, v, cu_tokens, sm_scale: float, cu_keys=None,
                     causal: bool = True, out=None, lse=None, return_lse: bool = True,
                     workspace=None, status=None, stream=None):
    """Attention over packed prompts: out [tokens, H, 128] BF16 and the base-2 lse
    [tokens, H] (None without return_lse) of q [tokens, H, 192] BF16 (128 nope, 64
    rotated rope dims) over k_nope and v [keys, kv_heads, 128] and k_rope [keys, 64]
    (rotated, one vector for all heads), BF16; tokens and heads of all may be strided.
    Request r has rows cu_tokens[r] .. cu_tokens[r + 1] of q and cu_keys[r] .. of the keys
    (None: the same). Causal: token i of n sees keys j <= i + m - n of m. Rows that
    belong to no request are not written. `workspace`: uint8, at least
    prompt_workspace_bytes (None: allocated for the call). See mla_prompt_attention in
    include/mlafold.h."""
    dev = _device("q", q, 3)
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return prompt_attention(q, k_nope, k_rope, v, cu_tokens, sm_scale, cu_keys, causal, out,
                                    lse, return_lse, workspace, status, stream)
    shape = _prompt_shape(dev, q, k_nope, k_rope, v, cu_tokens, cu_keys, causal, status)
    T, H = q.shape[:2]
    if out is None:
        out = _empty((T, H, 128), torch.bfloat16, q.device, stream)
    else:
        _check(dev, "out", out, _BF16, (T, H, 128))
    if not return_lse:
        lse = None
    elif lse is None:
        lse = _empty((T, H), torch.float32, q.device, stream)
    else:
        _check(dev, "lse", lse, _F32, (T, H))
    if workspace is None:
        workspace = _empty((_prompt_bytes(shape.R, shape.num_ctas),), torch.uint8, q.device, stream)
    else:
        _check(dev, "workspace", workspace, (torch.uint8,), workspace.shape)
    _lib.check("mla_prompt_attention", _lib.load().mla_prompt_attention(
        ctypes.byref(shape), q.data_ptr(), k_nope.data_ptr(), k_rope.data_ptr(), v.data_ptr(),
        cu_tokens.data_ptr(), _ptr(cu_keys), float(sm_scale), workspace.data_ptr(), workspace.numel(),
        out.data_ptr(), _ptr(lse), _ptr(status), _stream_on(dev, stream)))
    return out, lse


@functools.lru_cache(maxsize=None)
def _sms(dev: int) -> int:
    return torch.cuda.get_device_properties(dev).multi_processor_count


def _prompt_shape(dev, q, k_nope, k_rope, v, cu_tokens, cu_keys, causal, status) -> PromptShape:
    bf16 = torch.bfloat16
    for name, t, dims, width in (("q", q, 3, 192), ("k_nope", k_nope, 3, 128), ("k_rope", k_rope, 2, 64),
                                 ("v", v, 3, 128)):
        if not isinstance(t, torch.Tensor) or t.dim() != dims or t.get_device() != dev or \
                t.dtype is not bf16 or t.shape[-1] != width or t.stride(-1) != 1:
            raise ValueError(f"{name} is not a tensor of {dims} dims, the last {width} BF16 elements in a "
                             f"row, on cuda:{dev}")
    (T, H, _), (Tk, Hkv, _) = q.shape, k_nope.shape
    if v.shape != k_nope.shape or k_rope.shape[0] != Tk:
        raise ValueError(f"v {tuple(v.shape)} and k_rope {tuple(k_rope.shape)} do not go with k_nope "
                         f"{tuple(k_nope.shape)}")
    if not isinstance(cu_tokens, torch.Tensor) or cu_tokens.dim() != 1 or cu_tokens.shape[0] < 2:
        raise ValueError("cu_tokens is not [R + 1] int32")
    R1 = cu_tokens.shape[0]
    _check(dev, "cu_tokens", cu_tokens, _I32, (R1,))
    if cu_keys is not None:
        _check(dev, "cu_keys", cu_keys, _I32, (R1,))
    elif Tk != T:
        raise ValueError(f"{Tk} keys for {T} tokens without cu_keys")
    if status is not None:
        _check(dev, "status", status, _I32, (1,))
    # The stride over a dim of one element is never used: any that the library takes will do.
    q0, q1, _ = q.stride()
    k0, k1, _ = k_nope.stride()
    v0, v1, _ = v.stride()
    if T < 2:
        q0 = H * 192
    if H < 2:
        q1 = 192
    r0 = k_rope.stride(0)
    if Tk < 2:
        k0 = v0 = Hkv * 128
        r0 = 64
    if Hkv < 2:
        k1 = v1 = 128
    return PromptShape(R1 - 1, T, Tk, H, Hkv, 1 if causal else 0, _sms(dev), q0, q1, k0, k1, v0, v1, r0)


def prompt_attention_wait_test(q, k_nope, k_rope, v, cu_tokens, sm_scale: float, out, lse, workspace,
                               status, wait_limit_ns: int, cu_keys=None, causal: bool = True,
                               stream=None) -> None:
    """Failure-detection test hook: prompt_attention with every pipeline wait bounded
    by wait_limit_ns and CTA 0's first keys withheld, so that a wait runs out and
    MLA_FAULT_WAIT_TIMEOUT is set in `status` (see include/mlafold.h)."""
    shape = _prompt_shape(_device("q", q, 3), q, k_nope, k_rope, v, cu_tokens, cu_keys, causal, status)
    _lib.check("mla_prompt_attention_wait_test", _lib.load().mla_prompt_attention_wait_test(
        ctypes.byref(shape), _ptr(q), _ptr(k_nope), _ptr(k_rope), _ptr(v), _ptr(cu_tokens),
        _ptr(cu_keys), float(sm_scale), _ptr(workspace), workspace.numel(), _ptr(out), _ptr(lse),
        _ptr(status), int(wait_limit_ns), _stream(stream)))
