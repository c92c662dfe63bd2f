"""Device-side state and call sequencing for MLA decode through libxmla.

Holds the caller-owned buffers the C ABI expects (paged latent cache, block
table, sequence lengths, weights, workspace, output) and issues the library
calls in decode order.  No arithmetic of the method happens here.

One decode step over a layer ("the hot path"):
  1. xmla_cache_append of the step's q_len new tokens per sequence, rotating
     their k_pe with YaRN RoPE as it stores [c_kv | rotated k_pe],
  2. xmla_decode (q absorb with RoPE of q_pe -> split-K latent attention ->
     combine with W_UV).
With the 8-bit cache (cache="q8") the same two steps run as
xmla_cache_append_q8 and xmla_decode_q8 over a [num_blocks, 64, 608] byte pool.
A batch whose sequences begin with the same cache pages decodes through
SharedDecoder (xmla_decode_shared); norm_rope_rows and append_normed_rows norm
queries and new keys on the way, and read_back_q8 turns a context of the 8-bit
cache into bf16 pages, which a prompt chunk needs.
"""
from __future__ import annotations

import contextlib
from dataclasses import dataclass

import torch

from . import xmla
from .workloads import (D_LATENT, D_NOPE, D_ROPE, D_V, N_HEADS, PAGE, LayerInputs, Workload,
                        new_token_rows)


def num_sms(device=None) -> int:
    return torch.cuda.get_device_properties(device or torch.cuda.current_device()).multi_processor_count


@dataclass
class LayerState:
    pool: torch.Tensor         # [num_blocks, 64, 576] bf16
    block_table: torch.Tensor  # [B, max_blocks] int32
    seqlens: torch.Tensor      # [B] int32
    W_UK: torch.Tensor
    W_UV: torch.Tensor
    num_blocks: int
    max_blocks: int
    cache: str = "bf16"        # "bf16" or "q8" (pool [num_blocks, 64, 608] uint8)


def new_pool(num_blocks: int, device, fill: float | None = 0.0) -> torch.Tensor:
    if fill is None:
        return torch.empty((num_blocks, PAGE, D_LATENT + D_ROPE), dtype=torch.bfloat16, device=device)
    return torch.full((num_blocks, PAGE, D_LATENT + D_ROPE), fill, dtype=torch.bfloat16, device=device)


Q8_ROW = 608  # bytes of an 8-bit cache row (include/xmla.h)


def new_pool_q8(num_blocks: int, device) -> torch.Tensor:
    return torch.zeros((num_blocks, PAGE, Q8_ROW), dtype=torch.uint8, device=device)


def rope_rows(cfg, x: torch.Tensor, positions: torch.Tensor, stream=None) -> None:
    """Rotate, in place, the rope part of q [R, H, 192] or of k_pe [T, 64]."""
    if x.dim() == 3:
        R, H, D = x.shape
        xmla.xmla_rope_yarn(cfg, x, R, H, D, H * D, D_NOPE, positions, stream)
    else:
        T, D = x.shape
        xmla.xmla_rope_yarn(cfg, x, T, 1, D, D, 0, positions, stream)


@dataclass
class NewTokens:
    """The q_len newest tokens of every sequence: what one decode step appends."""

    c_kv: torch.Tensor       # [B*q_len, 512] bf16
    k_pe: torch.Tensor       # [B*q_len, 64] bf16, not rotated
    positions: torch.Tensor  # [B*q_len] int64
    seq_ids: torch.Tensor    # [B*q_len] int32


def split_prefix(wl: Workload, inp: LayerInputs) -> tuple[LayerInputs, NewTokens]:
    """Split a layer's token rows into the cached prefix and the step's new tokens."""
    T = inp.c_kv.shape[0]
    dev = inp.c_kv.device
    new_rows = torch.tensor(new_token_rows(wl, inp.offsets), dtype=torch.int64, device=dev)
    keep = torch.ones(T, dtype=torch.bool, device=dev)
    keep[new_rows] = False
    prefix = LayerInputs(q=inp.q, c_kv=inp.c_kv[keep], k_pe=inp.k_pe[keep], W_UK=inp.W_UK,
                         W_UV=inp.W_UV, block_table=inp.block_table, seqlens=inp.seqlens,
                         seq_ids=inp.seq_ids[keep], positions=inp.positions[keep],
                         num_blocks=inp.num_blocks, offsets=inp.offsets)
    new = NewTokens(c_kv=inp.c_kv[new_rows].contiguous(), k_pe=inp.k_pe[new_rows].contiguous(),
                    positions=inp.positions[new_rows].contiguous(),
                    seq_ids=inp.seq_ids[new_rows].contiguous())
    return prefix, new


def build_layer(cfg, wl: Workload, inp: LayerInputs, device, chunk: int = 1 << 20,
                pool_fill: float | None = 0.0, status: torch.Tensor | None = None,
                cache: str = "bf16") -> LayerState:
    """Upload one layer's inputs and fill its paged cache with every token of
    every sequence (RoPE on k_pe, then append), in chunks of `chunk` tokens.
    cache="q8": the 8-bit pool, filled through xmla_cache_append_q8."""
    q8 = cache == "q8"
    pool = new_pool_q8(inp.num_blocks, device) if q8 else new_pool(inp.num_blocks, device, pool_fill)
    append = xmla.xmla_cache_append_q8 if q8 else xmla.xmla_cache_append
    bt = inp.block_table.to(device)
    T = inp.c_kv.shape[0]
    for t0 in range(0, T, chunk):
        t1 = min(T, t0 + chunk)
        c = inp.c_kv[t0:t1].to(device, non_blocking=True)
        k = inp.k_pe[t0:t1].to(device, non_blocking=True).contiguous()
        pos = inp.positions[t0:t1].to(device)
        sid = inp.seq_ids[t0:t1].to(device)
        append(pool, inp.num_blocks, bt, bt.shape[1], wl.batch, sid, pos, c, k, cfg, t1 - t0,
               status)
    return LayerState(pool=pool, block_table=bt, seqlens=inp.seqlens.to(device),
                      W_UK=inp.W_UK.to(device), W_UV=inp.W_UV.to(device),
                      num_blocks=inp.num_blocks, max_blocks=bt.shape[1], cache=cache)


class Decoder:
    """Workspace and output buffers for xmla_decode at fixed sizes."""

    def __init__(self, batch: int, q_len: int, max_seqlen: int, device, num_splits: int = 0,
                 cache: str = "bf16"):
        self.batch, self.q_len, self.max_seqlen = batch, q_len, max_seqlen
        self.num_splits = num_splits
        self.cache = cache
        self.sms = num_sms(device)
        ws = xmla.xmla_decode_q8_workspace_size if cache == "q8" else xmla.xmla_decode_workspace_size
        self.ws_bytes = ws(batch, q_len, max_seqlen, self.sms, num_splits)
        if self.ws_bytes == 0:
            raise ValueError("unsupported decode sizes")
        self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=device)
        self.out = torch.empty((batch, q_len, N_HEADS, D_V), dtype=torch.bfloat16, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    @property
    def splits(self) -> int:
        f = xmla.xmla_decode_q8_num_splits if self.cache == "q8" else xmla.xmla_decode_num_splits
        return f(self.batch, self.q_len, self.max_seqlen, self.sms, self.num_splits)

    def decode(self, cfg, st: LayerState, q: torch.Tensor, softmax_scale: float, out=None,
               stream=None, events=None) -> torch.Tensor:
        """xmla_decode on raw q (q_pe rotated inside); `events` = (start, stop) CUDA
        events recorded around the split-K attention kernel (xmla_decode_profiled)."""
        out = self.out if out is None else out
        ev = events or (None, None)
        f = xmla.xmla_decode_q8_profiled if st.cache == "q8" else xmla.xmla_decode_profiled
        f(cfg, q, st.W_UK, st.W_UV, st.pool, st.num_blocks, st.block_table, st.max_blocks,
          st.seqlens, self.batch, self.q_len, self.max_seqlen, softmax_scale, self.num_splits,
          self.workspace, self.ws_bytes, self.status, out, stream, ev[0], ev[1])
        return out

    def step(self, cfg, st: LayerState, q: torch.Tensor, c_new: torch.Tensor,
             k_new: torch.Tensor, new_pos: torch.Tensor, new_seq: torch.Tensor,
             softmax_scale: float, out=None, stream=None, events=None,
             fused: bool = True) -> torch.Tensor:
        """One decode step on raw q: the q_len newest tokens (c_new, k_new raw)
        are appended with their rope keys rotated, then the layer attends.
        fused=True uses xmla_decode_step (append inside the first kernel);
        fused=False issues xmla_cache_append and then xmla_decode_profiled.  On the
        8-bit cache the append is always its own call (xmla_cache_append_q8)."""
        out = self.out if out is None else out
        if not fused or st.cache == "q8":
            append = xmla.xmla_cache_append_q8 if st.cache == "q8" else xmla.xmla_cache_append
            append(st.pool, st.num_blocks, st.block_table, st.max_blocks, self.batch, new_seq,
                   new_pos, c_new, k_new, cfg, c_new.shape[0], self.status, stream)
            return self.decode(cfg, st, q, softmax_scale, out, stream, events)
        ev = events or (None, None)
        xmla.xmla_decode_step(cfg, q, st.W_UK, st.W_UV, st.pool, st.num_blocks, st.block_table,
                              st.max_blocks, st.seqlens, self.batch, self.q_len, self.max_seqlen,
                              new_seq, new_pos, c_new, k_new, c_new.shape[0], softmax_scale,
                              self.num_splits, self.workspace, self.ws_bytes, self.status, out,
                              stream, ev[0], ev[1])
        return out

    def step_from_hidden(self, cfg, st: LayerState, q: torch.Tensor, hidden: torch.Tensor,
                         W_kva: torch.Tensor, new_pos: torch.Tensor, new_seq: torch.Tensor,
                         softmax_scale: float, out=None, stream=None, events=None,
                         bias: torch.Tensor | None = None) -> torch.Tensor:
        """One decode step from the new tokens' hidden states: their cache rows
        are produced (kv_a_proj_with_mqa, RoPE, append), then the layer attends."""
        out = self.out if out is None else out
        ev = events or (None, None)
        xmla.xmla_decode_step_from_hidden(cfg, q, st.W_UK, st.W_UV, hidden, W_kva, bias, st.pool,
                                          st.num_blocks, st.block_table, st.max_blocks,
                                          st.seqlens, self.batch, self.q_len, self.max_seqlen,
                                          new_seq, new_pos, hidden.shape[0], softmax_scale,
                                          self.num_splits, self.workspace, self.ws_bytes,
                                          self.status, out, stream, ev[0], ev[1])
        return out

    def check_status(self) -> int:
        return int(self.status.item())


class SharedDecoder:
    """Workspace and output buffers for xmla_decode_shared at fixed sizes: a batch
    whose sequences share their first prefix_pages cache pages."""

    def __init__(self, batch: int, q_len: int, prefix_pages: int, max_seqlen: int, device):
        self.batch, self.q_len, self.max_seqlen = batch, q_len, max_seqlen
        self.prefix_pages = prefix_pages
        self.ws_bytes = xmla.xmla_decode_shared_workspace_size(batch, q_len, prefix_pages,
                                                               max_seqlen, num_sms(device))
        if self.ws_bytes == 0:
            raise ValueError("unsupported shared-prefix decode sizes")
        self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=device)
        self.out = torch.empty((batch, q_len, N_HEADS, D_V), dtype=torch.bfloat16, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def decode(self, cfg, st: LayerState, prefix_table: torch.Tensor, q: torch.Tensor,
               softmax_scale: float, out=None, stream=None) -> torch.Tensor:
        """xmla_decode_shared on raw q (cfg None: q_pe is rotated already);
        st.seqlens are whole lengths, st.block_table is indexed by logical page.
        st's cache is the bf16 one (a page of the 8-bit pool is about half as long:
        read as bf16 rows it would end outside the pool)."""
        if st.cache != "bf16":
            raise ValueError("the shared-prefix decode reads a bf16 cache (read_back_q8 makes one)")
        units = self.batch * self.q_len
        _row(prefix_table, torch.int32, self.prefix_pages, "prefix_table")
        _row(q, torch.bfloat16, units * N_HEADS * (D_NOPE + D_ROPE), "q")
        if st.seqlens.numel() < self.batch or st.block_table.numel() < self.batch * st.max_blocks:
            raise ValueError(f"the state has fewer than {self.batch} sequences")
        if out is None:
            out = self.out
        else:
            _row(out, torch.bfloat16, units * N_HEADS * D_V, "out")
        xmla.xmla_decode_shared(cfg, q, st.W_UK, st.W_UV, st.pool, st.num_blocks, prefix_table,
                                self.prefix_pages, st.block_table, st.max_blocks, st.seqlens,
                                self.batch, self.q_len, self.max_seqlen, softmax_scale,
                                self.workspace, self.ws_bytes, self.status, out, stream)
        return out

    def check_status(self) -> int:
        return int(self.status.item())


def _on(stream):
    """What is allocated and filled inside belongs to `stream` (None: the current one)."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(stream if hasattr(stream, "cuda_stream")
                             else torch.cuda.ExternalStream(int(stream)))


class _Column:
    """The address of t's column c, for a library call (a slice of t costs the host 2 us,
    a quarter of the smallest append)."""

    def __init__(self, t: torch.Tensor, c: int):
        self.address = t.data_ptr() + c * t.element_size()

    def data_ptr(self) -> int:
        return self.address


def _row(t: torch.Tensor, dtype: torch.dtype, n: int, name: str) -> None:
    """t holds at least n values of dtype, one behind the other."""
    if t.dtype is not dtype or t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{name} must hold {n} values of {dtype}, one behind the other: "
                         f"it is {t.dtype} {tuple(t.shape)} with strides {t.stride()}")


def norm_rope_rows(cfg, x: torch.Tensor, weight: torch.Tensor | None, eps: float,
                   positions: torch.Tensor | None = None, out=None, stream=None) -> torch.Tensor:
    """Norm of every head of x [R, H, D] (weight [D] or [H, D]) and, with a cfg, the
    rotation of its last 64 values; x and out may be strided in R and H."""
    R, H, D = x.shape
    if out is None:
        with _on(stream):
            out = torch.empty((R, H, D), dtype=x.dtype, device=x.device)
    elif out.shape != x.shape or out.dtype is not x.dtype:
        raise ValueError(f"out is {out.dtype} {tuple(out.shape)}, x {x.dtype} {tuple(x.shape)}")
    if x.dtype is not torch.bfloat16:
        raise ValueError(f"x is {x.dtype}, not bfloat16")
    x_row, x_head, x_in = x.stride()
    o_row, o_head, o_in = out.stride()
    if D > 1 and (x_in != 1 or o_in != 1):
        raise ValueError("a head's values must be adjacent")
    wh = 0
    if weight is not None:
        if weight.dim() == 2:
            wh = weight.stride(0)
            if weight.shape != (H, D) or weight.dtype is not x.dtype or (D > 1 and weight.stride(1) != 1):
                raise ValueError("a weight of each head must be bfloat16 [H, D], its values adjacent")
        elif weight.dim() != 1 or weight.shape[0] != D:
            raise ValueError(f"weight is {tuple(weight.shape)}, neither ({D},) nor ({H}, {D})")
        else:
            _row(weight, torch.bfloat16, D, "weight")
    if cfg is not None and positions is not None:
        _row(positions, torch.int64, R, "positions")
    xmla.xmla_norm_rope(cfg, x, x_row, x_head, out, o_row, o_head, R, H, D, weight, wh, eps,
                        D - D_ROPE if cfg is not None else 0, positions, stream)
    return out


def append_normed_rows(cfg, st: LayerState, kv: torch.Tensor, kv_weight: torch.Tensor,
                       pe_weight: torch.Tensor | None, eps: float, positions: torch.Tensor,
                       seq_ids: torch.Tensor, status=None, stream=None) -> None:
    """Norm, rotate and append the rows of a raw key projection kv [T, 576] =
    [c_kv | k_pe] (rows at any multiple of 8 values, a row's values adjacent) to st's
    cache (bf16 or 8-bit)."""
    T, width = kv.shape
    stride, inner = kv.stride()
    if width < D_LATENT + D_ROPE or inner != 1 or kv.dtype is not torch.bfloat16:
        raise ValueError("kv must be bfloat16 [T, 576] with a row's values adjacent")
    _row(kv_weight, torch.bfloat16, D_LATENT, "kv_weight")
    if pe_weight is not None:
        _row(pe_weight, torch.bfloat16, D_ROPE, "pe_weight")
    _row(positions, torch.int64, T, "positions")
    _row(seq_ids, torch.int32, T, "seq_ids")
    if T == 1:
        stride = D_LATENT + D_ROPE  # (torch gives a single row any stride)
    append = xmla.xmla_cache_append_norm_q8 if st.cache == "q8" else xmla.xmla_cache_append_norm
    append(st.pool, st.num_blocks, st.block_table, st.max_blocks, st.block_table.shape[0], seq_ids,
           positions, kv, stride, _Column(kv, D_LATENT), stride, kv_weight, pe_weight, eps, cfg, T,
           status, stream)


def read_back_q8(st: LayerState, seqlens: list[int], status=None, stream=None) -> LayerState:
    """The sequences of an 8-bit cache (their first seqlens[b] tokens) as a bf16 cache
    of consecutive pages, on which any xmla_decode call on `stream` runs."""
    if st.cache != "q8":
        raise ValueError("the rows of an 8-bit cache are read back; this one is bf16 already")
    if len(seqlens) > st.block_table.shape[0] or any(not 0 <= n <= st.max_blocks * PAGE for n in seqlens):
        # (their rows would be skipped and read as zeros)
        raise ValueError("more sequences, or longer ones, than the cache's block table has")
    dev = st.pool.device
    pages = [(n + PAGE - 1) // PAGE for n in seqlens]
    first = [sum(pages[:b]) for b in range(len(pages))]
    table = torch.zeros((len(pages), max(pages + [1])), dtype=torch.int32)
    for b, n in enumerate(pages):
        table[b, :n] = torch.arange(first[b], first[b] + n, dtype=torch.int32)
    with _on(stream):
        # rows past a sequence's last token read nothing and stay zero
        pool = new_pool(max(sum(pages), 1), dev)
        for b, n in enumerate(seqlens):
            ids = torch.full((n,), b, dtype=torch.int32, device=dev)
            xmla.xmla_cache_read_q8(st.pool, st.num_blocks, st.block_table, st.max_blocks,
                                    st.block_table.shape[0], ids, torch.arange(n, device=dev), n,
                                    pool[first[b]:], D_LATENT + D_ROPE, status, stream)
        return LayerState(pool=pool, block_table=table.to(dev),
                          seqlens=torch.tensor(seqlens, dtype=torch.int32, device=dev),
                          W_UK=st.W_UK, W_UV=st.W_UV, num_blocks=pool.shape[0],
                          max_blocks=table.shape[1])
