"""Device-resident batch for the libdsa calls: tensors, dims and workspace.

``DecodeBatch.from_workload`` copies a batch drawn by ``workloads.generate`` to
the GPU once; its methods are one-line calls of the C ABI through the ctypes
binding.  PyTorch provides the device memory and the stream, nothing else.
"""
from __future__ import annotations

import contextlib
import copy
import math

import numpy as np
import torch

from . import dsa


def _i32(x, device):
    return torch.as_tensor(np.ascontiguousarray(x, dtype=np.int32)).to(device)


@contextlib.contextmanager
def _made_on(stream):
    """Tensors made inside belong to `stream` (None: the current one), which the call that writes them
    is launched on: their memory was free there and is free again, in its order, when the caller
    lets go of them.  On a stream that records a graph nothing can be allocated; what a recorded
    call writes comes from the current stream, and the caller keeps it as long as the graph."""
    if stream is None:
        yield
        return
    with torch.cuda.stream(stream):
        if not torch.cuda.is_current_stream_capturing():
            yield
            return
    yield


def estimated_kept_rows(lengths) -> np.ndarray:
    """Upper estimate of each request's kept rows, min(P,L) + min(W, L-1-min(P,L)) + 1,
    from host arrays (seq_len, prompt_len, window)."""
    L, P, W = (np.asarray(x, dtype=np.int64) for x in lengths)
    npr = np.minimum(P, L)
    return npr + np.minimum(np.maximum(L - 1 - npr, 0), W) + 1


def longest_first_order(lengths) -> np.ndarray:
    """int32 permutation of the requests by decreasing estimated kept rows (ties
    by index)."""
    return np.argsort(-estimated_kept_rows(lengths), kind="stable").astype(np.int32)


def schedule_order(lengths, spread: float = 1.25):
    """The request_order a serving host would pass: longest first when the
    estimated kept rows of the batch vary (max > spread * mean), else None
    (batch order; an order costs each CTA one dependent load)."""
    est = estimated_kept_rows(lengths)
    if est.size == 0 or est.max() <= spread * est.mean():
        return None
    return longest_first_order(lengths)


def page_rows(page_table, seq_len, num_pages) -> np.ndarray:
    """Rows that each page of a pool holds: of the requests that map it, the most (host arrays;
    entries of -1 and entries past a request's rows are not looked at)."""
    table, L = np.asarray(page_table), np.asarray(seq_len, dtype=np.int64)
    if L.size and L.max() > table.shape[1] * dsa.PAGE:
        raise ValueError(f"seq_len {L.max()} passes the page table's {table.shape[1]} pages")
    n = np.clip(L[:, None] - dsa.PAGE * np.arange(table.shape[1]), 0, dsa.PAGE)
    used = (n > 0) & (table >= 0)
    if used.any() and table[used].max() >= num_pages:
        raise ValueError(f"page id {table[used].max()} outside the pool of {num_pages}")
    rows = np.zeros(num_pages, np.int32)
    np.maximum.at(rows, table[used], n[used])
    return rows


def shared_groups(page_table, seq_len):
    """(group_start, prefix_len) for DecodeBatch.share_prefix from host arrays: runs of neighbouring
    requests whose tables begin with the same whole pages, cut so that the pages a step reads once
    instead of per request are the most there can be (of two such cuts the one with the longer
    group at the end).  Whether the shared calls are then faster than the plain ones is the
    caller's to say: dsa_shared_prefix in include/dsa.h says from how many rows on."""
    table, L = np.asarray(page_table), np.asarray(seq_len, dtype=np.int64)
    B, whole = len(L), np.maximum(L, 0) // dsa.PAGE
    common = np.zeros(B, np.int64)  # whole pages that request b begins with like request b - 1
    for b in range(1, B):
        n = int(min(whole[b - 1], whole[b], table.shape[1]))
        same = (table[b, :n] == table[b - 1, :n]) & (table[b, :n] >= 0)
        common[b] = n if same.all() else int(np.argmin(same))
    # Requests i .. j have the least of common[i + 1 .. j] pages in common.  best[j]: the pages that
    # requests 0 .. j - 1 save; at[j]: where their last group starts.
    best, at, pages = np.zeros(B + 1, np.int64), np.zeros(B + 1, np.int64), np.zeros(B, np.int64)
    run = 0  # no group reaches across two neighbours with nothing in common
    for b in range(B):
        if common[b] == 0:
            run = b
        pages[run:b] = np.minimum(pages[run:b], common[b])
        pages[b] = whole[b]
        saved = best[run:b + 1] + (b - np.arange(run, b + 1)) * pages[run:b + 1]
        at[b + 1] = run + int(np.argmax(saved))
        best[b + 1] = saved[at[b + 1] - run]
    start, rows = [B], np.zeros(B, np.int32)
    while start[-1] > 0:
        j = start[-1]
        i = int(at[j])
        if j - i > 1:  # a request alone shares nothing
            rows[i:j] = dsa.PAGE * int(common[i + 1:j].min())
        start.append(i)
    return np.array(start[::-1] if B else [0], dtype=np.int32), rows


class PackedIO:
    """One pinned host buffer and one device buffer per direction, so that a
    step's inputs go up in one copy and its results come back in one.  The
    batch's tensors become views into the device buffers."""

    def __init__(self, inputs: dict, outputs: dict, device):
        def layout(tensors):
            offs, at = {}, 0
            for name, t in tensors.items():
                offs[name] = at
                at += (t.numel() * t.element_size() + 255) // 256 * 256
            return offs, max(at, 256)
        self._in_off, n_in = layout(inputs)
        self._out_off, n_out = layout(outputs)
        self.dev_in = torch.empty(n_in, dtype=torch.uint8, device=device)
        self.dev_out = torch.empty(n_out, dtype=torch.uint8, device=device)
        self.host_in = torch.empty(n_in, dtype=torch.uint8).pin_memory()
        self.host_out = torch.empty(n_out, dtype=torch.uint8).pin_memory()
        self.dev, self.host = {}, {}
        for offs, dbuf, hbuf, tensors in ((self._in_off, self.dev_in, self.host_in, inputs),
                                          (self._out_off, self.dev_out, self.host_out, outputs)):
            for name, t in tensors.items():
                nb = t.numel() * t.element_size()
                o = offs[name]
                self.dev[name] = dbuf[o:o + nb].view(t.dtype).view(t.shape)
                self.host[name] = hbuf[o:o + nb].view(t.dtype).view(t.shape)
                self.dev[name].copy_(t)
                self.host[name].copy_(t.cpu())
        self.h2d_bytes = n_in
        self.d2h_bytes = n_out

    def upload(self):
        self.dev_in.copy_(self.host_in, non_blocking=True)

    def download(self):
        self.host_out.copy_(self.dev_out, non_blocking=True)

    def descriptor(self) -> dsa.dsa_host_io:
        """The two copies as a dsa_host_io, for the calls that issue them
        themselves (dsa_decode_sparse_masked_io)."""
        return dsa.host_io(self.host_in, self.dev_in, self.dev_out, self.host_out)


class DecodeBatch:
    def __init__(self, *, q, k_pages, v_pages, page_table, seq_len, prompt_len, window,
                 grid_w, keep_mask, max_window, mask_words, max_kept, device="cuda"):
        self.device = torch.device(device)
        self.q = q.to(self.device).contiguous()
        self.k_pages = k_pages.to(self.device).contiguous()
        self.v_pages = v_pages.to(self.device).contiguous()
        self.page_table = _i32(page_table, self.device)
        self.seq_len = _i32(seq_len, self.device)
        self.prompt_len = _i32(prompt_len, self.device)
        self.window = _i32(window, self.device)
        self.grid_w = _i32(grid_w, self.device)
        self._host_lengths = tuple(np.array(x, dtype=np.int32, copy=True)
                                   for x in (seq_len, prompt_len, window))
        B, Hq, D = self.q.shape
        num_pages, page, Hkv, _ = self.k_pages.shape
        self.batch, self.hq, self.hkv, self.head_dim = B, Hq, Hkv, D
        if keep_mask is None:
            keep_mask = np.zeros((B, Hkv, mask_words), dtype=np.uint32)
        self.keep_mask = torch.as_tensor(
            np.ascontiguousarray(keep_mask, dtype=np.uint32).view(np.int32)).to(self.device)
        self.dims = dsa.make_dims(B, Hq, Hkv, D, num_pages, self.page_table.shape[1], max_window,
                                  mask_words, max_kept, self.q.dtype, self.k_pages.dtype)
        self.scale = 1.0 / math.sqrt(D)
        self.ws = dsa.alloc_workspace(self.dims, self.device)
        self.kept_idx = torch.zeros((B, Hkv, max_kept), dtype=torch.int32, device=self.device)
        self.kept_cnt = torch.zeros((B, Hkv), dtype=torch.int32, device=self.device)
        self.out = torch.empty((B, Hq, D), dtype=torch.float32, device=self.device)
        self.lse = torch.empty((B, Hq), dtype=torch.float32, device=self.device)

    @classmethod
    def from_workload(cls, w: dict, device="cuda", keep_mask=None):
        return cls(q=w["q"], k_pages=w["k_pages"], v_pages=w["v_pages"],
                   page_table=w["page_table"], seq_len=w["seq_len"], prompt_len=w["prompt_len"],
                   window=w["window"], grid_w=w["grid_w"],
                   keep_mask=w["keep_mask"] if keep_mask is None else keep_mask,
                   max_window=w["max_window"], mask_words=w["mask_words"],
                   max_kept=w["max_kept"], device=device)

    def replicate(self) -> "DecodeBatch":
        """A second slot for the same batch shape: the KV cache is shared (not
        copied); the step inputs, kept lists, outputs and workspace are its own
        copies, so that two steps can be in flight at once (double-buffered
        host I/O: one slot's copies overlap the other's kernels)."""
        other = copy.copy(self)
        for name in ("q", "page_table", "seq_len", "prompt_len", "window", "grid_w", "keep_mask",
                     "kept_idx", "kept_cnt", "out", "lse", "ws"):
            setattr(other, name, getattr(self, name).clone())
        other.out_q = None
        other._host_lengths = tuple(x.copy() for x in self._host_lengths)
        return other

    def set_keep_mask(self, keep_mask):
        self.keep_mask.copy_(torch.as_tensor(
            np.ascontiguousarray(keep_mask, dtype=np.uint32).view(np.int32)))

    # -- the C ABI calls --------------------------------------------------
    def build_index(self, stream=None):
        dsa.dsa_build_index(self.dims, self.seq_len, self.prompt_len, self.window, self.keep_mask,
                            self.kept_idx, self.kept_cnt, self.ws, stream)

    def evict_pages(self, capacity=None, stream=None):
        """Unmap the pages no later step reads; returns (freed page ids tensor,
        count tensor) -- the ids are valid up to min(count, capacity)."""
        cap = self.page_table.numel() if capacity is None else capacity
        with _made_on(stream):
            freed = torch.full((max(cap, 1),), -1, dtype=torch.int32, device=self.device)
            count = torch.zeros(1, dtype=torch.int32, device=self.device)
        dsa.dsa_evict_pages(self.dims, self.seq_len, self.prompt_len, self.window, self.page_table,
                            freed[:cap] if cap > 0 else None, count, self.ws, stream)
        return freed, count

    def decode_sparse(self, out=None, lse=None, stream=None):
        out = self.out if out is None else out
        lse = self.lse if lse is None else lse
        dsa.dsa_decode_sparse(self.dims, self.q, self.k_pages, self.v_pages, self.page_table,
                              self.seq_len, self.kept_idx, self.kept_cnt, self.scale, out, lse,
                              self.ws, stream)
        return out, lse

    def decode_sparse_masked(self, out=None, lse=None, stream=None, request_order=None,
                             k_new=None, v_new=None):
        out = self.out if out is None else out
        lse = self.lse if lse is None else lse
        dsa.dsa_decode_sparse_masked(self.dims, self.q, self.k_pages, self.v_pages,
                                     self.page_table, self.seq_len, self.prompt_len, self.window,
                                     self.keep_mask, self.scale, out, lse, self.ws, stream,
                                     request_order, k_new, v_new)
        return out, lse

    def decode_step_io(self, io: PackedIO, request_order=None, stream=None, k_pages=None,
                       v_pages=None, prepare=False):
        """One step from host memory in one C call: io's inputs up, the fused
        sparse decode, out and lse back into io.host.  The batch must have been
        packed by pack_io(io); k_pages / v_pages default to the batch's cache.
        With prepare=True returns a dsa.Prepared that issues the step per call."""
        return dsa.dsa_decode_sparse_masked_io(
            io.descriptor(), self.dims, self.q, self.k_pages if k_pages is None else k_pages,
            self.v_pages if v_pages is None else v_pages, self.page_table, self.seq_len,
            self.prompt_len, self.window, self.keep_mask, self.scale, self.out, self.lse, self.ws,
            stream, request_order, prepare=prepare)

    def record_step_io(self, io: PackedIO, stream, request_order=None, k_pages=None,
                       v_pages=None) -> dsa.Graph:
        """decode_step_io recorded once as a dsa.Graph on `stream` (a non-default
        torch.cuda.Stream): each graph.launch(stream) uploads io's inputs, runs
        the fused decode and downloads out and lse, for one host launch."""
        dsa.dsa_graph_begin(stream)
        try:
            self.decode_step_io(io, request_order, stream, k_pages, v_pages)
        except BaseException:
            try:  # end the recording so that the stream is usable again
                dsa.dsa_graph_end(stream).close()
            except dsa.DSAError:
                pass
            raise
        graph = dsa.dsa_graph_end(stream)
        return graph.keep(io, request_order, k_pages, v_pages, self)

    def longest_first_order(self):
        """Requests by decreasing estimated kept rows: the request_order that
        shortens the tail of a mixed batch (host-side; the serving host knows
        these lengths when it builds the batch)."""
        return longest_first_order(self._host_lengths)

    def schedule_order(self):
        """longest_first_order() when the batch's lengths vary, else None."""
        return schedule_order(self._host_lengths)

    def pack_io(self, order=None) -> tuple:
        """Move the step's inputs (q, lengths, masks, page table, order) and
        results (out, lse) into packed buffers; returns the PackedIO and the
        device order tensor (or None)."""
        inputs = {"q": self.q, "seq_len": self.seq_len, "prompt_len": self.prompt_len,
                  "window": self.window, "keep_mask": self.keep_mask,
                  "page_table": self.page_table}
        if order is not None:
            inputs["order"] = torch.as_tensor(np.asarray(order, dtype=np.int32))
        io = PackedIO(inputs, {"out": self.out, "lse": self.lse}, self.device)
        self.q, self.seq_len, self.prompt_len = io.dev["q"], io.dev["seq_len"], io.dev["prompt_len"]
        self.window, self.keep_mask = io.dev["window"], io.dev["keep_mask"]
        self.page_table = io.dev["page_table"]
        self.out, self.lse = io.dev["out"], io.dev["lse"]
        return io, io.dev.get("order")

    def decode_dense(self, out=None, lse=None, stream=None):
        out = self.out if out is None else out
        lse = self.lse if lse is None else lse
        dsa.dsa_decode_dense(self.dims, self.q, self.k_pages, self.v_pages, self.page_table,
                             self.seq_len, self.scale, out, lse, self.ws, stream)
        return out, lse

    def share_prefix(self, group_start, prefix_len, max_suffix=None, max_prefix=None, masked=False):
        """dsa_shared_prefix for the *_shared calls from host arrays (see shared_groups): the requests
        group_start[g] .. group_start[g+1] - 1 have their first prefix_len rows in common.  The bounds
        default to those of the batch's lengths as they were given (with masked, of the rows that the
        masked call can keep); a batch that goes on growing passes its own."""
        group_start, prefix_len = (np.asarray(x, dtype=np.int32) for x in (group_start, prefix_len))
        if max_suffix is None:
            rows = estimated_kept_rows(self._host_lengths) if masked else self._host_lengths[0]
            max_suffix = int((rows - prefix_len).max(initial=0))
        if max_prefix is None:
            max_prefix = int(prefix_len.max(initial=0))
        return dsa.shared_prefix(_i32(group_start, self.device), _i32(prefix_len, self.device), max_prefix,
                                 max_suffix)

    def _out_of_q(self, out, stream):
        """Where a call on `stream` whose out has q's type writes it."""
        if out is not None:
            return out
        if getattr(self, "out_q", None) is None or self.out_q.dtype is not self.q.dtype:
            with _made_on(stream):
                self.out_q = torch.empty_like(self.q)
        return self.out_q

    def decode_dense_shared(self, shared, out=None, lse=None, stream=None):
        """decode_dense, a shared prefix once for its group; out has q's type (bf16)."""
        out, lse = self._out_of_q(out, stream), self.lse if lse is None else lse
        dsa.dsa_decode_dense_shared(self.dims, shared, self.q, self.k_pages, self.v_pages, self.page_table,
                                    self.seq_len, self.scale, out, lse, self.ws, stream)
        return out, lse

    def decode_sparse_masked_shared(self, shared, out=None, lse=None, stream=None):
        """decode_sparse_masked, a shared prefix of the prompts once for its group; out has q's
        type (bf16)."""
        out, lse = self._out_of_q(out, stream), self.lse if lse is None else lse
        dsa.dsa_decode_sparse_masked_shared(self.dims, shared, self.q, self.k_pages, self.v_pages,
                                            self.page_table, self.seq_len, self.prompt_len, self.window,
                                            self.keep_mask, self.scale, out, lse, self.ws, stream)
        return out, lse

    def write_rows(self, row_slot, k, v, stream=None):
        """Store rows k and v [tokens, hkv, d] at their slots (PagePool.assign)."""
        dsa.dsa_write_rows(self.dims, row_slot, k, v, self.k_pages, self.v_pages, self.ws, stream)

    def attention_mass(self, r_local=2, r_diag=2, with_offsets=True, stream=None):
        om = None
        with _made_on(stream):
            mass = torch.empty((self.batch, self.hq, 4), dtype=torch.float32, device=self.device)
            if with_offsets:
                om = torch.empty((self.batch, self.hq, self.dims.max_window + 1),
                                 dtype=torch.float32, device=self.device)
        dsa.dsa_attention_mass(self.dims, self.q, self.k_pages, self.page_table, self.seq_len,
                               self.prompt_len, self.window, self.grid_w, r_local, r_diag,
                               self.scale, mass, om, self.ws, stream)
        return mass, om

    def device_error(self) -> int:
        return dsa.dsa_get_device_error(self.ws)

    def check(self, what="libdsa"):
        dsa.check_device_error(self.ws, what)


class PagePool:
    """The free pages of a cache, on the GPU: eviction appends to the list, new rows take their
    pages from its end."""

    def __init__(self, num_pages, used=(), device="cuda"):
        free = np.setdiff1d(np.arange(num_pages), np.asarray(used, dtype=np.int64))[::-1]
        self.free = torch.full((max(num_pages, 1),), -1, dtype=torch.int32, device=device)
        self.free[:len(free)] = _i32(free, self.free.device)
        self.count = torch.full((1,), len(free), dtype=torch.int32, device=device)

    def assign(self, batch: DecodeBatch, new_len=None, max_tokens=None, stream=None):
        """Pages for the last new_len[b] rows of the batch's requests (its seq_len counts them; None:
        one row each) into its page table.  Returns (token_start, row_slot, row_pos): the packed new
        rows' slots and positions; max_tokens places (default: the sum of new_len, which reads it
        back)."""
        dev = batch.device
        if max_tokens is None:
            max_tokens = batch.batch if new_len is None else int(new_len.sum())
        with _made_on(stream):
            start = torch.empty(batch.batch + 1, dtype=torch.int32, device=dev)
            slot, pos = (torch.empty(max_tokens, dtype=torch.int32, device=dev) for _ in range(2))
        dsa.dsa_assign_pages(batch.dims, batch.seq_len, new_len, self.free, self.count, self.count,
                             batch.page_table, start, slot, pos, batch.ws, stream)
        return start, slot, pos

    def evict(self, batch: DecodeBatch, stream=None):
        """Take back the pages that no later step of the batch reads."""
        dsa.dsa_evict_pages(batch.dims, batch.seq_len, batch.prompt_len, batch.window, batch.page_table,
                            self.free, self.count, batch.ws, stream)


class QuantBatch:
    """The K/V cache of a DecodeBatch in 8 bits: e4m3 codes [num_pages, hkv, 16, d] and
    power-of-two scales [num_pages, hkv] (dsa_quant_cache).  Lengths, masks, page
    table and workspace are the batch's own; out has q's type.  The batch keeps its
    pages beside it (both forms of a cache for comparison); a program that wants the
    memory of the 8-bit form alone makes the tensors itself (dsa.quant_cache) and
    calls dsa.dsa_*_quant."""

    def __init__(self, batch: DecodeBatch):
        self.batch = batch
        d, dev = batch.dims, batch.device
        shape = (d.num_pages, d.hkv, dsa.PAGE, d.head_dim)
        self.k, self.v = (torch.zeros(shape, dtype=torch.uint8, device=dev)
                          .view(torch.float8_e4m3fn) for _ in range(2))
        self.k_scale, self.v_scale = (torch.ones(shape[:2], dtype=torch.float32, device=dev)
                                      for _ in range(2))
        self.cache = dsa.quant_cache(self.k, self.v, self.k_scale, self.v_scale)
        self.out = torch.empty_like(batch.q)
        self.lse = torch.empty_like(batch.lse)

    @classmethod
    def from_batch(cls, batch: DecodeBatch) -> "QuantBatch":
        """The batch's own pages quantised, with the lengths and the page table that are on the
        device now: every page is written like a request of its own, with as many rows as the
        longest request that maps it has there."""
        self = cls(batch)
        d = batch.dims
        rows = page_rows(batch.page_table.cpu().numpy(), batch.seq_len.cpu().numpy(), d.num_pages)
        used = np.flatnonzero(rows)
        dims = dsa.make_dims(len(used), d.hkv, d.hkv, d.head_dim, d.num_pages, 1, 0, 1, 1,
                             d.kv_dtype, d.kv_dtype)
        at = torch.as_tensor(used, device=batch.device)
        n = _i32(rows[used], batch.device)
        ws = dsa.alloc_workspace(dims, batch.device)
        dsa.dsa_quant_write(dims, self.cache, batch.k_pages[at], batch.v_pages[at],
                            at.to(torch.int32)[:, None].contiguous(), n, n, ws)
        dsa.check_device_error(ws, "QuantBatch.from_batch")
        return self

    def write(self, k_new, v_new, new_len=None, stream=None):
        """Append k_new / v_new [batch, max_new, hkv, d] as the last rows of the requests."""
        b = self.batch
        dsa.dsa_quant_write(b.dims, self.cache, k_new, v_new, b.page_table, b.seq_len, new_len,
                            b.ws, stream)

    def read(self, row_start, row_count, k_out, v_out, stream=None):
        b = self.batch
        dsa.dsa_quant_read(b.dims, self.cache, b.page_table, b.seq_len, row_start, row_count, k_out,
                           v_out, b.ws, stream)

    def decode_dense(self, out=None, lse=None, stream=None):
        b, out, lse = self.batch, self.out if out is None else out, self.lse if lse is None else lse
        dsa.dsa_decode_dense_quant(b.dims, b.q, self.cache, b.page_table, b.seq_len, b.scale, out,
                                   lse, b.ws, stream)
        return out, lse

    def decode_sparse(self, out=None, lse=None, stream=None):
        """Over the batch's kept lists (DecodeBatch.build_index)."""
        b, out, lse = self.batch, self.out if out is None else out, self.lse if lse is None else lse
        dsa.dsa_decode_sparse_quant(b.dims, b.q, self.cache, b.page_table, b.seq_len, b.kept_idx,
                                    b.kept_cnt, b.scale, out, lse, b.ws, stream)
        return out, lse

    def decode_sparse_masked(self, out=None, lse=None, stream=None, request_order=None):
        b, out, lse = self.batch, self.out if out is None else out, self.lse if lse is None else lse
        dsa.dsa_decode_sparse_masked_quant(b.dims, b.q, self.cache, b.page_table, b.seq_len,
                                           b.prompt_len, b.window, b.keep_mask, b.scale, out, lse,
                                           b.ws, stream, request_order)
        return out, lse

    def prefill_sparse(self, q, q_len, out, lse, stream=None, request_order=None):
        b = self.batch
        dsa.dsa_prefill_sparse_quant(b.dims, q, self.cache, b.page_table, b.seq_len, q_len,
                                     b.prompt_len, b.window, b.keep_mask, b.scale, out, lse, b.ws,
                                     stream, request_order)
        return out, lse
