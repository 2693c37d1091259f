"""Buffer management around the C ABI for one mapped prefill layer (allocation and calls only).

``PrefillLayer`` owns the device buffers of one (sender layer, receiver layer) pair with fixed
packed sequence lengths and runs the hot path through libiamap:

    compress(q, k)          -> lse, block masses, BSR index and bf16 tiles (no host sync)
    mapped_av(W, v)         -> out [n, H_r, d_v]
    step(q, k, W, v)        -> both

The value buffer is sized for the worst case (every head keeps every causal block) unless a
capacity is given, so the step needs no host synchronisation.
"""

from __future__ import annotations

import torch

from . import iamap as C


class PrefillLayer:
    def __init__(self, seqlens, H_s, d, H_r, d_v, tau, bias_window=0, bias_value=0.0, B=64,
                 capacity_tiles=None, device="cuda", H_kv=None):
        self.seqlens = [int(x) for x in seqlens]
        self.num_seqs = len(self.seqlens)
        cu = [0]
        for L in self.seqlens:
            cu.append(cu[-1] + L)
        self.cu_host = torch.tensor(cu, dtype=torch.int32)
        self.cu = self.cu_host.to(device)
        self.n = cu[-1]
        self.H_s, self.d, self.H_r, self.d_v, self.B = H_s, d, H_r, d_v, B
        self.H_kv = H_r if H_kv is None else int(H_kv)   # receiver value heads (grouped if < H_r)
        self.tau, self.bias_window, self.bias_value = float(tau), int(bias_window), float(bias_value)
        self.nrb, self.ncb, self.max_nb = C.iamap_plan(self.cu_host, self.num_seqs, B)
        self.bufs = C.alloc_compress_outputs(self.n, H_s, self.nrb, self.ncb, device)
        cap = H_s * self.ncb if capacity_tiles is None else int(capacity_tiles)
        self.capacity = cap
        self.vals = torch.empty(max(cap, 1), B, B, dtype=torch.bfloat16, device=device)
        self.ws = C.alloc_workspace(C.iamap_compress_workspace_bytes(self.num_seqs, self.nrb),
                                    device)
        self.out = torch.empty(self.n, H_r, d_v, dtype=torch.float32, device=device)

    def compress(self, q, k, stream=None):
        b = self.bufs
        C.iamap_compress(q, k, self.cu, self.cu_host, self.num_seqs, self.n, self.H_s, self.d,
                         self.B, self.tau, self.bias_window, self.bias_value, b["lse"], b["mass"],
                         b["headmask_dense"], b["row_ptr"], b["col_idx"], b["headmask"],
                         b["val_off"], b["counts"], self.vals, self.capacity, self.ws, stream)

    def mapped_av(self, W, v, stream=None, out=None):
        b = self.bufs
        out = self.out if out is None else out
        C.iamap_mapped_av_gqa(self.cu, self.cu_host, self.num_seqs, self.n, self.B, self.H_s,
                              b["row_ptr"], b["col_idx"], b["headmask"], b["val_off"], self.vals,
                              self.capacity, W, self.H_r, self.H_kv, v, self.d_v, out, self.ws,
                              stream)
        return out

    def step(self, q, k, W, v, stream=None, out=None):
        self.compress(q, k, stream)
        return self.mapped_av(W, v, stream, out)

    def compress_with_output(self, q, k, v_s, o_s, stream=None):
        """compress plus the sender's own attention output o_s [n, H_s, d_vs] from its values
        v_s [n, H_s, d_vs] (same pass over the keys)."""
        b = self.bufs
        C.iamap_compress_with_output(q, k, self.cu, self.cu_host, self.num_seqs, self.n,
                                     self.H_s, self.d, self.B, self.tau, self.bias_window,
                                     self.bias_value, v_s, int(v_s.shape[2]), o_s, b["lse"],
                                     b["mass"], b["headmask_dense"], b["row_ptr"], b["col_idx"],
                                     b["headmask"], b["val_off"], b["counts"], self.vals,
                                     self.capacity, self.ws, stream)
        return o_s

    def counts(self):
        """(nnz_blocks, nnz_tiles) -- synchronises."""
        c = self.bufs["counts"].cpu()
        return int(c[0]), int(c[1])


class ChunkPrefillLayer:
    """Buffers of one chunked-prefill step of a mapped layer pair: the query rows
    [starts[s], ends[s]) of every sequence s against its keys [0, ends[s]) (earlier chunks'
    keys and values cached). starts[s] is a multiple of B. Optionally (d_vs given) the sender's
    own attention output of the chunk rows is produced with the map.

        compress(q, k, v_s=None) -> lse, masses, BSR map of the chunk rows (+ o_s)
        mapped_av(W, v)          -> out [n_q, H_r, d_v]

    q holds the chunk rows packed by cu_q; k, v (and v_s) hold rows [0, ends[s]) packed by cu_k.
    """

    def __init__(self, starts, ends, H_s, d, H_r, d_v, tau, bias_window=0, bias_value=0.0, B=64,
                 capacity_tiles=None, device="cuda", H_kv=None, d_vs=None):
        self.starts = [int(x) for x in starts]
        self.ends = [int(x) for x in ends]
        self.num_seqs = len(self.starts)
        cu_q, cu_k = [0], [0]
        for c0, e in zip(self.starts, self.ends):
            cu_q.append(cu_q[-1] + e - c0)
            cu_k.append(cu_k[-1] + e)
        self.cu_q_host = torch.tensor(cu_q, dtype=torch.int32)
        self.cu_k_host = torch.tensor(cu_k, dtype=torch.int32)
        self.starts_host = torch.tensor(self.starts, dtype=torch.int32)
        self.cu_q = self.cu_q_host.to(device)
        self.cu_k = self.cu_k_host.to(device)
        self.starts_dev = self.starts_host.to(device)
        self.n_q, self.n_k = cu_q[-1], cu_k[-1]
        self.H_s, self.d, self.H_r, self.d_v, self.B = H_s, d, H_r, d_v, B
        self.H_kv = H_r if H_kv is None else int(H_kv)
        self.tau, self.bias_window, self.bias_value = float(tau), int(bias_window), float(bias_value)
        self.nrb, self.ncb, self.max_nb = C.iamap_chunk_plan(self.cu_q_host, self.cu_k_host,
                                                             self.starts_host, self.num_seqs, B)
        self.bufs = C.alloc_compress_outputs(self.n_q, H_s, self.nrb, self.ncb, device)
        cap = H_s * self.ncb if capacity_tiles is None else int(capacity_tiles)
        self.capacity = cap
        self.vals = torch.empty(max(cap, 1), B, B, dtype=torch.bfloat16, device=device)
        self.ws = C.alloc_workspace(C.iamap_compress_workspace_bytes(self.num_seqs, self.nrb),
                                    device)
        self.out = torch.empty(self.n_q, H_r, d_v, dtype=torch.float32, device=device)
        self.d_vs = None if d_vs is None else int(d_vs)
        self.o_s = (None if d_vs is None else
                    torch.empty(self.n_q, H_s, self.d_vs, dtype=torch.float32, device=device))

    def compress(self, q, k, v_s=None, stream=None):
        b = self.bufs
        C.iamap_compress_chunk(q, k, self.cu_q, self.cu_k, self.starts_dev, self.cu_q_host,
                               self.cu_k_host, self.starts_host, self.num_seqs, self.n_q,
                               self.n_k, self.H_s, self.d, self.B, self.tau, self.bias_window,
                               self.bias_value, v_s, self.d_vs or 0,
                               self.o_s if v_s is not None else None, b["lse"], b["mass"],
                               b["headmask_dense"], b["row_ptr"], b["col_idx"], b["headmask"],
                               b["val_off"], b["counts"], self.vals, self.capacity, self.ws,
                               stream)

    def mapped_av(self, W, v, stream=None, out=None):
        b = self.bufs
        out = self.out if out is None else out
        C.iamap_mapped_av_chunk(self.cu_q, self.cu_k, self.starts_dev, self.cu_q_host,
                                self.cu_k_host, self.starts_host, self.num_seqs, self.n_q,
                                self.n_k, self.B, self.H_s, b["row_ptr"], b["col_idx"],
                                b["headmask"], b["val_off"], self.vals, self.capacity, W,
                                self.H_r, self.H_kv, v, self.d_v, out, self.ws, stream)
        return out

    def step(self, q, k, W, v, v_s=None, stream=None, out=None):
        self.compress(q, k, v_s, stream)
        return self.mapped_av(W, v, stream, out)

    def counts(self):
        """(nnz_blocks, nnz_tiles) -- synchronises."""
        c = self.bufs["counts"].cpu()
        return int(c[0]), int(c[1])


class DecodeStep:
    """Buffers of one paged decode step on a mapped layer."""

    def __init__(self, batch, H_s, H_r, d_v, ctx_lens_host, ctx_stride, max_pages, page_size,
                 num_pages, device="cuda", H_kv=None):
        self.batch, self.H_s, self.H_r, self.d_v = batch, H_s, H_r, d_v
        self.H_kv = H_r if H_kv is None else int(H_kv)
        self.ctx_lens_host = torch.as_tensor(ctx_lens_host, dtype=torch.int32).cpu()
        self.ctx_lens = self.ctx_lens_host.to(device)
        self.ctx_stride, self.max_pages, self.page_size = ctx_stride, max_pages, page_size
        self.num_pages = num_pages
        max_ctx = int(self.ctx_lens_host.max())
        self.ws = C.alloc_workspace(
            C.iamap_mapped_av_paged_workspace_bytes(batch, H_r, d_v, max_ctx, page_size), device)
        self.out = torch.empty(batch, H_r, d_v, dtype=torch.float32, device=device)

    def run(self, p_rows, W, v_pages, page_table, stream=None):
        C.iamap_mapped_av_paged_gqa(p_rows, self.ctx_stride, W, v_pages, self.num_pages,
                                    page_table, self.max_pages, self.page_size, self.ctx_lens,
                                    self.ctx_lens_host, self.batch, self.H_s, self.H_r, self.H_kv,
                                    self.d_v, self.out, self.ws, stream)
        return self.out


def _expect(name, t, dtype, shape, device):
    """A tensor that the library will read through its address alone: right type, shape, device,
    and packed."""
    if (t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous()):
        return
    raise ValueError("%s must be a contiguous %s tensor of shape %s on %s, got %s %s on %s" % (
        name, dtype, tuple(shape), device, t.dtype, tuple(t.shape), t.device))


class QuantCache:
    """A paged cache of keys or values held in 8 or 4 bits: `num_pages` pages of `page_size` tokens,
    H heads of d elements (groups of 32 with one fp16 scale each; include/iamap.h states the
    format). ``over`` makes one of buffers that the caller already has.

        write(x, cu, starts, page_table)       new rows of packed sequences into their pages
        read(cu, starts, page_table, out)      ranges of sequences as packed bf16 rows
    """

    def __init__(self, num_pages, page_size, H, d, bits, device="cuda"):
        if bits not in (4, 8):
            raise ValueError("a cache holds 4 or 8 bits an element")
        if d not in (64, 128):
            raise ValueError("head dim must be 64 or 128")
        self._own(*C.alloc_quant_cache(num_pages, page_size, H, d, bits, device), bits)

    @classmethod
    def over(cls, codes, scales, bits):
        """The cache whose buffers are `codes` uint8 [num_pages, H, page_size, d * bits / 8] and
        `scales` fp16 [num_pages, H, page_size, d / 32]."""
        self = cls.__new__(cls)
        self._own(codes, scales, bits)
        return self

    def _own(self, codes, scales, bits):
        if codes.dim() != 4 or bits not in (4, 8):
            raise ValueError("codes [num_pages, H, page_size, d * bits / 8] in 4 or 8 bits expected")
        self.num_pages, self.H, self.page_size = (int(x) for x in codes.shape[:3])
        self.d, self.bits = int(codes.shape[3]) * 8 // bits, bits
        self.device = codes.device
        _expect("codes", codes, torch.uint8, tuple(codes.shape), self.device)
        _expect("scales", scales, torch.float16,
                (self.num_pages, self.H, self.page_size, self.d // 32), self.device)
        self.codes, self.scales = codes, scales

    def _ranges(self, cu, starts, page_table):
        num_seqs = starts.numel()
        _expect("cu", cu, torch.int32, (num_seqs + 1,), self.device)
        _expect("starts", starts, torch.int32, (num_seqs,), self.device)
        return num_seqs, self._table(page_table, num_seqs)

    def _table(self, page_table, num_seqs):
        """Checks a page table; its pages per sequence."""
        if self.device.index != torch._C._cuda_getDevice():
            raise ValueError("the cache lies on %s, which is not the current device" % self.device)
        shape = page_table.shape
        if len(shape) != 2:
            raise ValueError("page_table must be [sequences, max_pages]")
        _expect("page_table", page_table, torch.int32, (num_seqs, shape[1]), self.device)
        return shape[1]

    def write(self, x, cu, starts, page_table, stream=None):
        """Quantises row cu[s] + i of x as token starts[s] + i of sequence s. x: bf16 [n, H, d] or
        [n, H * d]; its rows may lie further apart than H * d (a slice of a fused projection).
        cu int32 [num_seqs + 1], starts int32 [num_seqs] and page_table int32
        [num_seqs, max_pages] on the device."""
        num_seqs, max_pages = self._ranges(cu, starts, page_table)
        shape, stride = x.shape, x.stride()
        n, width = shape[0], self.H * self.d
        packed = ((shape[1:] == (width,) and stride[1:] == (1,))
                  or (shape[1:] == (self.H, self.d) and stride[2] == 1
                      and (self.H == 1 or stride[1] == self.d)))
        if x.dtype is not torch.bfloat16 or x.device != self.device or not (packed or n == 0):
            raise ValueError("x must be bf16 [n, H, d] or [n, H * d] on %s with packed rows"
                             % self.device)
        C.iamap_cache_write(x, stride[0] if n > 1 else width, n, cu, starts, num_seqs,
                            page_table, max_pages, self.page_size, self.num_pages,
                            self.H, self.d, self.bits, self.codes, self.scales, stream)

    def read(self, cu, starts, page_table, out, stream=None):
        """Fills row cu[s] + i of out (bf16 [n, H, d]) with token starts[s] + i of sequence s and
        returns out; rows behind the last sequence stay as they are."""
        num_seqs, max_pages = self._ranges(cu, starts, page_table)
        n = out.shape[0]
        _expect("out", out, torch.bfloat16, (n, self.H, self.d), self.device)
        C.iamap_cache_read(self.codes, self.scales, self.num_pages, page_table,
                           max_pages, self.page_size, cu, starts, num_seqs, n, self.H,
                           self.d, self.bits, out, stream)
        return out


class QuantSenderRows:
    """Buffers of the small model's attention rows over a quantised key cache (H_k key heads,
    grouped if fewer than H_s): run(q, cache, page_table, ctx_lens) -> rows
    [batch, H_s, ctx_stride], the p_rows of a mapped decode step. ctx_lens stays on the device;
    max_ctx bounds it."""

    def __init__(self, batch, H_s, d, max_ctx, H_k=None, ctx_stride=None, device="cuda"):
        self.batch, self.H_s, self.d, self.max_ctx = batch, H_s, d, int(max_ctx)
        self.H_k = H_s if H_k is None else int(H_k)
        self.ctx_stride = max(1, self.max_ctx) if ctx_stride is None else int(ctx_stride)
        self.ws = C.alloc_workspace(
            C.iamap_sender_rows_quant_workspace_bytes(batch, H_s, self.max_ctx), device)
        self.rows = torch.empty(batch, H_s, self.ctx_stride, dtype=torch.float32, device=device)

    def run(self, q, cache, page_table, ctx_lens, stream=None):
        dev = self.rows.device
        _expect("q", q, torch.bfloat16, (self.batch, self.H_s, self.d), dev)
        _expect("ctx_lens", ctx_lens, torch.int32, (self.batch,), dev)
        _same_cache(cache, self.H_k, self.d, dev)
        max_pages = cache._table(page_table, self.batch)
        C.iamap_sender_rows_quant(q, cache.codes, cache.scales, cache.num_pages, page_table,
                                  max_pages, cache.page_size, ctx_lens, self.max_ctx,
                                  self.batch, self.H_s, self.H_k, self.d, cache.bits, self.rows,
                                  self.ctx_stride, self.ws, stream)
        return self.rows


class QuantDecodeStep:
    """Buffers of one decode step on a mapped layer over a quantised value cache:
    run(p_rows, W, cache, page_table, ctx_lens) -> out [batch, H_r, d_v]."""

    def __init__(self, batch, H_s, H_r, d_v, max_ctx, H_kv=None, ctx_stride=None, device="cuda"):
        self.batch, self.H_s, self.H_r, self.d_v = batch, H_s, H_r, d_v
        self.max_ctx = int(max_ctx)
        self.H_kv = H_r if H_kv is None else int(H_kv)
        self.ctx_stride = max(1, self.max_ctx) if ctx_stride is None else int(ctx_stride)
        self.ws = C.alloc_workspace(
            C.iamap_mapped_av_paged_quant_workspace_bytes(batch, H_r, d_v, self.max_ctx), device)
        self.out = torch.empty(batch, H_r, d_v, dtype=torch.float32, device=device)

    def run(self, p_rows, W, cache, page_table, ctx_lens, stream=None):
        dev = self.out.device
        _expect("p_rows", p_rows, torch.float32, (self.batch, self.H_s, self.ctx_stride), dev)
        _expect("W", W, torch.float32, (self.H_r, self.H_s), dev)
        _expect("ctx_lens", ctx_lens, torch.int32, (self.batch,), dev)
        _same_cache(cache, self.H_kv, self.d_v, dev)
        max_pages = cache._table(page_table, self.batch)
        C.iamap_mapped_av_paged_quant(p_rows, self.ctx_stride, W, cache.codes, cache.scales,
                                      cache.num_pages, page_table, max_pages,
                                      cache.page_size, ctx_lens, self.max_ctx, self.batch,
                                      self.H_s, self.H_r, self.H_kv, self.d_v, cache.bits,
                                      self.out, self.ws, stream)
        return self.out


class QuantAttention:
    """Buffers of one decode attention over quantised keys and values (a layer that is not mapped,
    or the small model's own): run(q, k_cache, v_cache, page_table, ctx_lens) -> out bf16
    [batch, H_q, d], or (out, lse fp32 [batch, H_q]) with want_lse."""

    def __init__(self, batch, H_q, d, max_ctx, H_kv=None, want_lse=False, device="cuda"):
        self.batch, self.H_q, self.d, self.max_ctx = batch, H_q, d, int(max_ctx)
        self.H_kv = H_q if H_kv is None else int(H_kv)
        self.ws = C.alloc_workspace(
            C.iamap_attention_paged_quant_workspace_bytes(batch, H_q, d, self.max_ctx), device)
        self.out = torch.empty(batch, H_q, d, dtype=torch.bfloat16, device=device)
        self.lse = torch.empty(batch, H_q, dtype=torch.float32, device=device) if want_lse else None

    def run(self, q, k_cache, v_cache, page_table, ctx_lens, stream=None):
        dev = self.out.device
        _expect("q", q, torch.bfloat16, (self.batch, self.H_q, self.d), dev)
        _expect("ctx_lens", ctx_lens, torch.int32, (self.batch,), dev)
        _same_cache(k_cache, self.H_kv, self.d, dev)
        _same_cache(v_cache, self.H_kv, self.d, dev)
        if k_cache.num_pages != v_cache.num_pages or k_cache.page_size != v_cache.page_size:
            raise ValueError("keys and values must share their pages")
        max_pages = k_cache._table(page_table, self.batch)
        C.iamap_attention_paged_quant(q, k_cache.codes, k_cache.scales, k_cache.bits,
                                      v_cache.codes, v_cache.scales, v_cache.bits,
                                      k_cache.num_pages, page_table, max_pages,
                                      k_cache.page_size, ctx_lens, self.max_ctx, self.batch,
                                      self.H_q, self.H_kv, self.d, self.out, self.lse, self.ws,
                                      stream)
        return self.out if self.lse is None else (self.out, self.lse)


def _same_cache(cache, H, d, device):
    if cache.H != H or cache.d != d or cache.device != device:
        raise ValueError("a cache of %d heads of %d on %s expected, got %d of %d on %s" % (
            H, d, device, cache.H, cache.d, cache.device))


class HeadMatch:
    """Buffers of one head-matching calibration."""

    def __init__(self, L_s, H_small, d_small, L_l, H_large, d_large, n, n_used=None,
                 want_sim=True, device="cuda", metric="cosine"):
        self.dims = (L_s, H_small, d_small, L_l, H_large, d_large)
        self.metric = C.SIM_METRICS[metric]
        self.n = n
        self.n_used = n if n_used is None else int(n_used)
        self.ws = C.alloc_workspace(
            C.iamap_head_match_workspace_bytes(L_s, H_small, L_l, H_large, self.n_used), device)
        self.argmax = torch.empty(L_l * H_large, dtype=torch.int32, device=device)
        self.sim = (torch.empty(L_l * H_large, L_s * H_small, dtype=torch.float32, device=device)
                    if want_sim else None)

    def run(self, q_small, k_small, q_large, k_large, stream=None):
        L_s, H_small, d_small, L_l, H_large, d_large = self.dims
        C.iamap_head_match_metric(q_small, k_small, L_s, H_small, d_small, q_large, k_large,
                                  L_l, H_large, d_large, self.n, self.n_used, self.metric,
                                  self.argmax, self.sim, self.ws, stream)
        return self.argmax, self.sim


def mapping_consistency(argmax_a, argmax_b, stream=None):
    """Number of large heads (device int32 tensor of one element) that two head mappings send to
    the same small head; divide by the head count for the consistency rate."""
    agree = torch.zeros(1, dtype=torch.int32, device=argmax_a.device)
    C.iamap_mapping_consistency(argmax_a, argmax_b, argmax_a.numel(), agree, stream)
    return agree


class PrefixIndex:
    """A device prefix-hash index of stored map blocks: `capacity` slots (a power of two) of
    uint64 keys (carried as int64 tensors) and int64 locations, keys made with `salt` (one salt
    per sender layer or model)."""

    def __init__(self, capacity, B=64, salt=0xCBF29CE484222325, device="cuda"):
        self.capacity, self.B, self.salt = int(capacity), int(B), int(salt)
        self.table_keys = torch.empty(self.capacity, dtype=torch.int64, device=device)
        self.table_vals = torch.empty(self.capacity, dtype=torch.int64, device=device)
        self.device = device
        self.clear()

    def clear(self, stream=None):
        C.iamap_prefix_index_clear(self.table_keys, self.table_vals, self.capacity, stream)

    def keys(self, tokens, cu_seqlens, cu_seqlens_host, stream=None):
        """(keys int64 [num_keys], key_cu int64 [num_seqs + 1]) of packed prompts."""
        num_seqs = len(cu_seqlens_host) - 1
        nk = C.iamap_prefix_num_keys(cu_seqlens_host, num_seqs, self.B)
        keys = torch.empty(max(nk, 1), dtype=torch.int64, device=self.device)
        key_cu = torch.empty(num_seqs + 1, dtype=torch.int64, device=self.device)
        C.iamap_prefix_keys(tokens, tokens.numel(), cu_seqlens, num_seqs, self.B, self.salt, keys,
                            nk, key_cu, stream)
        return keys[:nk], key_cu

    def insert(self, keys, values, stream=None):
        """Locations now stored for `keys` (int64 [count]); -1 where no slot was found."""
        stored = torch.empty(max(keys.numel(), 1), dtype=torch.int64, device=self.device)
        C.iamap_prefix_insert(keys, values, keys.numel(), self.table_keys, self.table_vals,
                              self.capacity, stored, stream)
        return stored[:keys.numel()]

    def lookup(self, keys, key_cu=None, stream=None):
        """(found int64 [count], hit_blocks int32 [num_seqs] or None)."""
        found = torch.empty(max(keys.numel(), 1), dtype=torch.int64, device=self.device)
        hits = None
        num_seqs = 0
        if key_cu is not None:
            num_seqs = key_cu.numel() - 1
            hits = torch.empty(num_seqs, dtype=torch.int32, device=self.device)
        C.iamap_prefix_lookup(keys, keys.numel(), key_cu, num_seqs, self.table_keys,
                              self.table_vals, self.capacity, found, hits, stream)
        return found[:keys.numel()], hits


# ------------------------------------------------------------------------------------------------
# Several GPUs: head matching split by large layers, prefill split by sequence
# ------------------------------------------------------------------------------------------------

def shard_range(total, world, rank):
    """[lo, hi) of `total` items given to `rank` of `world`: contiguous blocks of
    ceil(total / world), the last ones possibly short or empty."""
    per = -(-total // world)
    lo = min(total, rank * per)
    return lo, min(total, lo + per)


def causal_blocks(L, B=64):
    """Causal (row block, column block) pairs of a sequence of L tokens: its share of the work of
    compress and mapped_av."""
    nb = -(-int(L) // B)
    return nb * (nb + 1) // 2


def shard_sequences(seqlens, world, B=64):
    """Packed sequences -> ranks for a prefill split by sequence (no collective on the path).
    Longest-processing-time-first: sequences by decreasing causal blocks (ties: lower index)
    go to the rank with the least work so far (ties: lower rank). The most loaded rank then has
    at most (4/3 - 1/(3 world)) times the optimum. Returns per-rank lists of sequence indices in
    increasing order."""
    work = [0] * world
    out = [[] for _ in range(world)]
    order = sorted(range(len(seqlens)), key=lambda s: (-causal_blocks(seqlens[s], B), s))
    for s in order:
        r = min(range(world), key=lambda x: (work[x], x))
        out[r].append(s)
        work[r] += causal_blocks(seqlens[s], B)
    return [sorted(x) for x in out]


def gather_head_mapping(local_argmax, L_l, H_large, group=None):
    """All ranks' head mappings of their large-layer shards ([hi - lo, H_large] int32 on this
    rank's device, shards from shard_range) -> the full [L_l, H_large] mapping on every rank, with
    one all_gather of int32 (the only collective of a sharded calibration)."""
    import torch.distributed as dist
    world = dist.get_world_size(group)
    per = -(-L_l // world)
    pad = torch.zeros(per, H_large, dtype=torch.int32, device=local_argmax.device)
    pad[:local_argmax.shape[0]] = local_argmax.view(-1, H_large)
    parts = [torch.empty_like(pad) for _ in range(world)]
    dist.all_gather(parts, pad, group=group)
    return torch.cat(parts, dim=0)[:L_l]


class HostPrefillPipeline:
    """Prefill steps of one PrefillLayer on host-resident (pinned) inputs through the library's
    own host-buffer entry point (iamap_prefill_steps_host): every step uploads its q, k, v, W and
    reads its output back, and the upload of the next step and the read-back of the previous one
    overlap the current step's kernels (two device sets of inputs and outputs in `io`; the
    library's upload and download streams, ordered by events against the compute stream)."""

    def __init__(self, layer, device="cuda"):
        self.layer = layer
        L = layer
        self.io = C.alloc_workspace(C.iamap_prefill_io_bytes(L.n, L.H_s, L.d, L.H_r, L.H_kv,
                                                             L.d_v), device)

    def bytes_per_step(self):
        """(host-to-device, device-to-host) bytes of one step."""
        L = self.layer
        h2d = 2 * 2 * L.n * L.H_s * L.d + 2 * L.n * L.H_kv * L.d_v + 4 * L.H_r * L.H_s
        return h2d, 4 * L.n * L.H_r * L.d_v

    def run(self, host_inputs, host_outputs, stream=None):
        """host_inputs[i] = (q, k, v, W) pinned CPU tensors of step i; host_outputs[i] the pinned
        CPU tensor receiving its output (entries may repeat: a buffer is written in step order).
        Enqueues every step (the first upload follows everything enqueued on `stream` before)
        and returns the event recorded on `stream` after the last read-back."""
        comp = torch.cuda.current_stream() if stream is None else stream
        L = self.layer
        b = L.bufs
        if host_inputs:
            qs, ks, vs, Ws = (list(x) for x in zip(*host_inputs))
            C.iamap_prefill_steps_host(qs, ks, vs, Ws, list(host_outputs), L.cu, L.cu_host,
                                       L.num_seqs, L.n, L.H_s, L.d, L.H_r, L.H_kv, L.d_v, L.B,
                                       L.tau, L.bias_window, L.bias_value, b["lse"], b["mass"],
                                       b["headmask_dense"], b["row_ptr"], b["col_idx"],
                                       b["headmask"], b["val_off"], b["counts"], L.vals,
                                       L.capacity, self.io, L.ws, comp)
        done = torch.cuda.Event(enable_timing=True)
        done.record(comp)
        return done
