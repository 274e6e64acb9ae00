"""Device-memory plumbing around the C ABI: a paged quantized KV cache whose
buffers are torch CUDA tensors.  Every computation is a libkvq call."""
from __future__ import annotations

import ctypes

import torch

from . import _binding as B


def make_config(num_q_heads, num_kv_heads, head_dim, k, v, residual, page_size, rope_pre=0,
                rope_theta=10000.0, src_dtype=B.KVQ_F32, meta_dtype=B.KVQ_F32) -> B.kvq_config:
    """k, v: (fmt, mode, axis, group) tuples; meta_dtype: stored scales / minima (F32 or F16)."""
    cfg = B.kvq_config(num_q_heads, num_kv_heads, head_dim, B.kvq_qspec(*k), B.kvq_qspec(*v), residual,
                       page_size, rope_pre, rope_theta, src_dtype, meta_dtype)
    code = B.kvq_validate(cfg)
    if code != B.KVQ_OK:
        raise B.KvqError("kvq_validate", code)
    return cfg


def make_rope(cos_sin, rot_dim, pairing=B.KVQ_ROPE_INTERLEAVED) -> B.kvq_rope:
    """The position rotation of append_rope.  cos_sin: [positions, rot_dim] float32 device tensor, the cosines of the
    rot_dim / 2 pairs, then their sines; the caller keeps it alive."""
    if cos_sin.dtype != torch.float32 or cos_sin.dim() != 2 or cos_sin.shape[1] != rot_dim or not cos_sin.is_contiguous():
        raise ValueError("cos_sin must be a contiguous float32 tensor of [positions, rot_dim]")
    rope = B.kvq_rope(cos_sin.data_ptr(), cos_sin.shape[0], rot_dim, pairing)
    rope.tensor = cos_sin  # the table outlives the struct
    return rope


def src_torch_dtype(cfg) -> torch.dtype:
    return torch.bfloat16 if cfg.src_dtype == B.KVQ_BF16 else torch.float32


class PagedKVCache:
    """Caller-owned buffers of one cache (pages, block table, lengths, window,
    static scales, status word) and the kvq_cache struct pointing at them."""

    def __init__(self, cfg, batch, max_pages_per_seq, n_pages=None, block_table=None, device="cuda",
                 rope_table=True):
        """rope_table (pre-RoPE keys only): True builds a table for every position the
        pages can hold (rounded up to a multiple of 32, as the kernel reads whole
        32-position tables), False leaves the decode kernel to compute the cos/sin,
        and a (tensor, positions) pair shares a table built by kvq_rope_table_init."""
        n_pages = n_pages if n_pages is not None else batch * max_pages_per_seq
        dev = torch.device(device)
        pages = torch.zeros(n_pages * B.kvq_page_bytes(cfg), dtype=torch.uint8, device=dev)
        if block_table is None:
            block_table = torch.arange(batch * max_pages_per_seq, dtype=torch.int32).reshape(batch, -1)
        block_table = torch.as_tensor(block_table, dtype=torch.int32).reshape(batch, max_pages_per_seq).to(dev).contiguous()
        seq_lens = torch.zeros(batch, dtype=torch.int32, device=dev)
        R, H, D = cfg.residual, cfg.num_kv_heads, cfg.head_dim
        dt = src_torch_dtype(cfg)
        k_win = torch.zeros(batch, max(R, 1), H, D, dtype=dt, device=dev) if R else None
        v_win = torch.zeros(batch, max(R, 1), H, D, dtype=dt, device=dev) if R else None
        self._bind(cfg, pages, block_table, seq_lens, k_win, v_win, rope_table)

    @classmethod
    def over(cls, cfg, pages, block_table, seq_lens, k_win=None, v_win=None, rope_table=False):
        """A cache over buffers that the caller owns: pages (n_pages * kvq_page_bytes bytes), block_table
        [batch, max_pages_per_seq] and seq_lens [batch] int32, and the residual windows [batch, R, Hkv, D] in
        the source dtype (None when R is 0).  All contiguous, on one device."""
        if not pages.is_cuda:
            raise ValueError("a cache's buffers are CUDA tensors")
        page = B.kvq_page_bytes(cfg)
        if pages.dtype != torch.uint8 or not pages.is_contiguous() or pages.numel() == 0 or pages.numel() % page:
            raise ValueError(f"pages must be contiguous uint8 of a multiple of {page} bytes")
        batch = seq_lens.numel()
        for name, t, shape, dt in (("block_table", block_table, (batch, block_table.shape[-1]), torch.int32),
                                   ("seq_lens", seq_lens, (batch,), torch.int32),
                                   ("k_win", k_win, (batch, cfg.residual, cfg.num_kv_heads, cfg.head_dim), None),
                                   ("v_win", v_win, (batch, cfg.residual, cfg.num_kv_heads, cfg.head_dim), None)):
            if t is None and dt is None and cfg.residual == 0:
                continue
            if (t is None or tuple(t.shape) != shape or t.dtype != (dt or src_torch_dtype(cfg))
                    or not t.is_contiguous() or t.device != pages.device):
                raise ValueError(f"{name} must be contiguous {dt or src_torch_dtype(cfg)} of shape {shape} beside the pages")
        self = cls.__new__(cls)
        self._bind(cfg, pages, block_table, seq_lens, k_win, v_win, rope_table)
        return self

    def _bind(self, cfg, pages, block_table, seq_lens, k_win, v_win, rope_table):
        batch, max_pages_per_seq = block_table.shape
        self.cfg = cfg
        self.batch = batch
        self.max_pages = max_pages_per_seq
        self.page_bytes = B.kvq_page_bytes(cfg)
        self.n_pages = pages.numel() // self.page_bytes
        self.pages, self.block_table, self.seq_lens, self.k_win, self.v_win = pages, block_table, seq_lens, k_win, v_win
        dev, H = pages.device, cfg.num_kv_heads
        self.k_scale = torch.zeros(H, dtype=torch.float32, device=dev)
        self.v_scale = torch.zeros(H, dtype=torch.float32, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.workspace = torch.empty(
            max(B.kvq_workspace_bytes(cfg, batch, max_pages_per_seq * cfg.page_size), 256),
            dtype=torch.uint8, device=dev)
        self._outgrown, self._query_bytes = [], {}
        self._device, self._index, self._src = pages.device, pages.get_device(), src_torch_dtype(cfg)
        self._Hq, self._H, self._D = cfg.num_q_heads, H, cfg.head_dim
        self.rope_table, self.rope_positions = None, 0
        if cfg.rope_pre and rope_table is not False:
            if rope_table is True:
                n = (max_pages_per_seq * cfg.page_size + 31) // 32 * 32  # whole 32-position tables
                self.rope_table = torch.empty(B.kvq_rope_table_bytes(cfg, n), dtype=torch.uint8, device=dev)
                self.rope_positions = n
                B.kvq_rope_table_init(cfg, n, self.rope_table)
            else:
                self.rope_table, self.rope_positions = rope_table
        p = lambda t: None if t is None else t.data_ptr()
        self.c = B.kvq_cache(p(self.pages), p(self.block_table), p(self.seq_lens), p(self.k_win), p(self.v_win),
                             p(self.k_scale), p(self.v_scale), batch, max_pages_per_seq, self.n_pages,
                             p(self.status), p(self.rope_table), self.rope_positions)

    def _empty(self, shape, dtype, stream):
        """A new tensor, of the allocator's pool of the stream that is to write it: memory of the current stream's pool
        may still be in use there."""
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=self._device)
        if not isinstance(stream, torch.cuda.Stream):
            at = int(getattr(stream, "cuda_stream", stream))
            stream = (torch.cuda.default_stream(self._device) if at < 2  # no stream, or the legacy one by name
                      else torch.cuda.ExternalStream(at, device=self._device))
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=self._device)

    # --- thin wrappers over the C ABI
    def append(self, k_new, v_new, n_new_per_seq=None, stream=None):
        """k_new, v_new: [batch, n_new, Hkv, D], dense."""
        n = k_new.shape[1]
        for name, t in (("k_new", k_new), ("v_new", v_new)):
            if self._rows(name, t, n, self._H) != self._H * self._D and n:
                raise ValueError(f"{name} must be contiguous")
        if n_new_per_seq is not None:
            self._counts("n_new_per_seq", n_new_per_seq)
        B.kvq_quantize_append(self.cfg, self.c, k_new, v_new, n, n_new_per_seq, stream)

    def attention(self, q, out=None, softmax_scale=0.0, stream=None):
        if q.numel() != self.batch * self._Hq * self._D or q.dtype != self._src or not q.is_contiguous():
            raise ValueError(f"q must be contiguous {self._src} of shape {(self.batch, self._Hq, self._D)}")
        self._beside("q", q)
        if out is None:
            out = self._empty(q.shape, torch.float32, stream)
        elif out.numel() != q.numel() or out.dtype != torch.float32 or not out.is_contiguous():
            raise ValueError("out must be contiguous float32 of q's shape")
        else:
            self._beside("out", out)
        B.kvq_decode_attention(self.cfg, self.c, q, out, softmax_scale, self.workspace, stream)
        return out

    def _beside(self, name, t):
        """The library launches on the current device, over the cache's memory."""
        if t.get_device() != self._index or torch._C._cuda_getDevice() != self._index:
            raise ValueError(f"{name} must be on the cache's device ({self._device}), which must be the current one")

    def _counts(self, name, t):
        self._beside(name, t)
        if t.shape != (self.batch,) or t.dtype != torch.int32 or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous int32 of shape {(self.batch,)}")

    def _rows(self, name, t, n, heads):
        """Elements between consecutive tokens of t [batch, n, heads, D]: a token's row contiguous, tokens evenly spaced."""
        D = self._D
        if t.shape != (self.batch, n, heads, D) or t.dtype != self._src:
            raise ValueError(f"{name} must be {self._src} of shape {(self.batch, n, heads, D)}")
        sb, sn, sh, sd = t.stride()
        row = sn if n > 1 else sb if self.batch > 1 else heads * D
        # a row below heads * D: a broadcast view, whose storage holds fewer rows than the kernels would read
        if sd != 1 or (heads > 1 and sh != D) or (self.batch > 1 and n > 1 and sb != n * row) or (n and row < heads * D):
            raise ValueError(f"{name}: a token's row must be contiguous and the tokens evenly spaced")
        self._beside(name, t)
        return row

    def append_rope(self, rope, q, k_new, v_new, n_new_per_seq=None, q_out=None, stream=None):
        """append() with the position rotation on the way: k_new, v_new [batch, n_new, Hkv, D] and q
        [batch, n_new, Hq, D] (or None) may be slices of one fused projection (rows of one token contiguous,
        tokens evenly spaced).  Returns the rotated queries."""
        n = k_new.shape[1]
        if getattr(rope, "tensor", None) is not None:  # make_rope's
            self._beside("cos_sin", rope.tensor)
        if n_new_per_seq is not None:
            self._counts("n_new_per_seq", n_new_per_seq)
        qs = 0
        if q is not None:
            qs = self._rows("q", q, n, self._Hq)
            if q_out is None:
                q_out = self._empty(q.shape, q.dtype, stream)
            elif q_out.shape != q.shape or q_out.dtype != q.dtype or not q_out.is_contiguous():
                raise ValueError("q_out must be contiguous, of q's shape and dtype")
            else:
                self._beside("q_out", q_out)
        ks, vs = self._rows("k_new", k_new, n, self._H), self._rows("v_new", v_new, n, self._H)
        if stream is None:
            stream = torch._C._cuda_getCurrentRawStream(self._index)
        B.kvq_rope_append(self.cfg, self.c, rope, q, k_new, v_new, n, n_new_per_seq, q_out, qs, ks, vs, stream)
        return q_out

    def query_attention(self, q, causal=True, n_q_per_seq=None, out=None, softmax_scale=0.0, stream=None):
        """Attention of n_q queries per sequence, q [batch, n_q, Hq, D]: the sequence's newest n_q tokens over its
        own cache (causal), or a decoder's tokens over an encoder's states (causal=False).  The workspace grows
        with n_q on first use and is kept; calls on several streams at once need a cache object each, and an object
        outlives the calls on other streams than its own."""
        cfg, n = self.cfg, q.shape[1]
        if q.shape != (self.batch, n, self._Hq, self._D) or q.dtype != self._src or not q.is_contiguous():
            raise ValueError(f"q must be contiguous {self._src} of shape {(self.batch, n, cfg.num_q_heads, cfg.head_dim)}")
        self._beside("q", q)
        if out is None:
            out = self._empty(q.shape, q.dtype, stream)
        elif out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous():
            raise ValueError("out must be contiguous, of q's shape and dtype")
        else:
            self._beside("out", out)
        if n_q_per_seq is not None:
            self._counts("n_q_per_seq", n_q_per_seq)
        need = self._query_bytes.get(n)
        if need is None:
            need = self._query_bytes[n] = B.kvq_query_workspace_bytes(cfg, self.batch, max(n, 1))
        if self.workspace.numel() < need:
            self._outgrown.append(self.workspace)  # a captured graph may still use it
            # at least doubled, so that all of them together stay below the one in use
            self.workspace = self._empty(max(need, 2 * self.workspace.numel()), torch.uint8, stream)
        if stream is None:
            stream = torch._C._cuda_getCurrentRawStream(self._index)
        B.kvq_query_attention(cfg, self.c, q, n, n_q_per_seq, B.KVQ_MASK_CAUSAL if causal else B.KVQ_MASK_NONE, out,
                              softmax_scale, self.workspace, stream)
        return out

    def decode_kernel(self) -> int:
        """The decode kernel (KVQ_KERNEL_*) attention() launches for this cache."""
        return B.kvq_decode_kernel(self.cfg, self.c)

    def dequantize(self, seq, tok_begin, tok_end, stream=None):
        self._beside("the cache", self.pages)
        n = tok_end - tok_begin
        k, v = (self._empty((n, self.cfg.num_kv_heads, self.cfg.head_dim), torch.float32, stream) for _ in range(2))
        B.kvq_dequantize(self.cfg, self.c, seq, tok_begin, tok_end, k, v, stream)
        return k, v

    def calibrate(self, k_src, v_src, k_qmax, v_qmax, stream=None):
        """Set the static per-head scales from [N, Hkv, D] source tensors."""
        for name, t in (("k_src", k_src), ("v_src", v_src)):
            self._beside(name, t)
        B.kvq_calibrate_absmax(self.cfg, k_src, k_src.shape[0], k_qmax, self.k_scale, stream)
        B.kvq_calibrate_absmax(self.cfg, v_src, v_src.shape[0], v_qmax, self.v_scale, stream)

    def page_view(self):
        return self.pages.view(self.n_pages, self.page_bytes)
