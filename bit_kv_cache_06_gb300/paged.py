"""Paged, ragged KIVI cache (include/kivi.h, "paged cache"): a pool of key-group
records, a table of page numbers per (sequence, kv head), and the four
operations that fill it, attend to it, weigh its pages and evict them.

Argument checks and marshalling only; the work is in the CUDA kernels behind
the C ABI.  Nothing here waits for the GPU, and every call may be captured into
a CUDA graph: the sequences' lengths live on the device.
"""
import ctypes

import torch

from . import kivi
from .kivi import _check


class KiviPagedCache:
    """One layer's paged cache for `shape.batch` sequences of lengths of their
    own, each with up to `shape.capacity_tokens` quantised tokens held.

    buffers: (pool, k_fp16, v_fp16, table, n_tokens, n_evicted) to bind instead
    of allocating them: pool uint8 [num_pages, record bytes], k_fp16 / v_fp16
    fp16 [P, sink + R, d], table int32 [P, C], n_tokens and n_evicted int32
    [B], all contiguous on one device.  Allocated tables hold the pages in
    order (row p: p C .. p C + C - 1), which needs num_pages = P C or more.

    max_new, max_cached: the longest chunk one sequence will bring in a call of
    attention or weights, and the most cached tokens it will then hold (0: as
    many as the table does).  They size the workspace (which layers may share:
    workspace=, for calls that are ordered on the GPU); longer ones are refused."""

    def __init__(self, shape, num_pages=None, max_new=1, max_cached=0, device="cuda", buffers=None,
                 workspace=None):
        L = kivi.load()
        self.shape = shape
        self.params = shape.params()
        _check(L.kivi_params_validate(ctypes.byref(self.params)), "kivi_params_validate")
        self.columns = L.kivi_paged_columns(ctypes.byref(self.params))
        if self.columns == 0:
            raise kivi.KiviError(kivi.KIVI_ERR_UNSUPPORTED, "kivi_paged_columns")
        B, P = shape.batch, shape.batch * shape.num_kv_heads
        rec = kivi.history_record_bytes(self.params)
        num_pages = P * self.columns if num_pages is None else int(num_pages)
        want = (("pool", (num_pages, rec), torch.uint8),
                ("k_fp16", (P, shape.sink_tokens + shape.residual, shape.head_dim), torch.float16),
                ("v_fp16", (P, shape.sink_tokens + shape.residual, shape.head_dim), torch.float16),
                ("table", (P, self.columns), torch.int32),
                ("n_tokens", (B,), torch.int32), ("n_evicted", (B,), torch.int32))
        if buffers is None:
            if num_pages < P * self.columns:
                raise ValueError(f"{num_pages} pages for {P} rows of {self.columns} columns: "
                                 "hand in a table (buffers=) that says which pages a row uses")
            buffers = [torch.empty(s, dtype=t, device=device) for _, s, t in want[:3]]
            buffers.append(torch.arange(P * self.columns, dtype=torch.int32,
                                        device=device).view(P, self.columns))
            buffers += [torch.zeros(B, dtype=torch.int32, device=device) for _ in range(2)]
        self.device = buffers[0].device
        for t, (name, size, dtype) in zip(buffers, want):
            if tuple(t.shape) != size or t.dtype != dtype or not t.is_contiguous() or \
                    t.device != self.device:
                raise ValueError(f"{name}: {dtype} {list(size)}, contiguous, on {self.device} is wanted; "
                                 f"got {t.dtype} {list(t.shape)} on {t.device}")
        self.pool, self.k_fp16, self.v_fp16, self.table, self.n_tokens, self.n_evicted = buffers
        self.max_new, self.max_cached = int(max_new), int(max_cached)
        need = L.kivi_paged_workspace_bytes(ctypes.byref(self.params), self.max_new, self.max_cached)
        if need == 0:
            raise kivi.KiviError(kivi.KIVI_ERR_UNSUPPORTED, "kivi_paged_workspace_bytes")
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
        if workspace.numel() * workspace.element_size() < need:
            raise kivi.KiviError(kivi.KIVI_ERR_WORKSPACE, f"workspace of {need} bytes")
        if workspace.device != self.device or not workspace.is_contiguous():
            raise ValueError(f"workspace: contiguous on {self.device} is wanted")
        self.workspace = workspace
        self._ws, self._ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        self.control = torch.zeros(L.kivi_paged_control_bytes(ctypes.byref(self.params)) // 4,
                                   dtype=torch.int32, device=self.device)
        self.c = kivi.kivi_paged()
        _check(L.kivi_paged_init(ctypes.byref(self.c), ctypes.byref(self.params),
                                 self.pool.data_ptr(), num_pages, self.k_fp16.data_ptr(),
                                 self.v_fp16.data_ptr(), self.table.data_ptr(),
                                 self.n_tokens.data_ptr(), self.n_evicted.data_ptr(),
                                 self.control.data_ptr()), "kivi_paged_init")
        self._c, self._lib, self._index = ctypes.byref(self.c), L, self.device.index

    @classmethod
    def from_cache(cls, cache, max_new=1, max_cached=0, workspace=None):
        """A paged view of a KiviCache as it is now: its history buffer is the
        pool, row p names records p C .. p C + C - 1, every sequence has the
        cache's length.  The two share buffers, not state: tokens appended to
        one are not counted by the other."""
        s = cache.shape
        P = s.batch * s.num_kv_heads
        C = s.capacity_tokens // s.group
        pool = cache.view("history").view(P * C, -1)
        table = torch.arange(P * C, dtype=torch.int32, device=cache.device).view(P, C)
        n = cache.n_sink + cache.n_quant + cache.n_resid
        tokens = torch.full((s.batch,), n, dtype=torch.int32, device=cache.device)
        return cls(s, P * C, max_new, max_cached, buffers=(pool, cache.view("k_fp16"), cache.view("v_fp16"), table,
                                               tokens, torch.zeros_like(tokens)), workspace=workspace)

    # ---- state ------------------------------------------------------------
    def reset(self):
        """Forget all tokens (the table keeps its pages)."""
        self.n_tokens.zero_()
        self.n_evicted.zero_()

    def status(self) -> int:
        """Error bits the kernels set (0 = none); waits for the GPU."""
        return int(self.control[0].item())

    @property
    def kernel_launches(self) -> int:
        return self.c.kernel_launches

    # ---- calls ------------------------------------------------------------
    def _on(self, stream, tensors):
        """The stream a call goes to, as the C ABI takes it; tensors that a
        stream other than the current one uses, the cache's own among them, are
        kept from being handed out again before it is done with them."""
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(self._index)
        if stream == torch.cuda.current_stream(self.device):
            return stream.cuda_stream
        if not torch.cuda.is_current_stream_capturing():
            own = (self.pool, self.k_fp16, self.v_fp16, self.table, self.n_tokens, self.n_evicted, self.control,
                   self.workspace)
            for t in tensors + own:
                if t is not None:
                    t.record_stream(stream)
        return stream.cuda_stream

    def _call(self, name, *args):
        """A launch, with this cache's device current."""
        fn = getattr(self._lib, name)
        if torch._C._cuda_getDevice() == self._index:
            st = fn(self._c, *args)
        else:
            with torch.cuda.device(self.device):
                st = fn(self._c, *args)
        if st:
            _check(st, name)

    def _heads(self, name, x, heads, tokens):
        """Stride from token to token of x, fp16 [tokens, heads, d]."""
        shape, d = x.shape, self.shape.head_dim
        if len(shape) != 3 or shape[1] != heads or shape[2] != d or x.dtype is not torch.float16 or \
                x.device != self.device or (tokens is not None and shape[0] != tokens):
            raise ValueError(f"{name}: fp16 [{'tokens' if tokens is None else tokens}, {heads}, {d}] on "
                             f"{self.device} is wanted; got {x.dtype} {list(shape)} on {x.device}")
        stride = x.stride()
        if shape[0] > 0 and (stride[2] != 1 or (heads > 1 and stride[1] != d)):
            raise ValueError(f"{name}: one token's heads have to lie side by side (strides {stride})")
        return stride[0] if shape[0] > 1 else heads * d

    def _chunk(self, q, k, v, offsets, max_new, max_cached, softmax_scale, softcap, causal):
        s = self.shape
        if offsets is None or offsets.dtype != torch.int32 or offsets.numel() != s.batch + 1 or \
                not offsets.is_contiguous() or offsets.device != self.device:
            raise ValueError(f"offsets: contiguous int32 [{s.batch + 1}] on {self.device} is wanted")
        n, q_ptr, k_ptr, v_ptr, q_stride, kv_stride = None, None, None, None, 0, 0
        if q is not None:
            q_ptr, q_stride = q.data_ptr(), self._heads("q", q, s.num_q_heads, None)
            n = q.shape[0]
        if k is not None:
            k_ptr, kv_stride = k.data_ptr(), self._heads("k", k, s.num_kv_heads, n)
            n = k.shape[0]
        if v is not None:
            if k is None:
                raise ValueError("v without k")
            v_ptr = v.data_ptr()
            if self._heads("v", v, s.num_kv_heads, n) != kv_stride:
                raise ValueError("k and v have to have the same stride from token to token")
        return ctypes.byref(kivi.kivi_chunk(
            q_ptr, k_ptr, v_ptr, offsets.data_ptr(), q_stride, kv_stride, n,
            n if max_new is None else max_new, self.max_cached if max_cached is None else max_cached,
            softmax_scale, softcap, kivi.KIVI_MASK_CAUSAL if causal else kivi.KIVI_MASK_FULL, 0))

    def _pages(self, weights):
        want = (self.shape.batch * self.shape.num_kv_heads, self.columns)
        if weights.dtype != torch.float32 or tuple(weights.shape) != want or \
                not weights.is_contiguous() or weights.device != self.device:
            raise ValueError(f"weights: contiguous fp32 {list(want)} on {self.device} is wanted")
        return weights.data_ptr()

    def append(self, k, v, offsets, max_new=None, stream=None):
        """New tokens k, v fp16 [N, Hkv, d] of a ragged batch enter the cache:
        sequence b's are rows offsets[b] .. offsets[b + 1] - 1 (offsets int32
        [B + 1] on the device).  max_new bounds one sequence's count (default
        N).  n_tokens grows on the device."""
        x = self._chunk(None, k, v, offsets, max_new, 0, 0.0, 0.0, True)
        self._call("kivi_paged_append", x, self._on(stream, (k, v, offsets)))

    def attention(self, q, k=None, v=None, offsets=None, max_new=None, max_cached=None, softmax_scale=0.0,
                  softcap=0.0, causal=True, out=None, stream=None):
        """Attention of new tokens q fp16 [N, Hq, d] over their sequence's
        cached tokens and over k, v fp16 [N, Hkv, d] of the new tokens
        themselves (causally, or all of them with causal=False; without k, v
        over the cached tokens alone).  Appends nothing.  max_new bounds the new
        tokens of one sequence (default N: a batch of decode steps says 1), max_cached
        the cached tokens of any sequence (default: the cache's); the nearer
        it is, the better the work is split.  Returns out, fp16
        [N, Hq, d]; rows outside every sequence stay as they are."""
        x = self._chunk(q, k, v, offsets, max_new, max_cached, softmax_scale, softcap, causal)
        if out is None:
            if stream is None:
                out = q.new_empty(q.shape)
            else:
                with torch.cuda.stream(stream):
                    out = q.new_empty(q.shape)
        elif out.dtype != torch.float16 or out.shape != q.shape or not out.is_contiguous() or \
                out.device != self.device:
            raise ValueError(f"out: contiguous fp16 {list(q.shape)} on {self.device} is wanted")
        self._call("kivi_paged_attention", x, out.data_ptr(), self._ws, self._ws_bytes,
                   self._on(stream, (q, k, v, offsets, out)))
        return out

    def weights(self, weights, q, k=None, offsets=None, max_new=None, max_cached=None, softmax_scale=0.0,
                softcap=0.0, causal=True, stream=None):
        """Add to weights, fp32 [P, C], what each page gets of the softmax
        weights of `attention`'s queries."""
        x = self._chunk(q, k, None, offsets, max_new, max_cached, softmax_scale, softcap, causal)
        self._call("kivi_paged_weights", x, self._pages(weights), self._ws, self._ws_bytes,
                   self._on(stream, (q, k, offsets, weights)))
        return weights

    def evict(self, weights, budget, recent=0, stream=None):
        """Every pair that holds more than `budget` pages keeps the `recent`
        newest ones and the heaviest others; table, weights and n_evicted
        follow (include/kivi.h, kivi_paged_evict)."""
        self._call("kivi_paged_evict", self._pages(weights), budget, recent, self._ws, self._ws_bytes,
                   self._on(stream, (weights,)))
