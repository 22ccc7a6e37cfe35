"""A torch-tensor front end of the pre-attention C-ABI.

PyTorch provides device memory and streams only; every step of the
computation runs in libpre_attn.so.  ``PreAttn`` owns a handle and a
workspace and turns tensors into the C structs of include/pre_attn.h.
"""

from __future__ import annotations

import sys

import torch

from . import binding as B


class PreAttn:
    """One configured pre-attention step (one layer's shapes and formats)."""

    def __init__(self, hidden: int, n_kv_heads: int, *, weight_format: int, cache_format: int,
                 max_tokens: int, block_size: int = 16, eps: float = 1e-6, n_q_heads: int = 0,
                 n_iq_heads: int = 0, kv_page_stride: int = 8, flags: int = 0, gemm_grid: int = 0,
                 device: torch.device | str | None = None):
        B.load()
        self.cfg = B.pa_config(hidden, n_kv_heads, n_q_heads, n_iq_heads, weight_format, cache_format,
                               block_size, kv_page_stride, eps, max_tokens, flags, gemm_grid)
        self.handle = B.pre_attn_init(self.cfg)
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.N = B.pre_attn_out_features(self.handle)
        self.ws_bytes = B.pre_attn_workspace_bytes(self.handle, max_tokens)
        self.workspace = torch.empty(max(self.ws_bytes, 256), dtype=torch.uint8, device=self.device)
        B.pre_attn_workspace_init(self.workspace, self.ws_bytes, torch.cuda.current_stream(self.device))

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None:
            B.pre_attn_destroy(h)
            self.handle = None

    @staticmethod
    def weights(w, w_scale, g_in, g_q, g_k, g_iq, g_ik, cos_sin) -> B.pa_weights:
        return B.pa_weights(B.ptr(w), B.ptr(w_scale), B.ptr(g_in), B.ptr(g_q), B.ptr(g_k), B.ptr(g_iq),
                            B.ptr(g_ik), B.ptr(cos_sin), int(cos_sin.shape[0]))

    @staticmethod
    def fp8_caches(k_cache, v_cache, k_scale, v_scale, index_cache, num_pages16: int,
                   num_index_slots: int) -> B.pa_caches:
        c = B.pa_caches()
        c.k_cache, c.v_cache = B.ptr(k_cache), B.ptr(v_cache)
        c.k_scale, c.v_scale = B.ptr(k_scale), B.ptr(v_scale)
        c.index_cache = B.ptr(index_cache)
        c.num_pages16, c.num_index_slots = num_pages16, num_index_slots
        c.k_global_scale = c.v_global_scale = 1.0
        return c

    @staticmethod
    def nvfp4_caches(kv_cache, kv_pages: int, kv_page_bytes: int, idx_cache, idx_pages: int,
                     idx_page_bytes: int, k_global_scale: float = 1.0, v_global_scale: float = 1.0) -> B.pa_caches:
        c = B.pa_caches()
        c.kv_cache, c.kv_pages, c.kv_page_bytes = B.ptr(kv_cache), kv_pages, kv_page_bytes
        c.idx_cache, c.idx_pages, c.idx_page_bytes = B.ptr(idx_cache), idx_pages, idx_page_bytes
        c.k_global_scale, c.v_global_scale = k_global_scale, v_global_scale
        return c

    @staticmethod
    def outputs(residual=None, q=None, q_fp8=None, iq=None, iq_fp8=None, q_fp8_scale: float = 1.0, done=None,
                done_epoch: int = 0) -> B.pa_outputs:
        return B.pa_outputs(B.ptr(residual), B.ptr(q), B.ptr(q_fp8), B.ptr(iq), B.ptr(iq_fp8), q_fp8_scale,
                            B.ptr(done), done_epoch)

    def run(self, M: int, ar, res, positions, slot_mapping, weights: B.pa_weights, caches: B.pa_caches,
            outputs: B.pa_outputs, index_slot_mapping=None, stream=None, check: bool = True) -> int:
        inputs = B.pa_step_inputs(B.ptr(ar), B.ptr(res), B.ptr(positions), B.ptr(slot_mapping),
                                  B.ptr(index_slot_mapping))
        if stream is None:
            stream = torch.cuda.current_stream(self.device)
        return B.pre_attn_run(self.handle, M, inputs, weights, caches, outputs, self.workspace,
                              self.ws_bytes, stream, check=check)

    def device_status(self, stream=None) -> int:
        if stream is None:
            stream = torch.cuda.current_stream(self.device)
        return B.pre_attn_device_status(self.workspace, stream)


class CacheReader:
    """What a layer reads back of its caches: the indexer scores, the block
    selection and the attention, for up to ``max_requests`` requests of
    ``q_len`` rows whose block tables hold ``bt_width`` page-128 blocks.

    ``caches`` is PreAttn.fp8_caches(...) or PreAttn.nvfp4_caches(...), read at
    every call (and may be replaced by another of the same format): the fields
    that a call reads have to be set (the index cache for ``index_scores``, the
    K / V ones for ``attend``) and their tensors kept alive by the caller.  Owns a workspace, a status word and the calls'
    argument structs: one host thread uses a reader at a time, and its calls,
    replays of captured ones among them, are ordered on the GPU by their
    stream, or by the caller (calls that may run together take a reader each).
    Every tensor is on ``device``; seq_lens, block tables, block lists and
    counts are contiguous int32, scores and query rows have contiguous columns.
    A call without requests does nothing.  Making a reader waits for the
    current stream (its status word is cleared there, for calls on any stream),
    so it is made outside a capture.  A reader may be dropped while its calls
    run (its workspace is not reused before them), but has to outlive the
    graphs that hold captured ones.
    """

    def __init__(self, n_q_heads: int, n_kv_heads: int, *, cache_format: int, caches: B.pa_caches, max_requests: int,
                 q_len: int, bt_width: int, topk: int = 0, init_blocks: int = 0, local_blocks: int = 0,
                 block_size: int = 16, kv_page_stride: int = 0, sm_scale: float = 128 ** -0.5, flags: int = 0,
                 device: torch.device | str | None = None):
        self.device = torch.device("cuda" if device is None else device)
        if self.device.type != "cuda":
            raise ValueError(f"a CUDA device is wanted, not {self.device}")
        lib = B.load()
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.index = self.device.index
        self.n_q_heads, self.n_kv_heads, self.cache_format = n_q_heads, n_kv_heads, cache_format
        self.max_requests, self.q_len, self.bt_width, self.topk = max_requests, q_len, bt_width, topk
        self.init_blocks, self.local_blocks, self.block_size = init_blocks, local_blocks, block_size
        self.index_scale = B.pre_attn_index_scale_log2e(sm_scale)
        sms = torch.cuda.get_device_properties(self.device).multi_processor_count
        self.ws_bytes = B.pre_attn_attention_workspace_bytes(max_requests, q_len, n_kv_heads, sms)
        if self.ws_bytes == 0:
            raise ValueError(f"max_requests {max_requests}, q_len {q_len} or n_kv_heads {n_kv_heads} out of range")
        # the first 256 bytes hold the status word
        with torch.cuda.device(self.device):
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError("a CacheReader is made outside a capture")
            self.workspace = torch.empty(256 + self.ws_bytes, dtype=torch.uint8, device=self.device)
            made_on = torch.cuda.current_stream()
            B.pre_attn_workspace_init(self.workspace, 256, made_on)
            made_on.synchronize()
        self.status = self.workspace.data_ptr()
        self._made_on = made_on.cuda_stream
        self._used_on = set()  # streams of its calls
        # the calls' argument structs, of which a call sets what changes
        self._attn = B.pa_attention_args(None, None, 1.0, 0, n_q_heads, n_kv_heads, cache_format, block_size,
                                         kv_page_stride, None, None, None, None, None, topk, 0, q_len,
                                         bt_width, sm_scale, None, 0, self.status + 256, self.ws_bytes, self.status,
                                         flags)
        self.caches = caches
        self._select = B.pa_select_args(None, 0, 0, 0, None, 0, q_len, bt_width, init_blocks, local_blocks, topk, None,
                                        None, self.status, None, 0)
        if cache_format == B.PA_CACHE_FP8:
            self._scores = B.pa_index_args(None, 0, 0, caches.index_cache, caches.num_index_slots, None, None, 0, q_len,
                                           bt_width, init_blocks, local_blocks, 0.0, None, 0, self.status, 0)
            name = "pre_attn_index_scores"
        else:
            self._scores = B.pa_index_nvfp4_args(None, 0, 0, caches.idx_cache, caches.idx_pages, caches.idx_page_bytes,
                                                 block_size, None, None, 0, q_len, bt_width, init_blocks, local_blocks, 0.0,
                                                 None, 0, self.status)
            name = "pre_attn_index_scores_nvfp4"
        self._scores_entry = getattr(lib, name), B.ctypes.byref(self._scores), name
        self._select_entry = lib.pre_attn_select_blocks, B.ctypes.byref(self._select), "pre_attn_select_blocks"
        self._attn_entry = lib.pre_attn_attention, B.ctypes.byref(self._attn), "pre_attn_attention"

    @property
    def caches(self) -> B.pa_caches:
        return self._caches

    @caches.setter
    def caches(self, caches: B.pa_caches):
        self._caches, self._attn.caches = caches, B.ctypes.pointer(caches)

    def _on(self, stream):
        """The stream of a call: the reader's device has to be the current one, and the stream's."""
        if torch._C._cuda_getDevice() != self.index:
            raise ValueError(f"the current device is not the reader's ({self.device})")
        if stream is None:
            s = torch._C._cuda_getCurrentRawStream(self.index)
        else:
            if getattr(stream, "device_index", self.index) != self.index:
                raise ValueError(f"the stream is of another device than the reader's ({self.device})")
            s = B.stream_ptr(stream)
        self._used_on.add(s)
        return s

    def __del__(self):
        # the allocator hands the workspace out again behind the work that is on these streams now
        if sys is None or sys.is_finalizing():
            return
        for s in getattr(self, "_used_on", ()):
            if s != self._made_on:
                self.workspace.record_stream(torch.cuda.ExternalStream(s, device=self.device) if s else
                                             torch.cuda.default_stream(self.device))

    def _call(self, entry, stream, check):
        """Run a C entry point (its function, the reference to its argument struct, its name)."""
        fn, args, name = entry
        st = fn(args, self._on(stream))
        if check and st != B.PA_OK:
            raise B.PreAttnError(st, name + " " + (B.pre_attn_last_cuda_error() if st == B.PA_ERR_CUDA else ""))
        return st

    def _requests(self, seq_lens, block_table=None) -> int:
        R = seq_lens.shape[0]
        if R > self.max_requests:
            raise ValueError(f"{R} requests: the reader holds {self.max_requests}")
        self._ints(seq_lens, (R,), "seq_lens")
        if block_table is not None:
            self._ints(block_table, (R, self.bt_width), "block_table")
        return R

    def _ints(self, x, shape, name):
        if x.dtype is not torch.int32 or x.shape != shape or not x.is_contiguous() or x.get_device() != self.index:
            raise ValueError(f"{name}: a contiguous int32 tensor of shape {shape} on {self.device} is wanted")

    def _rows(self, x, dtype_ok, rows, cols, name):
        shape, stride = x.shape, x.stride()
        if (not dtype_ok or len(shape) != 2 or shape[0] != rows or shape[1] < cols or stride[1] != 1
                or x.get_device() != self.index):
            raise ValueError(f"{name}: [{rows}, >= {cols}] with contiguous columns on {self.device} is wanted, not "
                             f"{x.dtype} {tuple(shape)} on {x.device}")
        return stride[0] if rows > 1 else cols  # elements a row (a single row's stride says nothing)

    def index_scores(self, iq, head: int, block_table, seq_lens, scores, *, scale: float | None = None, stream=None,
                     check: bool = True) -> int:
        """Scores of index_q head ``head`` (iq [M, >= (head + 1) * 128] bf16) into scores [M, >= bt_width * 128] f32."""
        R = self._requests(seq_lens, block_table)
        M, a = R * self.q_len, self._scores
        a.iq_stride = self._rows(iq, iq.dtype is torch.bfloat16, M, (head + 1) * 128, "iq")
        a.score_stride = self._rows(scores, scores.dtype is torch.float32, M, self.bt_width * 128, "scores")
        a.iq, a.head, a.block_table, a.seq_lens = iq.data_ptr(), head, block_table.data_ptr(), seq_lens.data_ptr()
        a.R, a.scores = R, scores.data_ptr()
        a.index_scale = self.index_scale if scale is None else scale
        c = self._caches
        if self.cache_format == B.PA_CACHE_FP8:
            a.index_cache, a.num_index_slots = c.index_cache, c.num_index_slots
        else:
            a.idx_cache, a.idx_pages, a.idx_page_bytes = c.idx_cache, c.idx_pages, c.idx_page_bytes
        if R == 0:
            return B.PA_OK
        return self._call(self._scores_entry, stream, check)

    def select_blocks(self, scores, seq_lens, blocks, counts, *, block_table=None, stream=None, check: bool = True) -> int:
        """The blocks of each row and head from scores [heads, M, >= bt_width * 128] into blocks [M, heads, topk]; with
        the block table, none whose id lies outside the index cache (whose columns index_scores leaves as they were)."""
        R = self._requests(seq_lens, block_table)
        M, shape, stride, a = R * self.q_len, scores.shape, scores.stride(), self._select
        width = self.bt_width * 128
        if (scores.dtype is not torch.float32 or len(shape) != 3 or shape[0] < 1 or shape[1] != M or shape[2] < width
                or stride[2] != 1 or scores.get_device() != self.index):
            raise ValueError(f"scores: f32 [heads, {M}, >= {width}] with contiguous columns on {self.device} is wanted")
        heads = shape[0]
        self._ints(blocks, (M, heads, self.topk), "blocks")
        self._ints(counts, (M, heads), "counts")
        a.score_stride = stride[1] if M > 1 else width
        a.score_head_stride = stride[0] if heads > 1 else M * a.score_stride
        a.scores, a.n_heads, a.seq_lens, a.R = scores.data_ptr(), heads, seq_lens.data_ptr(), R
        a.blocks, a.counts = blocks.data_ptr(), counts.data_ptr()
        a.block_table = None
        if block_table is not None:
            c = self._caches
            slots = c.num_index_slots if self.cache_format == B.PA_CACHE_FP8 else c.idx_pages * self.block_size
            a.block_table, a.num_blocks = block_table.data_ptr(), slots // 128
        if R == 0:
            return B.PA_OK
        return self._call(self._select_entry, stream, check)

    def attend(self, q, block_table, seq_lens, out, *, blocks=None, counts=None, q_fp8_scale: float = 1.0, stream=None,
               check: bool = True) -> int:
        """Attention of q [M, >= n_q_heads * 128] (bf16, or E4M3 with q_fp8_scale) into out (bf16, as wide): over the
        blocks of each row and KV head (blocks [M, n_kv_heads, topk], counts [M, n_kv_heads]), or all without."""
        R = self._requests(seq_lens, block_table)
        M, a, cols = R * self.q_len, self._attn, self.n_q_heads * 128
        half = q.dtype is torch.bfloat16
        a.q_stride = self._rows(q, half or q.dtype is torch.float8_e4m3fn, M, cols, "q")
        a.out_stride = self._rows(out, out.dtype is torch.bfloat16, M, cols, "out")
        if half:
            a.q, a.q_fp8 = q.data_ptr(), None
        else:
            a.q, a.q_fp8, a.q_fp8_scale = None, q.data_ptr(), q_fp8_scale
        a.out, a.R, a.block_table, a.seq_lens = out.data_ptr(), R, block_table.data_ptr(), seq_lens.data_ptr()
        if blocks is None:
            if counts is not None:
                raise ValueError("counts come with their blocks")
            a.blocks = a.counts = None
        else:
            if counts is None or self.topk < 1:
                raise ValueError("blocks come with their counts, and a reader of lists has topk > 0")
            self._ints(blocks, (M, self.n_kv_heads, self.topk), "blocks")
            self._ints(counts, (M, self.n_kv_heads), "counts")
            a.blocks, a.counts = blocks.data_ptr(), counts.data_ptr()
        if R == 0:
            return B.PA_OK
        return self._call(self._attn_entry, stream, check)

    def device_status(self, stream=None) -> int:
        """PA_DEV_* bits of the calls since the last reading (read and cleared; synchronises)."""
        return B.pre_attn_device_status(self.workspace, self._on(stream))
