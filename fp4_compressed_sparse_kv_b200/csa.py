"""Thin Python binding of libcsa.so (include/csa.h): argument marshalling only.

Every step of the path runs in the library's CUDA kernels.  PyTorch provides device memory and
streams; tensors must live on the current CUDA device.  There is no CPU fallback: if the shared
library is missing or a tensor is not on the GPU, these functions raise.
"""
import ctypes
import math
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcsa.so")

PAGE = 64
BLOCK = 8
LATENT = 512
WINDOW = 128
IDX_HEADS = 8
IDX_DIM = 128
HEADER_BYTES = 256
MAX_TOPK = 8192
MAX_SHARDS = 64
FULL, REINDEX, REUSE = 0, 1, 2

STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported configuration", 3: "workspace too small",
          4: "CUDA error", 5: "device metadata out of range", 6: "device wait timed out"}


class CsaError(RuntimeError):
    def __init__(self, status, where):
        super().__init__("%s: %s (status %d)" % (where, STATUS.get(status, "unknown"), status))
        self.status = status


class KVLayerC(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("keys", ctypes.c_void_p),
                ("swa", ctypes.c_void_p), ("swa_scale", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("num_rows", ctypes.c_int32)]


class BatchC(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("seq_len", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("max_pages", ctypes.c_int32), ("swa_row", ctypes.c_void_p),
                ("max_seq_len", ctypes.c_int32)]


class LayerStepC(ctypes.Structure):
    _fields_ = [("mode", ctypes.c_int), ("iq", ctypes.c_void_p), ("iw", ctypes.c_void_p),
                ("k", ctypes.c_int32), ("prev_blocks", ctypes.c_void_p),
                ("prev_count", ctypes.c_void_p), ("prev_cap", ctypes.c_int32),
                ("blocks", ctypes.c_void_p), ("count", ctypes.c_void_p), ("cap", ctypes.c_int32),
                ("q", ctypes.c_void_p), ("H", ctypes.c_int32), ("sm_scale", ctypes.c_float),
                ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p)]


EXPORTS = ["csa_workspace_bytes", "csa_workspace_init", "csa_kv_pack_fp4", "csa_indexer_full",
           "csa_indexer_reindex", "csa_indexer_block_scores", "csa_topk_blocks", "csa_index_reuse", "csa_sparse_decode_attn", "csa_decode_layer",
           "csa_check_device_error", "csa_status_string", "csa_indexer_full_noalloc",
           "csa_indexer_screen_bounds", "csa_kv_norm_rope_pack_fp4", "csa_candidates_concat",
           "csa_shard_blocks", "csa_attn_merge", "csa_kv_record_bytes", "csa_kv_export", "csa_kv_import",
           "csa_kv_append_fp4", "csa_kv_unpack_fp4", "csa_dense_attn_workspace_bytes", "csa_dense_attn"]

_lib = None


def lib():
    """Load libcsa.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError("libcsa.so not found at %s; build it with "
                          "`python -m fp4_compressed_sparse_kv_b200.build`" % LIB_PATH)
    L = ctypes.CDLL(LIB_PATH)
    P, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    st = ctypes.c_int
    L.csa_workspace_bytes.restype = sz
    L.csa_workspace_bytes.argtypes = [i32, i32, i32, i32]
    L.csa_workspace_init.restype = st
    L.csa_workspace_init.argtypes = [P, sz, P]
    L.csa_kv_pack_fp4.restype = st
    L.csa_kv_pack_fp4.argtypes = [ctypes.POINTER(KVLayerC), P, P, P, P, i32, P, sz, P]
    L.csa_kv_norm_rope_pack_fp4.restype = st
    L.csa_kv_norm_rope_pack_fp4.argtypes = [ctypes.POINTER(KVLayerC), P, P, P, P, P, P, i32, P, sz, P]
    L.csa_indexer_full.restype = st
    L.csa_indexer_full.argtypes = [ctypes.POINTER(KVLayerC), ctypes.POINTER(BatchC), P, P, i32, P, P,
                                   P, sz, P]
    L.csa_indexer_reindex.restype = st
    L.csa_indexer_reindex.argtypes = [ctypes.POINTER(KVLayerC), ctypes.POINTER(BatchC), P, P, P, P,
                                      i32, i32, P, P, P, sz, P]
    L.csa_indexer_block_scores.restype = st
    L.csa_indexer_block_scores.argtypes = [ctypes.POINTER(KVLayerC), ctypes.POINTER(BatchC), P, P, P, P,
                                           i32, P, i32, P, sz, P]
    L.csa_indexer_screen_bounds.restype = st
    L.csa_indexer_screen_bounds.argtypes = [ctypes.POINTER(KVLayerC), ctypes.POINTER(BatchC), P, P, P, P,
                                            i32, P, sz, P]
    L.csa_topk_blocks.restype = st
    L.csa_topk_blocks.argtypes = [ctypes.POINTER(BatchC), P, i32, P, P, i32, i32, P, P, P, sz, P]
    L.csa_index_reuse.restype = st
    L.csa_index_reuse.argtypes = [i32, P, P, i32, P, P, i32, P, sz, P]
    L.csa_sparse_decode_attn.restype = st
    L.csa_sparse_decode_attn.argtypes = [ctypes.POINTER(KVLayerC), ctypes.POINTER(BatchC), P, i32,
                                         ctypes.c_float, P, P, i32, P, P, P, sz, P]
    L.csa_decode_layer.restype = st
    L.csa_decode_layer.argtypes = [ctypes.POINTER(KVLayerC), ctypes.POINTER(BatchC),
                                   ctypes.POINTER(LayerStepC), P, sz, P]
    L.csa_indexer_full_noalloc.restype = st
    L.csa_indexer_full_noalloc.argtypes = [ctypes.POINTER(KVLayerC), ctypes.POINTER(BatchC), P, P, i32, P, P,
                                           P, P]
    L.csa_candidates_concat.restype = st
    L.csa_candidates_concat.argtypes = [i32, i32, i32, P, P, P, P, P, P, P, P, sz, P]
    L.csa_shard_blocks.restype = st
    L.csa_shard_blocks.argtypes = [i32, P, P, i32, P, P, P, P, i32, P, sz, P]
    L.csa_attn_merge.restype = st
    L.csa_attn_merge.argtypes = [i32, i32, i32, P, P, P, P, P]
    L.csa_kv_record_bytes.restype = sz
    L.csa_kv_record_bytes.argtypes = [i32]
    L.csa_kv_export.restype = st
    L.csa_kv_export.argtypes = [ctypes.POINTER(KVLayerC), P, i32, P, P, sz, P]
    L.csa_kv_import.restype = st
    L.csa_kv_import.argtypes = [ctypes.POINTER(KVLayerC), P, i32, P, P, sz, P]
    # layer and batch: a structure's address or its bytes
    L.csa_kv_append_fp4.restype = st
    L.csa_kv_append_fp4.argtypes = [P, P, P, i32, P, P, P, P, i32, P, sz, P]
    L.csa_kv_unpack_fp4.restype = st
    L.csa_kv_unpack_fp4.argtypes = [P, P, P, i32, P, P, sz, P]
    L.csa_dense_attn_workspace_bytes.restype = sz
    L.csa_dense_attn_workspace_bytes.argtypes = []
    L.csa_dense_attn.restype = st
    L.csa_dense_attn.argtypes = [P, P, P, i32, P, i32, ctypes.c_float, ctypes.c_float, P, P, P, P, P, sz, P]
    L.csa_check_device_error.restype = st
    L.csa_check_device_error.argtypes = [P, P, ctypes.POINTER(ctypes.c_int64)]
    L.csa_status_string.restype = ctypes.c_char_p
    L.csa_status_string.argtypes = [ctypes.c_int]
    _lib = L
    return L


def _check(status, where):
    if status != 0:
        raise CsaError(status, where)


def _ptr(t, name):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor (the library has no CPU path)" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _buf_ptr(t, name):
    """A device tensor, or a page-locked host tensor (the kernel reads or writes it over the bus)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if not (t.is_cuda or t.is_pinned()):
        raise ValueError("%s must be a CUDA tensor or a pinned host tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _stream(stream):
    """Handle of `stream`, or of the current stream (without a Stream object, which costs 3 us)."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def default_sm_scale():
    return 1.0 / math.sqrt(LATENT)


# ------------------------------------------------------------------------------------------------
# Buffers
# ------------------------------------------------------------------------------------------------
class KVLayer:
    """One Full layer's caches: FP4 codes + E4M3 scales + E4M3 indexer keys (pages of 64 tokens)
    and the FP8 sliding-window ring (one 128-slot row per sequence)."""

    def __init__(self, num_pages, num_rows, device="cuda"):
        u8 = dict(dtype=torch.uint8, device=device)
        self.codes = torch.zeros((num_pages, PAGE, LATENT // 2), **u8)
        self.scales = torch.zeros((num_pages, PAGE, LATENT // 16), **u8)
        self.keys = torch.zeros((num_pages, PAGE, IDX_DIM), **u8)
        self.swa = torch.zeros((num_rows, WINDOW, LATENT), **u8)
        self.swa_scale = torch.zeros((num_rows, WINDOW), dtype=torch.float32, device=device)
        self.num_pages, self.num_rows = num_pages, num_rows

    def c(self):
        return KVLayerC(_ptr(self.codes, "codes"), _ptr(self.scales, "scales"),
                        _ptr(self.keys, "keys"), _ptr(self.swa, "swa"),
                        _ptr(self.swa_scale, "swa_scale"), self.num_pages, self.num_rows)


class Batch:
    """Decode-batch metadata: seq_len [B], block_table [B][max_pages], swa_row [B] (int32, device)
    and the host bound max_seq_len."""

    def __init__(self, seq_len, block_table, swa_row, max_seq_len):
        self.seq_len, self.block_table, self.swa_row = seq_len, block_table, swa_row
        self.B = int(seq_len.numel())
        self.max_pages = int(block_table.shape[1])
        self.max_seq_len = int(max_seq_len)

    def c(self):
        return BatchC(self.B, _ptr(self.seq_len, "seq_len"), _ptr(self.block_table, "block_table"),
                      self.max_pages, _ptr(self.swa_row, "swa_row"), self.max_seq_len)


def workspace_bytes(B, H, max_seq_len, cap):
    n = lib().csa_workspace_bytes(B, H, max_seq_len, cap)
    if n == 0:
        raise CsaError(1, "csa_workspace_bytes")
    return n


def workspace(B, H, max_seq_len, cap, device="cuda", stream=None):
    """Allocate (with torch) and initialise a workspace for these sizes."""
    ws = torch.empty(workspace_bytes(B, H, max_seq_len, cap), dtype=torch.uint8, device=device)
    workspace_init(ws, stream)
    return ws


def workspace_init(ws, stream=None):
    _check(lib().csa_workspace_init(_ptr(ws, "ws"), ws.numel(), _stream(stream)), "csa_workspace_init")


# ------------------------------------------------------------------------------------------------
# Entry points (same names as the C-ABI, without the csa_ prefix)
# ------------------------------------------------------------------------------------------------
def _bits(t):
    return t.view(torch.int16) if t.dtype == torch.bfloat16 else t


def kv_pack_fp4(layer, latent, idx_key, slot, swa_slot, ws, stream=None):
    n = int(slot.numel())
    lc = layer.c()
    _check(lib().csa_kv_pack_fp4(ctypes.byref(lc), _ptr(_bits(latent), "latent"),
                                 _ptr(_bits(idx_key), "idx_key"), _ptr(slot, "slot"),
                                 _ptr(swa_slot, "swa_slot"), n, _ptr(ws, "ws"), ws.numel(),
                                 _stream(stream)), "csa_kv_pack_fp4")


def kv_norm_rope_pack_fp4(layer, latent_prenorm, norm_weight, rope_cos_sin, idx_key, slot, swa_slot, ws,
                          stream=None):
    """Pack from the pre-norm latent: RMSNorm (norm_weight float32 [512]), RoPE on channels 448..511
    (rope_cos_sin float32 [n, 32, 2] of (cos, sin) pairs), bf16, then the FP4 / E4M3 / FP8 pack."""
    n = int(slot.numel())
    lc = layer.c()
    _check(lib().csa_kv_norm_rope_pack_fp4(ctypes.byref(lc), _ptr(_bits(latent_prenorm), "latent_prenorm"),
                                           _ptr(norm_weight, "norm_weight"), _ptr(rope_cos_sin, "rope_cos_sin"),
                                           _ptr(_bits(idx_key), "idx_key"), _ptr(slot, "slot"),
                                           _ptr(swa_slot, "swa_slot"), n, _ptr(ws, "ws"), ws.numel(),
                                           _stream(stream)), "csa_kv_norm_rope_pack_fp4")


def indexer_full(layer, batch, iq, iw, k, out_blocks, out_count, ws, stream=None):
    lc, bc = layer.c(), batch.c()
    _check(lib().csa_indexer_full(ctypes.byref(lc), ctypes.byref(bc), _ptr(_bits(iq), "iq"),
                                  _ptr(iw, "iw"), int(k), _ptr(out_blocks, "out_blocks"),
                                  _ptr(out_count, "out_count"), _ptr(ws, "ws"), ws.numel(),
                                  _stream(stream)), "csa_indexer_full")


def indexer_reindex(layer, batch, iq, iw, pool, pool_count, k_r, out_blocks, out_count, ws,
                    stream=None):
    lc, bc = layer.c(), batch.c()
    _check(lib().csa_indexer_reindex(ctypes.byref(lc), ctypes.byref(bc), _ptr(_bits(iq), "iq"),
                                     _ptr(iw, "iw"), _ptr(pool, "pool"),
                                     _ptr(pool_count, "pool_count"), int(pool.shape[1]), int(k_r),
                                     _ptr(out_blocks, "out_blocks"), _ptr(out_count, "out_count"),
                                     _ptr(ws, "ws"), ws.numel(), _stream(stream)),
           "csa_indexer_reindex")


def indexer_block_scores(layer, batch, iq, iw, scores, ws, pool=None, pool_count=None, stream=None):
    """Block scores into `scores` float32 [B, stride] (Full when pool is None, else Reindex)."""
    lc, bc = layer.c(), batch.c()
    _check(lib().csa_indexer_block_scores(ctypes.byref(lc), ctypes.byref(bc), _ptr(_bits(iq), "iq"),
                                          _ptr(iw, "iw"), _ptr(pool, "pool"),
                                          _ptr(pool_count, "pool_count"),
                                          int(pool.shape[1]) if pool is not None else 0,
                                          _ptr(scores, "scores"), int(scores.shape[1]), _ptr(ws, "ws"),
                                          ws.numel(), _stream(stream)), "csa_indexer_block_scores")


def indexer_screen_bounds(layer, batch, iq, iw, lower, upper, ws, stream=None):
    """Per-block bounds of the exact Full score from the tensor-core screen: float32 [B, stride] each,
    lower <= score <= upper in Top-K order (-NaN / +NaN where no bound could be formed)."""
    lc, bc = layer.c(), batch.c()
    if lower.shape != upper.shape:
        raise ValueError("lower and upper must have the same shape")
    _check(lib().csa_indexer_screen_bounds(ctypes.byref(lc), ctypes.byref(bc), _ptr(_bits(iq), "iq"),
                                           _ptr(iw, "iw"), _ptr(lower, "lower"), _ptr(upper, "upper"),
                                           int(lower.shape[1]), _ptr(ws, "ws"), ws.numel(), _stream(stream)),
           "csa_indexer_screen_bounds")


def topk_blocks(batch, scores, k, out_blocks, out_count, ws, pool=None, pool_count=None, stream=None):
    bc = batch.c()
    _check(lib().csa_topk_blocks(ctypes.byref(bc), _ptr(scores, "scores"), int(scores.shape[1]),
                                 _ptr(pool, "pool"), _ptr(pool_count, "pool_count"),
                                 int(pool.shape[1]) if pool is not None else 0, int(k),
                                 _ptr(out_blocks, "out_blocks"), _ptr(out_count, "out_count"),
                                 _ptr(ws, "ws"), ws.numel(), _stream(stream)), "csa_topk_blocks")


def index_reuse(prev_blocks, prev_count, out_blocks, out_count, ws, stream=None):
    _check(lib().csa_index_reuse(int(prev_blocks.shape[0]), _ptr(prev_blocks, "prev_blocks"),
                                 _ptr(prev_count, "prev_count"), int(prev_blocks.shape[1]),
                                 _ptr(out_blocks, "out_blocks"), _ptr(out_count, "out_count"),
                                 int(out_blocks.shape[1]), _ptr(ws, "ws"), ws.numel(),
                                 _stream(stream)), "csa_index_reuse")


def sparse_decode_attn(layer, batch, q, sm_scale, blocks, count, out, lse, ws, stream=None):
    lc, bc = layer.c(), batch.c()
    H = int(q.shape[1])
    _check(lib().csa_sparse_decode_attn(ctypes.byref(lc), ctypes.byref(bc), _ptr(_bits(q), "q"), H,
                                        float(sm_scale), _ptr(blocks, "blocks"),
                                        _ptr(count, "count"), int(blocks.shape[1]),
                                        _ptr(out, "out"), _ptr(lse, "lse"), _ptr(ws, "ws"),
                                        ws.numel(), _stream(stream)), "csa_sparse_decode_attn")


def decode_layer(mode, layer, batch, q, out, lse, blocks, count, ws, iq=None, iw=None, k=0,
                 prev_blocks=None, prev_count=None, sm_scale=None, stream=None):
    """One layer's decode step: Full (k), Reindex (pool = prev, k_r = k) or Reuse (prev)."""
    lc, bc = layer.c(), batch.c()
    step = LayerStepC(int(mode), _ptr(_bits(iq), "iq") if iq is not None else None,
                      _ptr(iw, "iw") if iw is not None else None, int(k),
                      _ptr(prev_blocks, "prev_blocks") if prev_blocks is not None else None,
                      _ptr(prev_count, "prev_count") if prev_count is not None else None,
                      int(prev_blocks.shape[1]) if prev_blocks is not None else 0,
                      _ptr(blocks, "blocks"), _ptr(count, "count"), int(blocks.shape[1]),
                      _ptr(_bits(q), "q"), int(q.shape[1]),
                      float(default_sm_scale() if sm_scale is None else sm_scale),
                      _ptr(out, "out"), _ptr(lse, "lse"))
    _check(lib().csa_decode_layer(ctypes.byref(lc), ctypes.byref(bc), ctypes.byref(step),
                                  _ptr(ws, "ws"), ws.numel(), _stream(stream)), "csa_decode_layer")


def indexer_full_noalloc(layer, batch, iq, iw, k, out_blocks, out_count, dev_status=None, stream=None):
    """csa_indexer_full without a workspace: the library's own fixed scratch array is used instead, so
    nothing is allocated.  For callers that cannot provide device memory; see include/csa.h for the
    size limit and the rule that calls overlapping on the GPU must not share a device."""
    lc, bc = layer.c(), batch.c()
    _check(lib().csa_indexer_full_noalloc(ctypes.byref(lc), ctypes.byref(bc), _ptr(_bits(iq), "iq"),
                                          _ptr(iw, "iw"), int(k), _ptr(out_blocks, "out_blocks"),
                                          _ptr(out_count, "out_count"), _ptr(dev_status, "dev_status"),
                                          _stream(stream)), "csa_indexer_full_noalloc")


def candidates_concat(ids, scores, counts, offsets, out_ids, out_scores, out_count, ws, stream=None):
    """ids int32 [R, B, cap] (local block ids), scores float32 [R, B, cap], counts / offsets int32
    [R, B] -> out_ids int32 [B, R * cap] (global ids), out_scores float32 [B, R * cap], out_count [B]."""
    R, B, cap = (int(x) for x in ids.shape)
    _check(lib().csa_candidates_concat(R, B, cap, _ptr(ids, "ids"), _ptr(scores, "scores"),
                                       _ptr(counts, "counts"), _ptr(offsets, "offsets"),
                                       _ptr(out_ids, "out_ids"), _ptr(out_scores, "out_scores"),
                                       _ptr(out_count, "out_count"), _ptr(ws, "ws"), ws.numel(),
                                       _stream(stream)), "csa_candidates_concat")


def shard_blocks(blocks, count, lo, hi, out_blocks, out_count, ws, stream=None):
    """Entries of blocks int32 [B, cap] (count [B]) in [lo[b], hi[b]) minus lo[b], in order."""
    B, cap = (int(x) for x in blocks.shape)
    _check(lib().csa_shard_blocks(B, _ptr(blocks, "blocks"), _ptr(count, "count"), cap, _ptr(lo, "lo"),
                                  _ptr(hi, "hi"), _ptr(out_blocks, "out_blocks"), _ptr(out_count, "out_count"),
                                  int(out_blocks.shape[1]), _ptr(ws, "ws"), ws.numel(), _stream(stream)),
           "csa_shard_blocks")


def attn_merge(out_parts, lse_parts, out, lse, stream=None):
    """out_parts float32 [R, B, H, 512], lse_parts float32 [R, B, H] -> out [B, H, 512], lse [B, H]."""
    R, B, H = (int(x) for x in lse_parts.shape)
    _check(lib().csa_attn_merge(R, B, H, _ptr(out_parts, "out_parts"), _ptr(lse_parts, "lse_parts"),
                                _ptr(out, "out"), _ptr(lse, "lse"), _stream(stream)), "csa_attn_merge")


def kv_record_bytes(n):
    """Bytes of the persistent record of an n-token sequence: 26,624 per 64-token page."""
    return int(lib().csa_kv_record_bytes(int(n)))


def _record_args(layer, block_table, n, buf, name):
    if buf.dtype != torch.uint8 or buf.numel() < kv_record_bytes(n):
        raise ValueError("%s must be a uint8 tensor of at least kv_record_bytes(n) bytes" % name)
    if block_table.dtype != torch.int32 or block_table.numel() < (int(n) + PAGE - 1) // PAGE:
        raise ValueError("block_table must be int32 with one entry per page of the sequence")
    return layer.c(), _ptr(block_table, "block_table"), _buf_ptr(buf, name)


def kv_export(layer, block_table, n, dst, ws, stream=None):
    """Copy the persistent record (FP4 codes, scales, indexer keys; no window) of the n-token sequence
    whose pages are block_table[0 .. ceil(n/64)) into dst (device, or pinned host)."""
    lc, bt, d = _record_args(layer, block_table, n, dst, "dst")
    _check(lib().csa_kv_export(ctypes.byref(lc), bt, int(n), d, _ptr(ws, "ws"), ws.numel(), _stream(stream)),
           "csa_kv_export")


def kv_import(layer, block_table, n, src, ws, stream=None):
    """Write a persistent record back into the pages block_table[0 .. ceil(n/64)).  The window is
    restored afterwards by replaying the last min(n, 128) tokens through kv_pack_fp4."""
    lc, bt, s = _record_args(layer, block_table, n, src, "src")
    _check(lib().csa_kv_import(ctypes.byref(lc), bt, int(n), s, _ptr(ws, "ws"), ws.numel(), _stream(stream)),
           "csa_kv_import")


_runs_mod = None


def _runs():
    """The extension that checks and marshals the arguments of append and read-back, bound to the library.  Their
    kernels run 2 to 4 us for a decode step, and marshalling in Python alone took 5."""
    global _runs_mod
    if _runs_mod is None:
        L = lib()
        try:
            from . import _runs as mod
        except ImportError as e:
            raise ImportError("_runs.so is missing or does not load; build it with "
                              "`python -m fp4_compressed_sparse_kv_b200.build`") from e
        built_for = getattr(mod, "torch_version", "another version")
        if built_for != torch.__version__:
            raise ImportError("_runs.so was built for PyTorch %s and this is %s; build it again with "
                              "`python -m fp4_compressed_sparse_kv_b200.build`" % (built_for, torch.__version__))
        mod.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (L.csa_kv_append_fp4, L.csa_kv_unpack_fp4)))
        _runs_mod = mod
    return _runs_mod


# The attention's layer and batch are packed as bytes laid out like KVLayerC and BatchC, which costs a third of a
# ctypes structure.
_pack_layer = struct.Struct("=5Q2i").pack
_pack_batch = struct.Struct("=i4xQQi4xQi4x").pack


def _run_device(t, name):
    """The current device, which has to be where the run's tensors are (`t` is one of them)."""
    dev = t.get_device() if isinstance(t, torch.Tensor) else -1
    if dev < 0:
        _ptr(t, name)
        raise TypeError("%s must be a torch tensor" % name)
    if dev != torch.cuda.current_device():
        raise ValueError("%s is on device %d, which is not the current one" % (name, dev))
    return dev


def _run_ptr(t, name, dev):
    """Address of a contiguous tensor on device dev; 0 for None."""
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor) or t.get_device() != dev or not t.is_contiguous():
        _ptr(t, name)
        raise ValueError("%s is not on the current device" % name)
    return t.data_ptr()


def _run_handles(layer, batch, dev):
    """Bytes of the C structures of a layer and a batch."""
    p = _run_ptr
    return (_pack_layer(p(layer.codes, "codes", dev), p(layer.scales, "scales", dev), p(layer.keys, "keys", dev),
                        p(layer.swa, "swa", dev), p(layer.swa_scale, "swa_scale", dev), layer.num_pages, layer.num_rows),
            _pack_batch(batch.B, p(batch.seq_len, "seq_len", dev), p(batch.block_table, "block_table", dev),
                        batch.max_pages, p(batch.swa_row, "swa_row", dev), batch.max_seq_len))


def _run_rows(batch, cu_rows):
    if cu_rows.dtype is not torch.int32 or cu_rows.numel() != batch.B + 1:
        raise ValueError("cu_rows must be int32 with batch.B + 1 entries")


def _run_array(t, name, dtype, shape):
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError("%s must be %s of shape %s" % (name, dtype, list(shape)))


def kv_append_fp4(layer, batch, cu_rows, latent, idx_key, ws, norm_weight=None, rope_table=None, stream=None):
    """Write a ragged run into the caches by position: rows cu_rows[b] .. cu_rows[b+1] - 1 of latent
    (bf16 [rows, 512]) and idx_key (bf16 [rows, 128]) are the last positions of sequence b (batch.seq_len
    counts them).  norm_weight float32 [512] and rope_table float32 [positions, 32, 2] of (cos, sin) apply
    RMSNorm and the rotation of each row's position first; the last 128 positions also go to the window."""
    _check(_runs().kv_append_fp4(layer, batch, cu_rows, latent, idx_key, ws, norm_weight, rope_table, stream),
           "csa_kv_append_fp4")


def kv_unpack_fp4(layer, batch, cu_rows, latent, ws, stream=None):
    """Read a ragged run's FP4 entries back as values into latent, bf16 [rows, 512] (exact)."""
    _check(_runs().kv_unpack_fp4(layer, batch, cu_rows, latent, ws, stream), "csa_kv_unpack_fp4")


def dense_attn_workspace(device="cuda", stream=None):
    """Allocate (with torch) and initialise a workspace for dense_attn; one size serves every call."""
    ws = torch.empty(lib().csa_dense_attn_workspace_bytes(), dtype=torch.uint8, device=device)
    workspace_init(ws, stream)
    return ws


def dense_attn(layer, batch, cu_rows, q, out, lse, ws, sm_scale=None, softcap=0.0, slopes=None, spans=None,
               stream=None):
    """Attention of a ragged run's queries q (bf16 [rows, H, 512], H <= 128) over every visible position of
    the FP4 cache: out bf16 [rows, H, 512], lse float32 [rows, H].  Causal, or spans int32 [rows, 2] of the
    positions lo <= j < hi each row sees; softcap > 0 caps scores by softcap * tanh(s / softcap); slopes
    float32 [H] subtracts slopes[h] * |p - j|.  The window ring, which sparse_decode_attn adds, takes no part."""
    rows, H = q.shape[0], q.shape[1]
    _run_rows(batch, cu_rows)
    _run_array(q, "q", torch.bfloat16, (rows, H, LATENT))
    _run_array(out, "out", torch.bfloat16, (rows, H, LATENT))
    _run_array(lse, "lse", torch.float32, (rows, H))
    if slopes is not None:
        _run_array(slopes, "slopes", torch.float32, (H,))
    if spans is not None:
        _run_array(spans, "spans", torch.int32, (rows, 2))
    dev, p = _run_device(ws, "ws"), _run_ptr
    lc, bc = _run_handles(layer, batch, dev)
    _check(lib().csa_dense_attn(lc, bc, p(cu_rows, "cu_rows", dev), rows, p(q, "q", dev), H,
                                default_sm_scale() if sm_scale is None else sm_scale, softcap,
                                p(slopes, "slopes", dev), p(spans, "spans", dev), p(out, "out", dev), p(lse, "lse", dev),
                                p(ws, "ws", dev), ws.numel(), _stream(stream)), "csa_dense_attn")


def check_device_error(ws, stream=None):
    """Synchronise, read and clear the workspace status.  Returns (status, detail)."""
    d = ctypes.c_int64(0)
    s = lib().csa_check_device_error(_ptr(ws, "ws"), _stream(stream), ctypes.byref(d))
    return s, d.value
