"""Absorbed MLA decode over a quantized paged latent KV cache, for GB300.

Thin Python binding over the C ABI in ``include/mla.h`` (``libmla_gb300.so``,
built in-tree by ``mla_latent_kv_append_gb300.build``).  The functions here
only marshal arguments - torch tensors supply device memory and the current
CUDA stream - and every step of the computation runs in the library's CUDA
kernels.  Importing this package without the built library raises; there is
no CPU fallback.

Names follow the C ABI:

    mla_cache_append(cache, c_new, kpe_new, slot, dev_err=None)
    mla_q_absorb(q_nope, w_uk, q_lat)
    mla_decode_absorbed(cache, q_lat, q_pe, block_table, seq_lens, workspace,
                        o_lat, lse=None, dev_err=None, softmax_scale=None,
                        num_splits=0)
    mla_out_unabsorb(o_lat, w_uv, o)

plus ``CacheLayer`` (one layer's pool, formats and, for the outlier-protected
format, its protected channels), ``mla_select_outlier_channels`` (their
calibration), ``mla_cache_page_layout``,
``mla_cache_pool_bytes``, ``mla_decode_workspace_bytes``,
``mla_decode_absorbed_unabsorb`` (the decode and the output projection in
one call), ``mla_decode_absorbed_noalloc`` (the decode for callers that cannot allocate),
``mla_prefill_absorbed`` / ``mla_prefill_workspace_bytes`` (causal attention
of a prefill chunk; ``mla_set_prefill_path`` / ``mla_prefill_path_taken``
choose and report its implementation: tcgen05 tensor cores or the decode
kernels) and ``mla_lse_merge`` (merges per-part results of a context-sharded decode;
the host side of that exchange is in ``sharded``).

A serving step over a ragged batch (decodes, drafts and prefill chunks
together, lengths on the device) is ``mla_plan_chunks`` (block tables, slots,
positions), ``mla_rope``, ``mla_cache_append`` and ``mla_chunk_attention``
(its workspace: ``mla_chunk_workspace_bytes``).
"""

import ctypes
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmla_gb300.so")

FMT_BF16, FMT_INT8_SYM, FMT_INT4_ASYM, FMT_INT4_SYM = 0, 1, 2, 3
FMT_INT8_G8, FMT_INT8_G32, FMT_INT8_G64, FMT_INT8_TOKEN = 4, 5, 6, 7    # INT8 latent, other block counts
FMT_INT8_OUTLIER = 8        # INT8 latent with OUTLIER_CHANNELS protected bf16 channels

PREFILL_AUTO = 0            # mla_set_prefill_path: tensor cores for large chunks, else decode kernels
PREFILL_DECODE_KERNELS = 1
PREFILL_TENSOR_CORES = 2
OUTLIER_CHANNELS = 25
DEVERR_SLOT, DEVERR_PAGE, DEVERR_SEQLEN, DEVERR_TIMEOUT, DEVERR_NO_PAGES = 1, 2, 4, 8, 16
CHUNK_SHORT = 64            # mla_chunk_attention: sequences with more new tokens count toward kv_tokens
KV_LORA_RANK, ROPE_DIM, QK_NOPE_DIM, V_DIM, PAGE_TOKENS = 512, 64, 128, 128, 64
DEFAULT_SOFTMAX_SCALE = 1.0 / math.sqrt(QK_NOPE_DIM + ROPE_DIM)

STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "CUDA error", 4: "device bounds error"}


class MlaError(RuntimeError):
    def __init__(self, fn, status, detail=""):
        super().__init__("%s failed: %s (status %d)%s" % (fn, STATUS.get(status, "?"), status,
                                                         ": " + detail if detail else ""))
        self.status = status


class _CacheLayer(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int32), ("latent_fmt", ctypes.c_int32), ("kpe_fmt", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("pool", ctypes.c_void_p),
                ("outlier_channels", ctypes.POINTER(ctypes.c_int32))]


class PageLayout(ctypes.Structure):
    _fields_ = [("page_bytes", ctypes.c_int64), ("block_bytes", ctypes.c_int64), ("codes_off", ctypes.c_int64),
                ("codes_row_bytes", ctypes.c_int64),
                ("scale_off", ctypes.c_int64), ("zero_off", ctypes.c_int64), ("kpe_off", ctypes.c_int64),
                ("kpe_row_bytes", ctypes.c_int64), ("kpe_scale_off", ctypes.c_int64),
                ("bound_off", ctypes.c_int64), ("outlier_off", ctypes.c_int64)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError("libmla_gb300.so is not built: run `python mla_latent_kv_append_gb300/build.py` "
                          "(or __graft_entry__.build()) on a machine with nvcc")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, SZ, F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
    I64 = ctypes.c_int64
    CP = ctypes.POINTER(_CacheLayer)
    sig = {
        "mla_abi_version": (I32, []),
        "mla_status_string": (ctypes.c_char_p, [I32]),
        "mla_last_cuda_error": (ctypes.c_char_p, []),
        "mla_cache_page_layout": (I32, [CP, ctypes.POINTER(PageLayout)]),
        "mla_cache_pool_bytes": (SZ, [CP]),
        "mla_cache_append": (I32, [CP, P, P, P, I32, P, P]),
        "mla_q_absorb": (I32, [P, P, P, I32, I32, P]),
        "mla_decode_workspace_bytes": (SZ, [I32, I32, I32]),
        "mla_decode_absorbed": (I32, [CP, P, P, P, I32, P, I32, I32, F32, I32, P, SZ, P, P, P, P]),
        "mla_decode_absorbed_unabsorb": (I32, [CP, P, P, P, I32, P, I32, I32, F32, I32, P, SZ, P, P, P, P, P, P]),
        "mla_decode_kernel_count": (I32, [CP, I32, I32, I32, I32]),
        "mla_out_unabsorb": (I32, [P, P, P, I32, I32, P]),
        "mla_decode_absorbed_noalloc": (I32, [CP, P, P, P, I32, P, I32, I32, F32, I32, P, P, P, P]),
        "mla_lse_merge": (I32, [P, P, I32, I32, I32, P, P, P]),
        "mla_prefill_workspace_bytes": (SZ, [I32, I32]),
        "mla_prefill_absorbed": (I32, [CP, P, P, P, I32, I32, I32, I32, F32, P, SZ, P, P, P, P]),
        "mla_set_wait_limit_ns": (ctypes.c_int64, [ctypes.c_int64]),
        "mla_set_prefill_path": (I32, [I32]),
        "mla_prefill_path_taken": (I32, [I32, I32, I32]),
        "mla_select_outlier_channels": (I32, [P, I32, P, P]),
        "mla_plan_chunks": (I32, [P, P, P, I32, P, I32, I32, P, I32, P, I32, I32, P, P, P, P, P, P, P, P, P]),
        "mla_rope": (I32, [P, I64, I64, P, I64, P, I32, P, P, I32, I32, I32, I32, F32, P, I64, I64, P, I64, P]),
        "mla_chunk_attention": (I32, [CP, P, I64, I64, P, I64, I64, P, P, P, I32, P, P, I32, I32, I32, I32, I64, F32,
                                      P, SZ, P, P, P]),
        "mla_chunk_workspace_bytes": (SZ, [I32, I32, I32, I32, I64]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn, status):
    if status != 0:
        detail = lib.mla_last_cuda_error().decode() if status == 3 else ""
        raise MlaError(fn, status, detail)


def _need(t, dtype, shape, name):
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous() or not t.is_cuda:
        raise ValueError("%s: expected contiguous CUDA %s %s, got %s %s" % (name, dtype, tuple(shape), t.dtype,
                                                                            tuple(t.shape)))


class CacheLayer:
    """One layer's paged latent cache: a caller-owned pool tensor plus formats
    (and, for FMT_INT8_OUTLIER, the layer's OUTLIER_CHANNELS protected
    channels: a sequence of increasing ints in [0, 512))."""

    def __init__(self, num_pages, latent_fmt, kpe_fmt, device="cuda", pool=None, outlier_channels=None):
        self.num_pages, self.latent_fmt, self.kpe_fmt = int(num_pages), int(latent_fmt), int(kpe_fmt)
        self.outlier_channels = None
        if outlier_channels is not None:
            ch = [int(c) for c in outlier_channels]
            self.outlier_channels = (ctypes.c_int32 * len(ch))(*ch)
        nbytes = mla_cache_pool_bytes(self.num_pages, self.latent_fmt, self.kpe_fmt)
        if nbytes == 0:
            raise ValueError("invalid cache descriptor")
        if pool is None:
            pool = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        if pool.numel() < nbytes or pool.dtype != torch.uint8 or pool.data_ptr() % 256:
            raise ValueError("pool must be a uint8 tensor of >= %d bytes, 256-byte aligned" % nbytes)
        self.pool = pool
        self.layout = mla_cache_page_layout(self.latent_fmt, self.kpe_fmt)

    def c_struct(self):
        oc = None if self.outlier_channels is None else ctypes.cast(self.outlier_channels,
                                                                      ctypes.POINTER(ctypes.c_int32))
        return _CacheLayer(self.num_pages, self.latent_fmt, self.kpe_fmt, 0, self.pool.data_ptr(), oc)


def mla_cache_page_layout(latent_fmt, kpe_fmt):
    out = PageLayout()
    c = _CacheLayer(1, latent_fmt, kpe_fmt, 0, None)
    _check("mla_cache_page_layout", lib.mla_cache_page_layout(ctypes.byref(c), ctypes.byref(out)))
    return out


def mla_cache_pool_bytes(num_pages, latent_fmt, kpe_fmt):
    c = _CacheLayer(num_pages, latent_fmt, kpe_fmt, 0, None)
    return int(lib.mla_cache_pool_bytes(ctypes.byref(c)))


def mla_select_outlier_channels(c_sample, out=None, stream=None):
    """Protected channels of FMT_INT8_OUTLIER from a calibration sample
    (bf16 [n, 512] on the GPU): the OUTLIER_CHANNELS channels with the
    largest max |x|, increasing; returns the int32 device tensor."""
    n = c_sample.shape[0]
    _need(c_sample, torch.bfloat16, (n, KV_LORA_RANK), "c_sample")
    if out is None:
        out = torch.empty(OUTLIER_CHANNELS, dtype=torch.int32, device=c_sample.device)
    _need(out, torch.int32, (OUTLIER_CHANNELS,), "out")
    _check("mla_select_outlier_channels", lib.mla_select_outlier_channels(_ptr(c_sample), n, _ptr(out),
                                                                          _stream(stream)))
    return out


def mla_decode_workspace_bytes(batch, heads, num_splits=0):
    return int(lib.mla_decode_workspace_bytes(batch, heads, num_splits))


def mla_cache_append(cache, c_new, kpe_new, slot, dev_err=None, stream=None):
    n = slot.numel()
    _need(c_new, torch.bfloat16, (n, KV_LORA_RANK), "c_new")
    _need(kpe_new, torch.bfloat16, (n, ROPE_DIM), "kpe_new")
    _need(slot, torch.int32, (n,), "slot")
    cs = cache.c_struct()
    _check("mla_cache_append", lib.mla_cache_append(ctypes.byref(cs), _ptr(c_new), _ptr(kpe_new), _ptr(slot), n,
                                                    _ptr(dev_err), _stream(stream)))


def mla_q_absorb(q_nope, w_uk, q_lat, stream=None):
    B, H = q_nope.shape[0], q_nope.shape[1]
    _need(q_nope, torch.bfloat16, (B, H, QK_NOPE_DIM), "q_nope")
    _need(w_uk, torch.bfloat16, (H, QK_NOPE_DIM, KV_LORA_RANK), "w_uk")
    _need(q_lat, torch.float32, (B, H, KV_LORA_RANK), "q_lat")
    _check("mla_q_absorb", lib.mla_q_absorb(_ptr(q_nope), _ptr(w_uk), _ptr(q_lat), B, H, _stream(stream)))


def mla_out_unabsorb(o_lat, w_uv, o, stream=None):
    B, H = o_lat.shape[0], o_lat.shape[1]
    _need(o_lat, torch.float32, (B, H, KV_LORA_RANK), "o_lat")
    _need(w_uv, torch.bfloat16, (H, KV_LORA_RANK, V_DIM), "w_uv")
    _need(o, torch.float32, (B, H, V_DIM), "o")
    _check("mla_out_unabsorb", lib.mla_out_unabsorb(_ptr(o_lat), _ptr(w_uv), _ptr(o), B, H, _stream(stream)))


def mla_decode_absorbed(cache, q_lat, q_pe, block_table, seq_lens, workspace, o_lat, lse=None, dev_err=None,
                        softmax_scale=None, num_splits=0, stream=None):
    B, H = q_lat.shape[0], q_lat.shape[1]
    _need(q_lat, torch.float32, (B, H, KV_LORA_RANK), "q_lat")
    _need(q_pe, torch.bfloat16, (B, H, ROPE_DIM), "q_pe")
    _need(block_table, torch.int32, (B, block_table.shape[1]), "block_table")
    _need(seq_lens, torch.int32, (B,), "seq_lens")
    _need(o_lat, torch.float32, (B, H, KV_LORA_RANK), "o_lat")
    if lse is not None:
        _need(lse, torch.float32, (B, H), "lse")
    scale = DEFAULT_SOFTMAX_SCALE if softmax_scale is None else float(softmax_scale)
    cs = cache.c_struct()
    _check("mla_decode_absorbed", lib.mla_decode_absorbed(
        ctypes.byref(cs), _ptr(q_lat), _ptr(q_pe), _ptr(block_table), block_table.shape[1], _ptr(seq_lens), B, H,
        scale, int(num_splits), _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(o_lat),
        _ptr(lse), _ptr(dev_err), _stream(stream)))


def mla_decode_kernel_count(cache, batch, heads, num_splits=0, with_unabsorb=False):
    cs = cache.c_struct()
    return int(lib.mla_decode_kernel_count(ctypes.byref(cs), batch, heads, num_splits, 1 if with_unabsorb else 0))


def mla_decode_absorbed_unabsorb(cache, q_lat, q_pe, block_table, seq_lens, workspace, o_lat, w_uv, o, lse=None,
                                 dev_err=None, softmax_scale=None, num_splits=0, stream=None):
    """mla_decode_absorbed then mla_out_unabsorb on its o_lat, in one call
    (the projection fused into the combine where its grid allows)."""
    B, H = q_lat.shape[0], q_lat.shape[1]
    _need(q_lat, torch.float32, (B, H, KV_LORA_RANK), "q_lat")
    _need(q_pe, torch.bfloat16, (B, H, ROPE_DIM), "q_pe")
    _need(block_table, torch.int32, (B, block_table.shape[1]), "block_table")
    _need(seq_lens, torch.int32, (B,), "seq_lens")
    _need(o_lat, torch.float32, (B, H, KV_LORA_RANK), "o_lat")
    _need(w_uv, torch.bfloat16, (H, KV_LORA_RANK, V_DIM), "w_uv")
    _need(o, torch.float32, (B, H, V_DIM), "o")
    if lse is not None:
        _need(lse, torch.float32, (B, H), "lse")
    scale = DEFAULT_SOFTMAX_SCALE if softmax_scale is None else float(softmax_scale)
    cs = cache.c_struct()
    _check("mla_decode_absorbed_unabsorb", lib.mla_decode_absorbed_unabsorb(
        ctypes.byref(cs), _ptr(q_lat), _ptr(q_pe), _ptr(block_table), block_table.shape[1], _ptr(seq_lens), B, H,
        scale, int(num_splits), _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(o_lat),
        _ptr(lse), _ptr(w_uv), _ptr(o), _ptr(dev_err), _stream(stream)))


def mla_decode_absorbed_noalloc(cache, q_lat, q_pe, block_table, seq_lens, o_lat, lse=None, dev_err=None,
                                softmax_scale=None, num_splits=0, stream=None):
    """mla_decode_absorbed without a workspace argument: for callers that
    cannot allocate device memory (see include/mla.h).  Concurrent calls on
    different streams share the library's scratch array and race."""
    B, H = q_lat.shape[0], q_lat.shape[1]
    _need(q_lat, torch.float32, (B, H, KV_LORA_RANK), "q_lat")
    _need(q_pe, torch.bfloat16, (B, H, ROPE_DIM), "q_pe")
    _need(block_table, torch.int32, (B, block_table.shape[1]), "block_table")
    _need(seq_lens, torch.int32, (B,), "seq_lens")
    _need(o_lat, torch.float32, (B, H, KV_LORA_RANK), "o_lat")
    if lse is not None:
        _need(lse, torch.float32, (B, H), "lse")
    scale = DEFAULT_SOFTMAX_SCALE if softmax_scale is None else float(softmax_scale)
    cs = cache.c_struct()
    _check("mla_decode_absorbed_noalloc", lib.mla_decode_absorbed_noalloc(
        ctypes.byref(cs), _ptr(q_lat), _ptr(q_pe), _ptr(block_table), block_table.shape[1], _ptr(seq_lens), B, H,
        scale, int(num_splits), _ptr(o_lat), _ptr(lse), _ptr(dev_err), _stream(stream)))


def mla_prefill_workspace_bytes(n, heads):
    return int(lib.mla_prefill_workspace_bytes(int(n), int(heads)))


def mla_prefill_absorbed(cache, q_lat, q_pe, block_table, ctx_before, workspace, o_lat, lse=None, dev_err=None,
                         softmax_scale=None, stream=None):
    """Causal attention of n just-appended query tokens of one sequence:
    query i (position ctx_before + i) attends to positions 0 .. ctx_before + i.
    block_table is the sequence's int32 page list [max_pages]."""
    n, H = q_lat.shape[0], q_lat.shape[1]
    _need(q_lat, torch.float32, (n, H, KV_LORA_RANK), "q_lat")
    _need(q_pe, torch.bfloat16, (n, H, ROPE_DIM), "q_pe")
    _need(block_table, torch.int32, (block_table.shape[0],), "block_table")
    _need(o_lat, torch.float32, (n, H, KV_LORA_RANK), "o_lat")
    if lse is not None:
        _need(lse, torch.float32, (n, H), "lse")
    scale = DEFAULT_SOFTMAX_SCALE if softmax_scale is None else float(softmax_scale)
    cs = cache.c_struct()
    _check("mla_prefill_absorbed", lib.mla_prefill_absorbed(
        ctypes.byref(cs), _ptr(q_lat), _ptr(q_pe), _ptr(block_table), block_table.shape[0], int(ctx_before), n, H,
        scale, _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(o_lat), _ptr(lse),
        _ptr(dev_err), _stream(stream)))


def mla_lse_merge(o_parts, lse_parts, o_lat, lse=None, stream=None):
    """Merge R per-part results (o_lat, lse) of the same sequences over
    disjoint context parts into the result over their union."""
    R, B, H = o_parts.shape[0], o_parts.shape[1], o_parts.shape[2]
    _need(o_parts, torch.float32, (R, B, H, KV_LORA_RANK), "o_parts")
    _need(lse_parts, torch.float32, (R, B, H), "lse_parts")
    _need(o_lat, torch.float32, (B, H, KV_LORA_RANK), "o_lat")
    if lse is not None:
        _need(lse, torch.float32, (B, H), "lse")
    _check("mla_lse_merge", lib.mla_lse_merge(_ptr(o_parts), _ptr(lse_parts), R, B, H, _ptr(o_lat), _ptr(lse),
                                              _stream(stream)))


# The serving-step calls run a few microseconds on the GPU, so their bindings
# keep to cheap checks and pass addresses as plain integers.  All tensors of a
# call lie on one GPU, ``dev`` (a host tensor's get_device() is -1).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _gpu(t, name):
    """The index of a CUDA tensor's device."""
    if not t.is_cuda:
        raise ValueError("%s: expected a CUDA tensor, got one on %s" % (name, t.device))
    return t.get_device()


def _elsewhere(t, name, dev):
    return ValueError("%s: expected a tensor on cuda:%d, as the call's others, got one on %s" % (name, dev, t.device))


def _rows(t, shape, name, dev):
    """(token stride, head stride) of a bf16 tensor [n, heads, width] whose rows are contiguous."""
    s = t.stride()
    if t.dtype is not torch.bfloat16 or t.shape != shape or s[2] != 1:
        raise ValueError("%s: expected CUDA bfloat16 %s with contiguous rows, got %s %s" % (name, shape, t.dtype,
                                                                                           tuple(t.shape)))
    if t.get_device() != dev:
        raise _elsewhere(t, name, dev)
    return s


def _flat(t, dtype, shape, name, dev):
    """The address of a contiguous tensor."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s: expected contiguous CUDA %s %s, got %s %s" % (name, dtype, shape, t.dtype, tuple(t.shape)))
    if t.get_device() != dev:
        raise _elsewhere(t, name, dev)
    return t.data_ptr()


def _err(t, dev=None):
    """The address of an error word, or None."""
    if t is None:
        return None
    if t.dtype is not torch.int32 or not t.is_cuda:
        raise ValueError("dev_err: expected CUDA int32, got %s on %s" % (t.dtype, t.device))
    if dev is not None and t.get_device() != dev:
        raise _elsewhere(t, "dev_err", dev)
    return t.data_ptr()


def _step(fn, dev, stream, *args):
    """Calls a library function on device ``dev``: on ``stream``, or that device's current one."""
    if dev == _device():
        status = fn(*args, stream.cuda_stream if stream is not None else _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, stream.cuda_stream if stream is not None else _raw_stream(dev))
    if status:
        _check(fn.__name__, status)


def mla_plan_chunks(ctx_lens, new_lens, req, page_table, free_pages, free_range, num_pages, block_table, q_start,
                    seq_lens, positions, token_req, slot, free_head, dev_err=None, stream=None):
    """Block tables, slot map, positions and lengths of a serving step from
    the requests' lengths (int32 CUDA tensors; see include/mla.h).  Takes the
    new pages from ``free_pages[free_range[0]:free_range[1]]``, writes them
    into the persistent ``page_table`` and fills the outputs ``block_table``
    .. ``free_head``."""
    B, n = ctx_lens.shape[0], slot.shape[0]
    rows, max_pages = page_table.shape
    i32, dev = torch.int32, _gpu(ctx_lens, "ctx_lens")
    _step(lib.mla_plan_chunks, dev, stream,
          _flat(ctx_lens, i32, (B,), "ctx_lens", dev), _flat(new_lens, i32, (B,), "new_lens", dev),
          _flat(req, i32, (B,), "req", dev), B,
          _flat(page_table, i32, (rows, max_pages), "page_table", dev), rows, max_pages,
          _flat(free_pages, i32, (free_pages.shape[0],), "free_pages", dev), free_pages.shape[0],
          _flat(free_range, i32, (2,), "free_range", dev), num_pages, n,
          _flat(block_table, i32, (B, max_pages), "block_table", dev), _flat(q_start, i32, (B + 1,), "q_start", dev),
          _flat(seq_lens, i32, (B,), "seq_lens", dev), _flat(positions, i32, (n,), "positions", dev),
          _flat(token_req, i32, (n,), "token_req", dev), _flat(slot, i32, (n,), "slot", dev),
          _flat(free_head, i32, (1,), "free_head", dev),
          _err(dev_err, dev))


def mla_rope(q_pe, k_pe, positions, inv_freq, q_out, k_out, pair_axis=None, interleaved=True, inverse=False,
             amplitude=1.0, stream=None):
    """Rotary positions: q_pe [n, heads, 64] and k_pe [n, 64] (bf16, any token
    and head strides that are multiples of 8; k_pe and k_out may be None) into
    q_out and k_out, which may be the inputs.  positions int32 [n] or [axes,
    n]; inv_freq fp32 [32]; pair_axis: the axis of each of the 32 pairs."""
    n, H, _ = q_pe.shape
    axes = 1 if positions.dim() == 1 else positions.shape[0]
    dev = _gpu(q_pe, "q_pe")
    qs, qos = _rows(q_pe, (n, H, ROPE_DIM), "q_pe", dev), _rows(q_out, (n, H, ROPE_DIM), "q_out", dev)
    if (k_pe is None) != (k_out is None):
        raise ValueError("k_pe and k_out go together")
    kp = ko = None
    ks = kos = (0,)
    if k_pe is not None:
        ks, kos = k_pe.stride(), k_out.stride()
        for t, s in ((k_pe, ks), (k_out, kos)):
            if t.dtype is not torch.bfloat16 or t.shape != (n, ROPE_DIM) or s[1] != 1:
                raise ValueError("k_pe, k_out: expected CUDA bfloat16 %s with contiguous rows, got %s %s" % (
                    (n, ROPE_DIM), t.dtype, tuple(t.shape)))
            if t.get_device() != dev:
                raise _elsewhere(t, "k_pe, k_out", dev)
        kp, ko = k_pe.data_ptr(), k_out.data_ptr()
    if pair_axis is not None:
        pair_axis = bytes(pair_axis)
        if len(pair_axis) != ROPE_DIM // 2:
            raise ValueError("pair_axis: expected %d axes" % (ROPE_DIM // 2))
    _step(lib.mla_rope, dev, stream, q_pe.data_ptr(), qs[0], qs[1], kp, ks[0],
          _flat(positions, torch.int32, (n,) if positions.dim() == 1 else (axes, n), "positions", dev), axes, pair_axis,
          _flat(inv_freq, torch.float32, (ROPE_DIM // 2,), "inv_freq", dev), n, H, 1 if interleaved else 0, 1 if inverse else 0,
          amplitude, q_out.data_ptr(), qos[0], qos[1], ko, kos[0])


def mla_chunk_workspace_bytes(batch, n_tokens, heads, max_new, kv_tokens=0):
    return int(lib.mla_chunk_workspace_bytes(int(batch), int(n_tokens), int(heads), int(max_new), int(kv_tokens)))


def mla_chunk_attention(cache, q_nope, q_pe, w_uk, w_uv, block_table, q_start, seq_lens, workspace, o, max_new,
                        kv_tokens=0, dev_err=None, softmax_scale=None, stream=None):
    """Causal attention of a ragged batch of just-appended tokens over the
    paged cache, from q_nope [n, H, 128] and q_pe [n, H, 64] (bf16, strided)
    to o [n, H, 128] (bf16).  Sequence b's tokens are rows q_start[b] ..
    q_start[b + 1] - 1 (lengths on the device); max_new bounds their number,
    kv_tokens the lengths of the sequences with more than CHUNK_SHORT."""
    n, H, _ = q_nope.shape
    B, max_pages = block_table.shape
    dev = _gpu(q_nope, "q_nope")
    qn, qp = _rows(q_nope, (n, H, QK_NOPE_DIM), "q_nope", dev), _rows(q_pe, (n, H, ROPE_DIM), "q_pe", dev)
    bf16, i32 = torch.bfloat16, torch.int32
    if not workspace.is_contiguous():
        raise ValueError("workspace: expected a contiguous CUDA tensor")
    if workspace.get_device() != dev:
        raise _elsewhere(workspace, "workspace", dev)
    if cache.pool.get_device() != dev:
        raise _elsewhere(cache.pool, "the cache's pool", dev)
    cs = cache.c_struct()
    _step(lib.mla_chunk_attention, dev, stream, ctypes.byref(cs), q_nope.data_ptr(), qn[0], qn[1], q_pe.data_ptr(), qp[0], qp[1],
          _flat(w_uk, bf16, (H, QK_NOPE_DIM, KV_LORA_RANK), "w_uk", dev),
          _flat(w_uv, bf16, (H, KV_LORA_RANK, V_DIM), "w_uv", dev),
          _flat(block_table, i32, (B, max_pages), "block_table", dev), max_pages, _flat(q_start, i32, (B + 1,), "q_start", dev),
          _flat(seq_lens, i32, (B,), "seq_lens", dev), B, n, H, max_new, kv_tokens,
          DEFAULT_SOFTMAX_SCALE if softmax_scale is None else softmax_scale, workspace.data_ptr(),
          workspace.numel() * workspace.element_size(), _flat(o, bf16, (n, H, V_DIM), "o", dev),
          _err(dev_err, dev))


def mla_set_prefill_path(path):
    """Select the prefill implementation for later calls (PREFILL_AUTO,
    PREFILL_DECODE_KERNELS or PREFILL_TENSOR_CORES); returns the previous one."""
    prev = int(lib.mla_set_prefill_path(int(path)))
    if prev < 0:
        raise ValueError("unknown prefill path %r" % (path,))
    return prev


def mla_prefill_path_taken(ctx_before, n, heads):
    """PREFILL_DECODE_KERNELS or PREFILL_TENSOR_CORES: the implementation a
    prefill call with these sizes takes under the current setting."""
    return int(lib.mla_prefill_path_taken(int(ctx_before), int(n), int(heads)))


def mla_set_wait_limit_ns(ns):
    """Bound (ns) on every wait inside the decode kernels launched afterwards;
    returns the previous bound.  A test and diagnostic hook (default 10 s)."""
    prev = int(lib.mla_set_wait_limit_ns(int(ns)))
    if prev < 0:
        raise ValueError("wait limit must be >= 0")
    return prev


def abi_version():
    return int(lib.mla_abi_version())
