"""MI355X-native paged <-> chunk KV-cache movement: Python binding of libkvmove.so.

Argument marshalling only.  Every byte is moved by the HIP kernels behind the
C ABI in ``include/kvmove.h``; this module turns torch device tensors,
streams and events into the raw addresses and handles that ABI takes.  There
is no fallback: if ``libkvmove.so`` is missing the first call raises.

Typical use::

    import paged_kv_movement_amd as kvm
    pool = torch.empty(L, 2, num_pages, 16, H, D, dtype=torch.bfloat16, device="cuda")
    paged = kvm.Paged.from_pool(pool, chunk_size=256)
    chunks = [torch.empty(paged.chunk_bytes(n), dtype=torch.uint8, device="cuda") for n in ...]
    batch = kvm.Batch(paged, [kvm.Seq(block_table, 0, 10000, chunks)])
    kvm.store(paged, batch)                            # gather pages -> chunks
    n = kvm.retrieve(paged, batch, masks=[hit_mask])   # scatter hit chunks -> pages

A model step on the same pool (``Tables``, ``Step``, ``Rope``): ``append``,
``attend``, ``add_weights`` and ``evict``; append takes a ``Norm``, attend a
window, and both a ``Paged8``, the pool in 8 bits that ``pack8`` and ``unpack8``
convert from and to.

Chunk tensors made with ``pin_memory=True`` instead of on the device turn the
same calls into the offload to host memory and the onload from it.
"""
from __future__ import annotations

import ctypes
import os

__all__ = ["FMT_BF16", "FMT_FP8", "FMT_FP8_E5M2", "FMT_K16_V8", "FMT_CACHEGEN", "KvError", "Paged", "Seq", "Batch",
           "store", "store_layer", "store_layers", "store_cachegen", "retrieve_cachegen",
           "retrieve", "retrieve_noalloc", "retrieve_layer", "retrieve_layer_ex", "retrieve_layers", "take_faults",
           "copy_bytes",
           "Tables", "Step", "Rope", "append", "attend", "add_weights", "evict",
           "Paged8", "Norm", "pack8", "unpack8",
           "library_path", "load"]

FMT_BF16 = 0          # K and V bf16, copied bit for bit
FMT_FP8 = 1           # K and V e4m3 + one float32 scale per (layer, K/V)
FMT_FP8_E5M2 = 2      # K and V e5m2 + one float32 scale per (layer, K/V)
FMT_K16_V8 = 3        # K bf16, V e4m3 + one float32 scale per layer
FMT_CACHEGEN = 4      # CacheGen symbols + one float32 max1 per (layer, K/V, token); store_cachegen / retrieve_cachegen

KV_OK, KV_EINVAL, KV_ERANGE, KV_EHIP = 0, -1, -2, -3

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libkvmove.so")
_lib = None


class KvError(RuntimeError):
    """A non-OK status from libkvmove (the message is kv_last_error())."""

    def __init__(self, code: int, msg: str):
        super().__init__(f"kvmove error {code}: {msg}")
        self.code = code


class _KvPaged(ctypes.Structure):
    _fields_ = [
        ("num_layers", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("chunk_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int64),
        ("k_pages", ctypes.c_void_p),
        ("v_pages", ctypes.c_void_p),
    ]


class _KvSeq(ctypes.Structure):
    _fields_ = [
        ("block_table", ctypes.c_void_p),
        ("n_bt", ctypes.c_int64),
        ("tok_start", ctypes.c_int64),
        ("tok_end", ctypes.c_int64),
        ("chunks", ctypes.c_void_p),
    ]


class _KvTables(ctypes.Structure):
    _fields_ = [
        ("n", ctypes.c_int32),
        ("max_len", ctypes.c_int32),
        ("table", ctypes.c_void_p),
        ("stride", ctypes.c_int64),
        ("lens", ctypes.c_void_p),
    ]


class _KvStep(ctypes.Structure):
    _fields_ = [
        ("own", _KvTables),
        ("prefix", _KvTables),
        ("q_start", ctypes.c_void_p),
        ("group_start", ctypes.c_void_p),
        ("n_rows", ctypes.c_int32),
        ("max_new", ctypes.c_int32),
        ("max_group_rows", ctypes.c_int32),
    ]


class _KvRows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class _KvRope(ctypes.Structure):
    _fields_ = [("freqs", ctypes.c_void_p), ("rot", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("gain", ctypes.c_float)]


class _KvPaged8(ctypes.Structure):
    _fields_ = [("pages", _KvPaged), ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p)]


class _KvNorm(ctypes.Structure):
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("q_stride", ctypes.c_int64),
                ("k_stride", ctypes.c_int64), ("eps", ctypes.c_float), ("centered", ctypes.c_int32)]


class _KvWindow(ctypes.Structure):
    _fields_ = [("window", ctypes.c_int32), ("sinks", ctypes.c_int32)]


class _KvSlots(ctypes.Structure):
    _fields_ = [("weights", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("heads", ctypes.c_int32),
                ("cap", ctypes.c_int64)]


class _KvSums(ctypes.Structure):
    _fields_ = [("inp", ctypes.c_void_p), ("out", ctypes.c_void_p), ("cap", ctypes.c_int64)]


def library_path() -> str:
    return _LIB_PATH


def load():
    """Load libkvmove.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise KvError(KV_EHIP, f"{_LIB_PATH} is missing: build it with "
                               "`python -m paged_kv_movement_amd.build` (there is no fallback)")
    L = ctypes.CDLL(_LIB_PATH)
    P, S = ctypes.POINTER(_KvPaged), ctypes.POINTER(_KvSeq)
    T, B, R, O, W, M = (ctypes.POINTER(c) for c in (_KvStep, _KvTables, _KvRows, _KvRope, _KvSlots, _KvSums))
    P8, N, V = (ctypes.POINTER(c) for c in (_KvPaged8, _KvNorm, _KvWindow))
    i32, i64, vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
    sig = {
        "kv_chunk_bytes": (ctypes.c_size_t, [P, i64, ctypes.c_int]),
        "kv_num_chunks": (i64, [P, i64, i64]),
        "kv_chunk_tokens": (i64, [P, i64, i64, i64]),
        "kv_store_chunks": (ctypes.c_int, [P, S, ctypes.c_int, ctypes.c_int, vp]),
        "kv_store_layer": (ctypes.c_int, [P, S, ctypes.c_int, ctypes.c_int, i32, i32, vp, vp]),
        "kv_store_layers": (ctypes.c_int, [P, S, ctypes.c_int, ctypes.c_int, i32, i32, vp, vp, vp, vp, vp]),
        "kv_retrieve_chunks": (ctypes.c_int, [P, S, vp, ctypes.c_int, ctypes.c_int, vp, vp]),
        "kv_retrieve_layer": (ctypes.c_int, [P, S, vp, ctypes.c_int, ctypes.c_int, i32, vp, vp]),
        "kv_retrieve_layer_ex": (ctypes.c_int, [P, S, vp, ctypes.c_int, ctypes.c_int, i32, vp, i32, vp, vp]),
        "kv_retrieve_layers": (ctypes.c_int, [P, S, vp, ctypes.c_int, ctypes.c_int, i32, i32, vp, vp, vp, vp,
                                              vp]),
        "kv_store_chunks_cachegen": (ctypes.c_int, [P, S, ctypes.c_int, vp, vp, vp]),
        "kv_retrieve_workspace_bytes": (ctypes.c_size_t, [P]),
        "kv_store_workspace_bytes": (ctypes.c_size_t, [P, S, ctypes.c_int, ctypes.c_int]),
        "kv_store_chunks_ws": (ctypes.c_int, [P, S, ctypes.c_int, ctypes.c_int, vp, ctypes.c_size_t, vp]),
        "kv_retrieve_chunks_ws": (ctypes.c_int, [P, S, vp, ctypes.c_int, ctypes.c_int, vp, vp, ctypes.c_size_t, vp]),
        "kv_retrieve_chunks_noalloc": (ctypes.c_int, [P, S, vp, ctypes.c_int, ctypes.c_int, vp, vp]),
        "kv_retrieve_chunks_cachegen": (ctypes.c_int, [P, S, vp, ctypes.c_int, vp, vp, vp, vp, ctypes.c_size_t, vp]),
        "kv_append": (ctypes.c_int, [P, T, i32, R, R, R, R, i32, ctypes.c_int, ctypes.c_int, vp, O, W, vp]),
        "kv_attend_workspace_bytes": (ctypes.c_size_t, [P, T, i32]),
        "kv_attend": (ctypes.c_int, [P, T, i32, R, i32, ctypes.c_float, R, vp, vp, ctypes.c_size_t, vp]),
        "kv_add_weights": (ctypes.c_int, [P, T, i32, R, vp, i32, ctypes.c_float, M, M, vp]),
        "kv_evict_workspace_bytes": (ctypes.c_size_t, [P, B, i32, i32, i32]),
        "kv_evict": (ctypes.c_int, [P, B, i32, i32, W, W, i32, i32, vp, vp, ctypes.c_size_t, vp]),
        "kv_append_normed": (ctypes.c_int, [P, T, i32, R, R, R, R, i32, ctypes.c_int, ctypes.c_int, vp, O, N, W, vp]),
        "kv_append8": (ctypes.c_int, [P8, T, i32, R, R, R, R, i32, ctypes.c_int, ctypes.c_int, vp, O, N, vp]),
        "kv_attend_window_workspace_bytes": (ctypes.c_size_t, [P, T, i32, V]),
        "kv_attend_window": (ctypes.c_int, [P, T, i32, R, i32, ctypes.c_float, V, R, vp, vp, ctypes.c_size_t, vp]),
        "kv_attend8_workspace_bytes": (ctypes.c_size_t, [P8, T, i32, V]),
        "kv_attend8": (ctypes.c_int, [P8, T, i32, R, i32, ctypes.c_float, V, R, vp, vp, ctypes.c_size_t, vp]),
        "kv_pack8": (ctypes.c_int, [P, B, P8, vp, i64, i32, i32, vp]),
        "kv_unpack8": (ctypes.c_int, [P8, B, P, vp, i64, i32, i32, vp]),
        "kv_last_error": (ctypes.c_char_p, []),
        "kv_take_faults": (ctypes.c_int, []),
        "kv_copy_bytes": (ctypes.c_int, [vp, vp, ctypes.c_size_t, vp]),
        "kv_copy_blocks": (ctypes.c_int, [vp, vp, ctypes.c_size_t, ctypes.c_size_t, ctypes.c_int, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def _check(rc: int):
    if rc != KV_OK:
        raise KvError(rc, load().kv_last_error().decode())


def _need(cond, msg: str):
    """Argument check that stays on under ``python -O``."""
    if not cond:
        raise KvError(KV_EINVAL, msg)


def _stream_handle(stream) -> int | None:
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    h = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    return h or None


def _used_on(stream, tensors, seen=None) -> None:
    """Tell torch's caching allocator that kernels on ``stream`` read these
    tensors (``record_stream``): the binding makes some device tensors itself
    (address arrays) on the current stream, and a caller may pass a workspace
    made inline; without this, freeing them while the side stream still runs
    could hand their memory to new work too early.  With ``seen`` (a set kept
    by the owner of the tensors, which keeps them alive) each (tensor, stream)
    is recorded once.  Nothing is done for stream=None (the current stream,
    see _used_on_current) or a raw stream handle (the caller then keeps the
    tensors alive)."""
    if stream is None or not hasattr(stream, "cuda_stream"):
        return
    for t in tensors:
        if t is None or not getattr(t, "is_cuda", False):
            continue
        if seen is None:
            t.record_stream(stream)
            continue
        key = (id(t), stream.cuda_stream)
        if key not in seen:
            t.record_stream(stream)
            seen.add(key)


def _used_on_current(tensors, seen) -> None:
    """_used_on for the current stream, of device tensors that the binding made
    and the caller does not see: made on one stream and used under
    ``torch.cuda.stream`` of another, they may be dropped before the kernels
    have run.  Once per stream (its handle goes into ``seen``)."""
    if not getattr(tensors[0], "is_cuda", False):
        return
    dev = tensors[0].get_device()
    h = _t()._C._cuda_getCurrentRawStream(dev)
    if h not in seen:
        _used_on(_t().cuda.current_stream(dev), tensors, seen)
        seen.add(h)


class Paged:
    """The engine's paged pool: per-layer K and V base addresses on the device.

    ``k_addrs`` / ``v_addrs`` are device int64 tensors [num_layers] holding the
    address of each layer's bf16 [num_pages][page_size][H][D] K / V pool.
    """

    def __init__(self, k_addrs, v_addrs, num_layers, num_kv_heads, head_dim, page_size,
                 chunk_size, num_pages, keepalive=()):
        self.k_addrs, self.v_addrs = k_addrs, v_addrs
        self._keep = tuple(keepalive)
        self.num_layers, self.num_kv_heads, self.head_dim = num_layers, num_kv_heads, head_dim
        self.page_size, self.chunk_size, self.num_pages = page_size, chunk_size, num_pages
        self.c = _KvPaged(num_layers, num_kv_heads, head_dim, page_size, chunk_size, num_pages,
                          k_addrs.data_ptr(), v_addrs.data_ptr())
        self._arrays = (k_addrs, v_addrs)
        self._on_streams = set()        # streams that calls without a Batch or Step of their own were made on

    @classmethod
    def from_pool(cls, pool, chunk_size: int = 256) -> "Paged":
        """From one bf16 tensor [L, 2, num_pages, page_size, H, D] (K at [:, 0], V at [:, 1])."""
        import torch
        _need(pool.dtype == torch.bfloat16 and pool.is_contiguous() and pool.dim() == 6 and pool.is_cuda,
              "pool must be a contiguous bf16 device tensor [L, 2, num_pages, page_size, H, D]")
        L, two, n, P, H, D = pool.shape
        _need(two == 2, "pool's second dimension must be 2 (K, V)")
        slab = n * P * H * D * pool.element_size()
        base = pool.data_ptr()
        k = torch.tensor([base + (2 * l) * slab for l in range(L)], dtype=torch.int64)
        v = torch.tensor([base + (2 * l + 1) * slab for l in range(L)], dtype=torch.int64)
        return cls(k.to(pool.device), v.to(pool.device), L, H, D, P, chunk_size, n, keepalive=(pool,))

    @classmethod
    def from_layers(cls, k_layers, v_layers, chunk_size: int = 256) -> "Paged":
        """From per-layer bf16 tensors, each [num_pages, page_size, H, D]."""
        import torch
        n, P, H, D = k_layers[0].shape
        _need(len(k_layers) == len(v_layers) > 0, "need one K and one V tensor per layer")
        for t in list(k_layers) + list(v_layers):
            _need(t.dtype == torch.bfloat16 and t.is_contiguous() and t.is_cuda and tuple(t.shape) == (n, P, H, D),
                  "per-layer pools must be contiguous bf16 device tensors of one shape [num_pages, page_size, H, D]")
        dev = k_layers[0].device
        k = torch.tensor([t.data_ptr() for t in k_layers], dtype=torch.int64).to(dev)
        v = torch.tensor([t.data_ptr() for t in v_layers], dtype=torch.int64).to(dev)
        return cls(k, v, len(k_layers), H, D, P, chunk_size, n, keepalive=(*k_layers, *v_layers))

    def chunk_bytes(self, n_tokens: int, fmt: int = FMT_BF16) -> int:
        n = load().kv_chunk_bytes(ctypes.byref(self.c), n_tokens, fmt)
        if n == 0 and n_tokens > 0:
            _check(KV_EINVAL)
        return int(n)

    def retrieve_workspace_bytes(self) -> int:
        """Device bytes retrieve(..., workspace=...) needs for this pool."""
        n = load().kv_retrieve_workspace_bytes(ctypes.byref(self.c))
        if n == 0:
            _check(KV_EINVAL)
        return int(n)

    def new_workspace(self):
        """A device tensor of retrieve_workspace_bytes() bytes (torch aligns it to 256)."""
        import torch
        return torch.empty(self.retrieve_workspace_bytes(), dtype=torch.uint8, device="cuda")

    def num_chunks(self, tok_start: int, tok_end: int) -> int:
        n = load().kv_num_chunks(ctypes.byref(self.c), tok_start, tok_end)
        if n < 0:
            _check(KV_EINVAL)
        return int(n)

    def chunk_tokens(self, tok_start: int, tok_end: int, c: int) -> int:
        """Tokens of chunk c of [tok_start, tok_end) (kv_chunk_tokens)."""
        n = load().kv_chunk_tokens(ctypes.byref(self.c), tok_start, tok_end, c)
        if n < 0:
            _check(KV_EINVAL)
        return int(n)


def _addresses(tensors):
    """Their addresses, as a device int64 tensor."""
    import torch
    return torch.tensor([t.data_ptr() for t in tensors], dtype=torch.int64).to(tensors[0].device)


class Paged8:
    """A paged pool in 8 bits: e4m3 bytes, and for each block (one head's tokens
    in one page) of K and of V a float32 scale, the least power of two of which
    448 reach every value of the block.  A byte stands for byte * scale.

    append, attend, pack8 and unpack8 take it; the chunk movers, add_weights
    and evict work on the bf16 pool (unpack8 and store, retrieve and pack8)."""

    def __init__(self, k_layers, v_layers, k_scales, v_scales):
        import torch
        _need(len(k_layers) == len(v_layers) == len(k_scales) == len(v_scales) > 0,
              "need one K and one V tensor per layer, and their scales")
        _need(k_layers[0].dim() == 4, "per-layer pools must be [num_pages, page_size, H, D]")
        n, P, H, D = k_layers[0].shape
        for t in (*k_layers, *v_layers):
            _need(t.dtype in (torch.uint8, torch.float8_e4m3fn) and t.is_contiguous() and t.is_cuda
                  and tuple(t.shape) == (n, P, H, D),
                  "per-layer pools must be contiguous uint8 or float8_e4m3fn device tensors of one shape "
                  "[num_pages, page_size, H, D]")
        for t in (*k_scales, *v_scales):
            _need(t.dtype == torch.float32 and t.is_contiguous() and t.is_cuda and tuple(t.shape) == (n, H),
                  "scales must be contiguous float32 device tensors [num_pages, H]")
        dev = k_layers[0].device
        _need(all(t.device == dev for t in (*k_layers, *v_layers, *k_scales, *v_scales)),
              "a pool's tensors must be on one device")
        _need(D % 16 == 0, "head_dim must be a multiple of 16 in an 8-bit pool")
        # a view of bytes can begin anywhere; the kernels move 16 at a time
        _need(all(t.data_ptr() % 16 == 0 for t in (*k_layers, *v_layers)) and
              all(t.data_ptr() % 4 == 0 for t in (*k_scales, *v_scales)),
              "per-layer pools must begin at multiples of 16 bytes, scales of 4")
        self._keep = (*k_layers, *v_layers, *k_scales, *v_scales)
        self.num_layers, self.num_kv_heads, self.head_dim = len(k_layers), H, D
        self.page_size, self.num_pages = P, n
        self.k_addrs, self.v_addrs = _addresses(k_layers), _addresses(v_layers)
        self.k_scale_addrs, self.v_scale_addrs = _addresses(k_scales), _addresses(v_scales)
        self._arrays = (self.k_addrs, self.v_addrs, self.k_scale_addrs, self.v_scale_addrs)
        self._on_streams = set()
        self.c = _KvPaged8(_KvPaged(self.num_layers, H, D, P, P, n, self.k_addrs.data_ptr(), self.v_addrs.data_ptr()),
                           self.k_scale_addrs.data_ptr(), self.v_scale_addrs.data_ptr())

    @classmethod
    def from_pool(cls, pool, scales) -> "Paged8":
        """From one tensor [L, 2, num_pages, page_size, H, D] (uint8 or float8_e4m3fn; K at [:, 0], V at [:, 1])
        and its float32 scales [L, 2, num_pages, H]."""
        _need(pool.dim() == 6 and pool.size(1) == 2 and scales.dim() == 4 and scales.shape[:3] == pool.shape[:3],
              "need a pool [L, 2, num_pages, page_size, H, D] and scales [L, 2, num_pages, H]")
        return cls(pool[:, 0].unbind(0), pool[:, 1].unbind(0), scales[:, 0].unbind(0), scales[:, 1].unbind(0))


def _bf16_pool(paged, call: str) -> None:
    if isinstance(paged, Paged8):
        raise KvError(KV_EINVAL, f"{call} works on a bf16 pool, not on a Paged8")


class Seq:
    """One sequence's job: a device int32 block table, a token range and its
    chunk buffers (device int64 tensor of addresses, or uint8 tensors).

    A chunk tensor lives either in device memory or in pinned host memory
    (``pin_memory=True``): the kernels address pinned host memory directly,
    so a store into host chunks is the offload and a retrieve from them the
    onload, both over PCIe with no staging copy.  Pageable host tensors are
    refused, since the GPU cannot reach them."""

    def __init__(self, block_table, tok_start: int, tok_end: int, chunks):
        import torch
        self.block_table = block_table
        self.tok_start, self.tok_end = int(tok_start), int(tok_end)
        if isinstance(chunks, torch.Tensor) and chunks.dtype == torch.int64:
            _need(chunks.is_cuda and chunks.is_contiguous() and chunks.dim() == 1,
                  "chunk addresses must be a contiguous 1-D int64 device tensor")
            self.chunk_addrs, self._chunks = chunks, None
        else:
            self._chunks = list(chunks)
            for i, c in enumerate(self._chunks):
                if not c.is_contiguous():
                    raise KvError(KV_EINVAL, f"chunk {i} is not contiguous")
                if not (c.is_cuda or c.is_pinned()):
                    raise KvError(KV_EINVAL, f"chunk {i} is pageable host memory; "
                                             "use a device tensor or pin_memory=True")
            addrs = torch.tensor([c.data_ptr() for c in self._chunks], dtype=torch.int64)
            dev = block_table.device if isinstance(block_table, torch.Tensor) else "cuda"
            self.chunk_addrs = addrs.to(dev)
        # the kernels read the block table from device memory
        _need(isinstance(block_table, torch.Tensor) and block_table.dtype == torch.int32
              and block_table.is_contiguous() and block_table.is_cuda,
              "block_table must be a contiguous int32 device tensor")

    def c(self) -> _KvSeq:
        return _KvSeq(self.block_table.data_ptr(), self.block_table.numel(), self.tok_start,
                      self.tok_end, self.chunk_addrs.data_ptr() if self.chunk_addrs.numel() else 0)


class Batch:
    """Prebuilt C descriptors for a list of Seq (reusable across calls)."""

    def __init__(self, paged: Paged, seqs):
        _bf16_pool(paged, "a Batch")
        self.seqs = list(seqs)
        self.paged = paged
        n = len(self.seqs)
        self.arr = (_KvSeq * max(1, n))(*[s.c() for s in self.seqs])
        self.n = n
        self._mask_bufs = None
        self._mask_ptrs = None
        self.out = (ctypes.c_int64 * max(1, n))()
        self._checked_fmts = set()      # formats whose chunk tensors were sized against the library
        self._on_streams = set()        # (tensor, stream) pairs already given to record_stream
        # device tensors the kernels read besides the caller's own
        self._dev_tensors = [paged.k_addrs, paged.v_addrs] + [s.chunk_addrs for s in self.seqs]

    def set_masks(self, masks):
        """Host hit masks, one uint8 flag per chunk per sequence."""
        _need(len(masks) == self.n, f"need {self.n} hit masks, got {len(masks)}")
        bufs = []
        for i, (sq, m) in enumerate(zip(self.seqs, masks)):
            b = bytes(int(x) & 0xFF for x in (m.tolist() if hasattr(m, "tolist") else m))
            # the library reads one flag for every chunk of the sequence
            n_chunks = self.paged.num_chunks(sq.tok_start, sq.tok_end)
            _need(len(b) >= n_chunks, f"sequence {i}: hit mask has {len(b)} flags for {n_chunks} chunks")
            bufs.append(ctypes.create_string_buffer(b, max(1, len(b))))
        self._mask_bufs = bufs
        self._mask_ptrs = (ctypes.c_void_p * max(1, self.n))(
            *[ctypes.cast(b, ctypes.c_void_p).value for b in bufs])
        return self

    def check_chunks(self, fmt: int) -> "Batch":
        """For sequences whose chunks were given as tensors: one tensor per
        chunk of the range, each at least kv_chunk_bytes(tokens of the chunk,
        fmt) bytes, sizes from the library (kv_num_chunks, kv_chunk_tokens,
        kv_chunk_bytes).  The kernels write every chunk buffer up to that size
        and cannot see a buffer's end, so a short list or a small tensor is
        refused here, before anything runs.  Chunks given as an address
        tensor cannot be checked.  Done once per format."""
        if fmt in self._checked_fmts:
            return self
        p = self.paged
        for i, sq in enumerate(self.seqs):
            if sq._chunks is None:
                continue
            n = p.num_chunks(sq.tok_start, sq.tok_end)
            _need(len(sq._chunks) >= n, f"sequence {i}: {len(sq._chunks)} chunk tensors for {n} chunks")
            for c in range(n):
                need = p.chunk_bytes(p.chunk_tokens(sq.tok_start, sq.tok_end, c), fmt)
                have = sq._chunks[c].numel() * sq._chunks[c].element_size()
                _need(have >= need, f"sequence {i}, chunk {c}: {have} bytes, format {fmt} needs {need}")
        self._checked_fmts.add(fmt)
        return self

    def store_workspace_bytes(self, fmt: int = FMT_BF16) -> int:
        """Device bytes store(..., workspace=...) needs for these sequences
        in this format (kv_store_workspace_bytes; 0 for the fp8 formats)."""
        n = load().kv_store_workspace_bytes(ctypes.byref(self.paged.c), self.arr, self.n, fmt)
        if n == 0:
            _check(KV_OK if load().kv_last_error() == b"" else KV_EINVAL)
        return int(n)

    def new_store_workspace(self, fmt: int = FMT_BF16):
        """A device tensor of store_workspace_bytes(fmt) bytes (torch aligns it
        to 256), or None when the format needs none."""
        import torch
        n = self.store_workspace_bytes(fmt)
        return torch.empty(n, dtype=torch.uint8, device="cuda") if n > 0 else None

    def used_on(self, stream, *extra) -> None:
        """record_stream for the Batch's own device tensors (once per stream)
        and for ``extra`` tensors of this call (every time)."""
        _used_on(stream, self._dev_tensors, self._on_streams)
        _used_on(stream, extra)


def _batch(paged, seqs, fmt, stream, *extra) -> Batch:
    """The Batch for a call: chunk tensors sized for fmt, and the device
    tensors the call reads marked as used on stream."""
    b = seqs if isinstance(seqs, Batch) else Batch(paged, seqs)
    b.check_chunks(fmt)
    if stream is None:
        _used_on_current(b._dev_tensors, b._on_streams)
    else:
        b.used_on(stream, *extra)
    return b


def store(paged: Paged, seqs, fmt: int = FMT_BF16, stream=None, workspace=None) -> None:
    """Gather every chunk of every sequence (kv_store_chunks).  With
    ``workspace`` (a device uint8 tensor of at least
    batch.store_workspace_bytes(fmt)) the bf16 gather runs through an address
    plan (kv_store_chunks_ws)."""
    b = _batch(paged, seqs, fmt, stream, workspace)
    if workspace is None:
        _check(load().kv_store_chunks(ctypes.byref(paged.c), b.arr, b.n, fmt, _stream_handle(stream)))
    else:
        ws_ptr, ws_bytes = _workspace(workspace)
        _check(load().kv_store_chunks_ws(ctypes.byref(paged.c), b.arr, b.n, fmt, ws_ptr, ws_bytes,
                                         _stream_handle(stream)))


def _event_handle(event, stream):
    if event is None:
        return None
    if not event.cuda_event:        # torch creates the event lazily on first record
        import torch
        event.record(stream if stream is not None else torch.cuda.current_stream())
    return event.cuda_event


def store_layer(paged: Paged, seqs, layer: int, fmt: int = FMT_BF16, stream=None, event=None,
                max_workgroups: int = 0) -> None:
    """Gather one layer of every chunk on ``stream``, then record ``event``
    (a torch.cuda.Event) on it (kv_store_layer)."""
    b = _batch(paged, seqs, fmt, stream)
    _check(load().kv_store_layer(ctypes.byref(paged.c), b.arr, b.n, fmt, layer, max_workgroups,
                                 _stream_handle(stream), _event_handle(event, stream)))


def _alt_handle(alt_stream) -> int | None:
    """Handle of a layer-range call's second stream (None: none)."""
    if alt_stream is None:
        return None
    h = alt_stream.cuda_stream if hasattr(alt_stream, "cuda_stream") else int(alt_stream)
    _need(h != 0, "alt_stream must be a stream of its own, not the null stream")
    return h


def _layer_arrays(n, max_workgroups, events, stream):
    """Host arrays of a layer-range call: caps (or None) and event handles (or None)."""
    caps = None
    if max_workgroups is not None:
        caps = [int(m) for m in max_workgroups]
        _need(len(caps) == n, f"need {n} workgroup caps, got {len(caps)}")
        caps = (ctypes.c_int32 * n)(*caps)
    evs = None
    if events is not None:
        _need(len(events) == n, f"need {n} events, got {len(events)}")
        evs = (ctypes.c_void_p * n)(*[_event_handle(e, stream) for e in events])
    return caps, evs


def store_layers(paged: Paged, seqs, layer_begin: int, layer_end: int, fmt: int = FMT_BF16, stream=None,
                 wait_events=None, events=None, max_workgroups=None, alt_stream=None) -> None:
    """Gather layers [layer_begin, layer_end) on ``stream`` in one call
    (kv_store_layers): before layer l, wait for ``wait_events[l - layer_begin]``
    (torch.cuda.Event, already recorded by the producer); after it, record
    ``events[l - layer_begin]``.  ``max_workgroups``: one cap per layer.
    ``alt_stream``: a second torch stream that takes every other layer, so
    consecutive layers' kernels may overlap."""
    b = _batch(paged, seqs, fmt, stream)
    b.used_on(alt_stream)
    n = layer_end - layer_begin
    caps, evs = _layer_arrays(n, max_workgroups, events, stream)
    waits = None
    if wait_events is not None:
        _need(len(wait_events) == n, f"need {n} wait events, got {len(wait_events)}")
        _need(all(e.cuda_event for e in wait_events), "wait events must have been recorded")
        waits = (ctypes.c_void_p * n)(*[e.cuda_event for e in wait_events])
    _check(load().kv_store_layers(ctypes.byref(paged.c), b.arr, b.n, fmt, layer_begin, layer_end, caps,
                                  _stream_handle(stream), _alt_handle(alt_stream), waits, evs))


def _workspace(workspace):
    """(address, bytes) of a workspace tensor, or (None, 0)."""
    if workspace is None:
        return None, 0
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise KvError(KV_EINVAL, "workspace must be a contiguous device tensor")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _bins(bins, n):
    """One bin count per layer as a host int32 array."""
    bins = [int(b) for b in bins]
    if len(bins) != n:
        raise KvError(KV_EINVAL, f"need {n} bin counts, got {len(bins)}")
    return (ctypes.c_int32 * max(1, n))(*bins)


def store_cachegen(paged: Paged, seqs, key_bins, value_bins, stream=None) -> None:
    """CacheGen quantiser: gather + quantise every chunk (kv_store_chunks_cachegen).
    key_bins / value_bins: one bin count per layer, each in [4, 129]."""
    b = _batch(paged, seqs, FMT_CACHEGEN, stream)
    L = paged.c.num_layers
    _check(load().kv_store_chunks_cachegen(ctypes.byref(paged.c), b.arr, b.n, _bins(key_bins, L),
                                           _bins(value_bins, L), _stream_handle(stream)))


def retrieve_cachegen(paged: Paged, seqs, key_bins, value_bins, masks=None, stream=None, workspace=None) -> list:
    """Dequantise + scatter the leading hit chunks (kv_retrieve_chunks_cachegen);
    in pool-address order when a ``workspace`` (as for retrieve) is given.
    Returns the tokens made available per sequence."""
    b = _batch(paged, seqs, FMT_CACHEGEN, stream, workspace)
    if masks is not None:
        b.set_masks(masks)
    _need(b._mask_ptrs is not None, "hit masks are required")
    L = paged.c.num_layers
    ws_ptr, ws_bytes = _workspace(workspace)
    _check(load().kv_retrieve_chunks_cachegen(ctypes.byref(paged.c), b.arr, b._mask_ptrs, b.n,
                                              _bins(key_bins, L), _bins(value_bins, L), b.out,
                                              ws_ptr, ws_bytes, _stream_handle(stream)))
    return [int(b.out[i]) for i in range(b.n)]


def retrieve(paged: Paged, seqs, masks=None, fmt: int = FMT_BF16, stream=None, workspace=None) -> list:
    """Scatter the leading hit chunks back into pages (kv_retrieve_chunks).
    With ``workspace`` (a device uint8 tensor of at least
    paged.retrieve_workspace_bytes()) the bf16 scatter runs in pool-address
    order (kv_retrieve_chunks_ws).  Returns the tokens made available per
    sequence."""
    b = _batch(paged, seqs, fmt, stream, workspace)
    if masks is not None:
        b.set_masks(masks)
    _need(b._mask_ptrs is not None, "hit masks are required")
    if workspace is None:
        _check(load().kv_retrieve_chunks(ctypes.byref(paged.c), b.arr, b._mask_ptrs, b.n, fmt, b.out,
                                         _stream_handle(stream)))
    else:
        ws_ptr, ws_bytes = _workspace(workspace)
        _check(load().kv_retrieve_chunks_ws(ctypes.byref(paged.c), b.arr, b._mask_ptrs, b.n, fmt, b.out,
                                            ws_ptr, ws_bytes, _stream_handle(stream)))
    return [int(b.out[i]) for i in range(b.n)]


def retrieve_noalloc(paged: Paged, seqs, masks=None, fmt: int = FMT_BF16, stream=None) -> list:
    """retrieve in pool-address order with the library's own scratch array
    instead of a caller's workspace (kv_retrieve_chunks_noalloc): no device
    allocation anywhere in the call.  Calls that overlap on one GPU race.
    Returns the tokens made available per sequence."""
    b = _masked(paged, seqs, masks, fmt, stream)
    _check(load().kv_retrieve_chunks_noalloc(ctypes.byref(paged.c), b.arr, b._mask_ptrs, b.n, fmt, b.out,
                                             _stream_handle(stream)))
    return [int(b.out[i]) for i in range(b.n)]


def _masked(paged, seqs, masks, fmt, stream) -> Batch:
    b = _batch(paged, seqs, fmt, stream)
    if masks is not None:
        b.set_masks(masks)
    _need(b._mask_ptrs is not None, "hit masks are required")
    return b


def retrieve_layer(paged: Paged, seqs, layer: int, masks=None, fmt: int = FMT_BF16, stream=None,
                   event=None) -> None:
    """Scatter one layer of the leading hit chunks on ``stream``, then record
    ``event`` (a torch.cuda.Event) on it (kv_retrieve_layer)."""
    b = _masked(paged, seqs, masks, fmt, stream)
    _check(load().kv_retrieve_layer(ctypes.byref(paged.c), b.arr, b._mask_ptrs, b.n, fmt, layer,
                                    _stream_handle(stream), _event_handle(event, stream)))


def retrieve_layer_ex(paged: Paged, seqs, layer: int, masks=None, fmt: int = FMT_BF16, stream=None,
                      event=None, max_workgroups: int = 0) -> list:
    """retrieve_layer with a workgroup cap (kv_retrieve_layer_ex): a positive
    ``max_workgroups`` caps the grid so compute on another stream keeps most
    of the GPU.  Returns the tokens made available per sequence."""
    b = _masked(paged, seqs, masks, fmt, stream)
    _check(load().kv_retrieve_layer_ex(ctypes.byref(paged.c), b.arr, b._mask_ptrs, b.n, fmt, layer,
                                       b.out, max_workgroups, _stream_handle(stream),
                                       _event_handle(event, stream)))
    return [int(b.out[i]) for i in range(b.n)]


def retrieve_layers(paged: Paged, seqs, layer_begin: int, layer_end: int, masks=None, fmt: int = FMT_BF16,
                    stream=None, events=None, max_workgroups=None, alt_stream=None) -> list:
    """Scatter layers [layer_begin, layer_end) of the leading hit chunks on
    ``stream`` in one call, recording ``events[l - layer_begin]`` after layer
    l (kv_retrieve_layers).  ``max_workgroups``: one cap per layer, or None.
    ``alt_stream``: a second torch stream that takes every other layer, so
    consecutive layers' kernels may overlap.  Returns the tokens made
    available per sequence."""
    b = _masked(paged, seqs, masks, fmt, stream)
    b.used_on(alt_stream)
    caps, evs = _layer_arrays(layer_end - layer_begin, max_workgroups, events, stream)
    _check(load().kv_retrieve_layers(ctypes.byref(paged.c), b.arr, b._mask_ptrs, b.n, fmt, layer_begin,
                                     layer_end, caps, b.out, _stream_handle(stream), _alt_handle(alt_stream), evs))
    return [int(b.out[i]) for i in range(b.n)]


def take_faults() -> int:
    """Synchronise the device; return and clear the kernels' fault bits."""
    rc = load().kv_take_faults()
    if rc < 0:
        _check(rc)
    return rc


def copy_bytes(dst, src, nbytes: int, stream=None) -> None:
    """Plain contiguous device copy (measurement aid)."""
    _check(load().kv_copy_bytes(dst.data_ptr(), src.data_ptr(), nbytes, _stream_handle(stream)))


COPY_SCATTERED_READS, COPY_SCATTERED_WRITES = 1, 2


def copy_blocks(dst, src, nbytes: int, block_bytes: int, permute: int, stream=None) -> None:
    """Device copy with one side visited in scattered blocks (measurement aid,
    kv_copy_blocks): permute = COPY_SCATTERED_READS or COPY_SCATTERED_WRITES."""
    _check(load().kv_copy_blocks(dst.data_ptr(), src.data_ptr(), nbytes, block_bytes, permute,
                                 _stream_handle(stream)))


# ---- a model step on the paged pool: append, attend, add_weights, evict

_torch = None


def _t():
    """torch, imported on the first use and kept: a step's calls are made every few microseconds."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _int32(what: str, *numbers) -> None:
    """Refuse what a C int32 does not hold: ctypes would pass its low bits.
    The calls of a step ask only where a number has bits past the 31st."""
    for x in numbers:
        if not -0x80000000 <= x <= 0x7FFFFFFF:
            raise KvError(KV_EINVAL, f"{what} = {x} does not fit 32 bits")


def _here(*tensors) -> int:
    """The current device; every tensor must be on it (the calls launch there)."""
    cur = _t().cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != cur:
            raise KvError(KV_EINVAL, f"every tensor must be on the current device (cuda:{cur}), got {t.device}")
    return cur


def _ref(struct):
    return None if struct is None else ctypes.byref(struct)


class Tables:
    """Block tables and lengths of a batch, both on the device.

    ``table``: int32 [n, entries], page ids of each sequence in token order (the
    last dimension contiguous); ``lens``: int32 [n], tokens cached, read when
    a call's kernels run; ``max_len``: the host's bound of them, which sizes
    the launches (a longer length is cut to it)."""

    def __init__(self, table, lens, max_len: int):
        import torch
        _need(table.dtype == torch.int32 and table.dim() == 2 and table.is_cuda
              and (table.stride(1) == 1 or table.size(1) <= 1),
              "table must be an int32 device tensor [sequences, entries], entries contiguous")
        _need(lens.dtype == torch.int32 and lens.is_contiguous() and lens.is_cuda
              and tuple(lens.shape) == (table.size(0),), "lens must be a contiguous int32 device tensor [sequences]")
        _need(0 <= max_len <= 1 << 30, "max_len must be in [0, 2^30]")
        self.table, self.lens, self.max_len, self.n = table, lens, int(max_len), table.size(0)
        # rows further apart than their entries (a view) are reached through the stride
        _need(table.size(0) <= 1 or table.stride(0) >= table.size(1), "table's rows must not overlap")
        self._entries = table.size(1)
        self.c = _KvTables(self.n, self.max_len, table.data_ptr(), table.stride(0) if self.n > 1 else table.size(1),
                           lens.data_ptr())

    def _check(self, paged: Paged) -> None:
        if self.max_len > self._entries * paged.page_size:
            raise KvError(KV_ERANGE, f"max_len {self.max_len} beyond the block table "
                                     f"({self._entries} pages of {paged.page_size})")

    def evict_workspace_bytes(self, paged: Paged, n_layers: int, heads: int, keep: int) -> int:
        """Device bytes evict needs (kv_evict_workspace_bytes)."""
        _int32("n_layers, heads or keep", n_layers, heads, keep)
        n = load().kv_evict_workspace_bytes(ctypes.byref(paged.c), ctypes.byref(self.c), n_layers, heads, keep)
        if n == 0:
            _check(KV_EINVAL)
        return int(n)

    def new_evict_workspace(self, paged: Paged, n_layers: int, heads: int, keep: int):
        """A device tensor of evict_workspace_bytes (torch aligns it to 256)."""
        import torch
        return torch.empty(self.evict_workspace_bytes(paged, n_layers, heads, keep), dtype=torch.uint8,
                           device=self.table.device)


class Step:
    """One step of a batch: which rows of q, k and v are whose new tokens, and
    which sequences share a prefix.

    ``own``: Tables of the sequences' own pages, lengths with the new tokens
    counted; ``new_tokens``: the new tokens of each sequence; ``prefix``:
    Tables of the shared prefixes, one row per group; ``group_sizes``: the
    sequences of each group, in order (sequences left over share nothing).
    The tables' contents and lengths may change between calls; a Step keeps
    no result.  A graph that captured calls reads the Step's, the Rope's and
    the Paged's own arrays: keep the three for as long as it is replayed."""

    def __init__(self, paged: Paged, own: Tables, new_tokens, prefix: Tables | None = None, group_sizes=None):
        import torch
        new = [int(x) for x in new_tokens]
        sizes = [int(x) for x in (group_sizes or [])]
        _need(len(new) == own.n and all(x >= 0 for x in new), f"need {own.n} counts of new tokens, none negative")
        _need(len(sizes) == (0 if prefix is None else prefix.n) and all(x >= 0 for x in sizes),
              "need one group size per row of prefix, none negative")
        _need(sum(sizes) <= own.n, "the groups hold more sequences than there are")
        own._check(paged)
        if prefix is not None:
            prefix._check(paged)
        starts, groups = [0], [0]
        for x in new:
            starts.append(starts[-1] + x)
        for x in sizes:
            groups.append(groups[-1] + x)
        _need(starts[-1] < 1 << 31, "too many rows")
        dev = own.table.device
        self.own, self.prefix, self.n_rows = own, prefix, starts[-1]
        self.q_start = torch.tensor(starts, dtype=torch.int32).to(dev)
        self.group_start = torch.tensor(groups, dtype=torch.int32).to(dev)
        self.paged = paged
        self.c = _KvStep(own.c, prefix.c if prefix is not None else _KvTables(), self.q_start.data_ptr(),
                         self.group_start.data_ptr(), self.n_rows, max(new, default=0),
                         max((starts[groups[i + 1]] - starts[groups[i]] for i in range(len(sizes))), default=0))
        self._tensors = [*paged._arrays, own.table, own.lens, self.q_start, self.group_start]
        if prefix is not None:
            self._tensors += [prefix.table, prefix.lens]
        self._on_streams = set()
        self._dim = paged.head_dim
        self._device = _here(*self._tensors)
        self._ref = ctypes.byref(self.c)

    def attend_workspace_bytes(self, q_heads: int, window: int | None = None, sinks: int = 0,
                               paged: Paged | Paged8 | None = None) -> int:
        """Device bytes attend needs with this window over ``paged`` (None: the
        step's own pool); kv_attend_workspace_bytes and its other forms.  An
        8-bit pool can need more than a bf16 one, and a window more than
        another or none: a workspace for several calls has to be as large as
        the largest of theirs."""
        _int32("q_heads", q_heads)
        paged = self.paged if paged is None else paged
        w, p, c = _window(window, sinks), ctypes.byref(paged.c), ctypes.byref(self.c)
        if isinstance(paged, Paged8):
            n = load().kv_attend8_workspace_bytes(p, c, q_heads, _ref(w))
        elif w is not None:
            n = load().kv_attend_window_workspace_bytes(p, c, q_heads, _ref(w))
        else:
            n = load().kv_attend_workspace_bytes(p, c, q_heads)
        if n == 0:
            _check(KV_EINVAL)
        return int(n)

    def new_attend_workspace(self, q_heads: int, window: int | None = None, sinks: int = 0,
                             paged: Paged | Paged8 | None = None):
        """A device tensor of attend_workspace_bytes (torch aligns it to 256)."""
        import torch
        return torch.empty(self.attend_workspace_bytes(q_heads, window, sinks, paged), dtype=torch.uint8,
                           device=self.own.table.device)

    def _rows(self, t, heads, what, types):
        """kv_rows of a tensor [n_rows, heads, head_dim] of one of the types."""
        if t.dtype not in types:
            raise KvError(KV_EINVAL, f"{what} has type {t.dtype}")
        if t.shape != (self.n_rows, heads, self._dim):
            raise KvError(KV_EINVAL, f"{what} must be [{self.n_rows}, {heads}, {self._dim}], got {list(t.shape)}")
        row, head, last = t.stride()
        if last != 1 and self._dim != 1:
            raise KvError(KV_EINVAL, f"{what}: the last dimension must be contiguous")
        # the stride of a dimension of one is never used, and torch may give any
        return _KvRows(t.data_ptr(), row if self.n_rows > 1 else 0, head if heads > 1 else 0)

    def _call(self, paged, stream, *tensors) -> int | None:
        """Checks of every call; the handle of its stream (None: the current one)."""
        if paged is not self.paged and (paged.page_size, paged.head_dim, paged.num_kv_heads) != \
                (self.paged.page_size, self._dim, self.paged.num_kv_heads):
            raise KvError(KV_EINVAL, "the step was made for a pool of another shape")
        if _here(*tensors) != self._device:
            raise KvError(KV_EINVAL, f"the step's tables are on cuda:{self._device}, not on the current device")
        if paged is not self.paged:
            _here(paged.k_addrs)
        if stream is None:
            h = _t()._C._cuda_getCurrentRawStream(self._device)
            if h not in self._on_streams:
                _used_on_current(self._tensors, self._on_streams)
            if paged is not self.paged and h not in paged._on_streams:
                _used_on_current(paged._arrays, paged._on_streams)
            return h or None
        _used_on(stream, self._tensors, self._on_streams)
        if paged is not self.paged:
            _used_on(stream, paged._arrays)
        _used_on(stream, tensors)
        return _stream_handle(stream)


class Rope:
    """Rotary positions: ``rot`` elements of each head turn in pairs, (j, j +
    rot/2) or, ``interleaved``, (2j, 2j + 1); pair j by position * base^(-2j/rot).

    ``scaling`` for contexts longer than ``original_length``, by ``factor``:
    "linear" (all positions divided), "ntk" (base * factor^(rot/(rot-2))),
    "yarn" (pairs of more than ``fast`` turns in the original length stay,
    those of fewer than ``slow`` are divided, a ramp between; rotated values
    times 0.1 ln(factor) + 1 unless ``gain`` is given) or "wavelength" (the
    same by wavelength, with the ramp between ``low`` and ``high`` turns)."""

    def __init__(self, rot: int, base: float = 10000.0, interleaved: bool = False, scaling: str = "none",
                 factor: float = 1.0, original_length: int = 8192, fast: float = 32.0, slow: float = 1.0,
                 low: float = 1.0, high: float = 4.0, gain: float | None = None, device="cuda"):
        import torch
        f, g = self.frequencies(rot, base, scaling, factor, original_length, fast, slow, low, high)
        self.rot, self.interleaved = int(rot), bool(interleaved)
        self.gain = float(g if gain is None else gain)
        self.freqs = torch.tensor(f, dtype=torch.float64).to(device)
        self._on_streams = set()
        self.c = _KvRope(self.freqs.data_ptr(), self.rot, int(self.interleaved), self.gain)

    @staticmethod
    def frequencies(rot, base=10000.0, scaling="none", factor=1.0, original_length=8192, fast=32.0, slow=1.0,
                    low=1.0, high=4.0):
        """(radians per position of each pair, gain), in Python's 64-bit floats."""
        import math
        _need(rot >= 0 and rot % 2 == 0, "rot must be even")
        _need(base > 1.0 and factor > 0.0 and original_length > 0, "need base > 1, factor > 0, original_length > 0")
        _need(scaling in ("none", "linear", "ntk", "yarn", "wavelength"), f"unknown scaling {scaling!r}")
        gain = 1.0
        if scaling == "ntk":
            _need(rot >= 4, "ntk needs rot >= 4")
            base = base * factor ** (rot / (rot - 2))
        f = [base ** (-2.0 * j / rot) for j in range(rot // 2)]
        if scaling == "linear":
            f = [x / factor for x in f]
        elif scaling == "yarn":
            _need(fast > slow > 0.0, "need fast > slow > 0")

            def pair_of(turns):
                return rot * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))
            lo, hi = max(math.floor(pair_of(fast)), 0), min(math.ceil(pair_of(slow)), rot - 1)
            keep = [1.0 - min(max((j - lo) / max(hi - lo, 0.001), 0.0), 1.0) for j in range(rot // 2)]
            f = [x / factor * (1.0 - k) + x * k for x, k in zip(f, keep)]
            gain = 0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0
        elif scaling == "wavelength":
            _need(high > low, "need high > low")
            turns = [original_length * x / (2 * math.pi) for x in f]
            keep = [min(max((t - low) / (high - low), 0.0), 1.0) for t in turns]
            f = [(1.0 - k) * x / factor + k * x for x, k in zip(f, keep)]
        return f, gain


class Norm:
    """Normalisation of each head of q and k before the rotation:
    (x - c) / sqrt(mean((x - c)^2) + eps) * weight, c = 0 or, ``centered``, the
    head's mean.  ``q_weight`` / ``k_weight``: [head_dim], [heads, head_dim], or
    None for ones; contiguous, 16-byte aligned float32 device tensors are read
    where they are at each call, others are copied once.  A graph that captured calls reads the Norm's
    arrays: keep it for as long as it is replayed."""

    def __init__(self, q_weight=None, k_weight=None, eps: float = 1e-6, centered: bool = False, device="cuda"):
        import torch

        def held(w, name):
            if w is None:
                return None
            _need(w.dim() in (1, 2) and w.dtype.is_floating_point, f"{name} must be [head_dim] or [heads, head_dim]")
            w = w.to(device=device, dtype=torch.float32).contiguous()
            return w.clone() if w.data_ptr() % 16 else w
        self.q_weight, self.k_weight = held(q_weight, "q_weight"), held(k_weight, "k_weight")
        self.eps, self.centered = float(eps), bool(centered)
        self._on_streams = set()
        self._tensors = [w for w in (self.q_weight, self.k_weight) if w is not None]

        def stride(w):
            return 0 if w is None or w.dim() == 1 else w.size(1)
        self.c = _KvNorm(0 if self.q_weight is None else self.q_weight.data_ptr(),
                         0 if self.k_weight is None else self.k_weight.data_ptr(),
                         stride(self.q_weight), stride(self.k_weight), self.eps, int(self.centered))

    def _fits(self, w, heads, dim, name):
        if w is not None and tuple(w.shape) not in ((dim,), (heads, dim)):
            raise KvError(KV_EINVAL, f"{name} must be [{dim}] or [{heads}, {dim}], got {list(w.shape)}")


def _window(window, sinks):
    """kv_window, or None without one."""
    if window is None:
        if sinks:
            raise KvError(KV_EINVAL, "sinks without a window")
        return None
    if (window | sinks) >> 31:
        _int32("window or sinks", window, sinks)
    return _KvWindow(window, sinks)


_type_codes = None


def _empty(shape, dtype, device, stream):
    """A new device tensor for a call on ``stream``: allocated for that stream
    (the caching allocator then orders its memory's earlier use before it) and
    free to be used on the current one."""
    if stream is None:
        return _t().empty(shape, dtype=dtype, device=device)
    if not hasattr(stream, "cuda_stream"):
        raise KvError(KV_EINVAL, "a call on a raw stream handle needs its outputs and workspace given")
    with _t().cuda.stream(stream):
        t = _t().empty(shape, dtype=dtype, device=device)
    if t.is_cuda:
        t.record_stream(_t().cuda.current_stream(t.device))
    return t


def _types():
    global _type_codes
    if _type_codes is None:
        _type_codes = {_t().bfloat16: 0, _t().float16: 1, _t().float32: 2}
    return _type_codes


def _slots(weights, positions, shape, what):
    """kv_slots of contiguous [*shape, heads, cap] tensors."""
    torch = _t()
    for t, dt, name in ((weights, torch.float32, "weights"), (positions, torch.int32, "positions")):
        if t is None or t.dtype != dt or not t.is_contiguous() or t.dim() != len(shape) + 2 or t.shape[:-2] != shape:
            raise KvError(KV_EINVAL,
                          f"{what} {name} must be a contiguous {dt} device tensor {list(shape)} + [heads, slots]")
    if weights.shape != positions.shape:
        raise KvError(KV_EINVAL, f"{what} weights and positions must have one shape")
    return _KvSlots(weights.data_ptr(), positions.data_ptr(), weights.shape[-2], weights.shape[-1])


def append(paged: Paged | Paged8, step: Step, layer: int, q, k, v, positions, rope: Rope, q_out=None, weights=None,
           slot_positions=None, stream=None, norm: Norm | None = None):
    """Rotate the new tokens' q and k, normalised first by ``norm`` if one is
    given, and write k and v into layer ``layer``'s pages (kv_append,
    kv_append_normed; of a Paged8 kv_append8, which takes no eviction state).
    q [rows, q_heads, D] (None: only k and v), k and v [rows, H, D]: bf16, fp16
    or float32, any row and head strides;
    ``positions``: int32 [rows].  ``q_out``: where the rotated q goes (q
    itself, or a tensor of q's type or bf16; None: a new tensor of q's type).
    ``weights`` / ``slot_positions`` [sequences, H or 1, slots]: this layer's
    eviction state; the new slots' weights become 0 and their positions the
    tokens'.  Returns the rotated q."""
    if layer >> 31:
        _int32("layer", layer)
    torch = _t()
    types = _types()
    st = step
    H = paged.num_kv_heads
    ck, cv = st._rows(k, H, "k", types), st._rows(v, H, "v", types)
    if k.dtype != v.dtype or (q is not None and q.dtype != k.dtype):
        raise KvError(KV_EINVAL, "q, k and v must have one type")
    if positions.dtype != torch.int32 or not positions.is_contiguous() or positions.shape != (st.n_rows,):
        raise KvError(KV_EINVAL, f"positions must be a contiguous int32 device tensor [{st.n_rows}]")
    cq = co = None
    q_heads, out_type = 0, types[k.dtype]
    if q is not None:
        _need(q.dim() == 3, "q must be [rows, q_heads, head_dim]")
        q_heads = q.shape[1]
        cq = st._rows(q, q_heads, "q", types)
        if q_out is None:
            q_out = _empty((st.n_rows, q_heads, paged.head_dim), q.dtype, q.device, stream)
        co = st._rows(q_out, q_heads, "q_out", (q.dtype, torch.bfloat16))
        out_type = types[q_out.dtype]
    else:
        _need(q_out is None, "q_out without q")
    cs = None
    if weights is not None or slot_positions is not None:
        cs = _slots(weights, slot_positions, (st.own.n,), "append:")
    bits8 = isinstance(paged, Paged8)
    cn, more = None, ()
    if norm is not None:
        norm._fits(norm.q_weight if q is not None else None, q_heads, paged.head_dim, "q_weight")
        norm._fits(norm.k_weight, H, paged.head_dim, "k_weight")
        cn, more = ctypes.byref(norm.c), norm._tensors
    h = st._call(paged, stream, q, k, v, positions, rope.freqs, q_out, weights, slot_positions, *more)
    if stream is None and (h or 0) not in rope._on_streams:
        _used_on_current((rope.freqs,), rope._on_streams)
    if stream is None and more and (h or 0) not in norm._on_streams:
        _used_on_current(more, norm._on_streams)
    if bits8:
        _need(cs is None, "a Paged8 keeps no eviction state")
        rc = load().kv_append8(ctypes.byref(paged.c), st._ref, layer, _ref(cq), ctypes.byref(ck), ctypes.byref(cv),
                               _ref(co), q_heads, types[k.dtype], out_type, positions.data_ptr(),
                               ctypes.byref(rope.c), cn, h)
    elif cn is not None:
        rc = load().kv_append_normed(ctypes.byref(paged.c), st._ref, layer, _ref(cq), ctypes.byref(ck),
                                     ctypes.byref(cv), _ref(co), q_heads, types[k.dtype], out_type,
                                     positions.data_ptr(), ctypes.byref(rope.c), cn, _ref(cs), h)
    else:
        rc = load().kv_append(ctypes.byref(paged.c), st._ref, layer, _ref(cq), ctypes.byref(ck), ctypes.byref(cv),
                              _ref(co), q_heads, types[k.dtype], out_type, positions.data_ptr(),
                              ctypes.byref(rope.c), _ref(cs), h)
    if rc != KV_OK:
        _check(rc)
    return q_out


def _q(paged, step, q):
    torch = _t()
    _need(q.dim() == 3, "q must be [rows, q_heads, head_dim]")
    return step._rows(q, q.shape[1], "q", (torch.bfloat16,)), q.shape[1]


def _scale(paged, scale) -> float:
    return paged.head_dim ** -0.5 if scale is None else float(scale)


def attend(paged: Paged | Paged8, step: Step, layer: int, q, scale=None, out=None, lse=None, workspace=None,
           stream=None, window: int | None = None, sinks: int = 0):
    """Attention of the new tokens' bf16 q [rows, q_heads, D] over their
    group's shared prefix and their own pages up to themselves (kv_attend; of a
    Paged8 kv_attend8).  With ``window`` (kv_attend_window) a row sees only the
    last ``window`` tokens up to its own, counted over prefix and own pages,
    and the first ``sinks`` of all.  ``scale``: 1/sqrt(D) unless given.
    ``workspace``: a device uint8 tensor of step.attend_workspace_bytes(q_heads,
    window, sinks, paged) (None: one is allocated for the call).
    Returns (out bf16 like q, lse float32 [rows, q_heads])."""
    if layer >> 31:
        _int32("layer", layer)
    torch = _t()
    cq, heads = _q(paged, step, q)
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    if lse is None:
        lse = _empty((step.n_rows, heads), torch.float32, q.device, stream)
    co = step._rows(out, heads, "out", (torch.bfloat16,))
    if lse.dtype != torch.float32 or not lse.is_contiguous() or lse.shape != (step.n_rows, heads):
        raise KvError(KV_EINVAL, f"lse must be a contiguous float32 device tensor [{step.n_rows}, {heads}]")
    cw = _window(window, sinks)
    if workspace is None:
        workspace = _empty(step.attend_workspace_bytes(heads, window, sinks, paged), torch.uint8, q.device, stream)
    ws, n_ws = _workspace(workspace)
    h = step._call(paged, stream, q, out, lse, workspace)
    if isinstance(paged, Paged8):
        rc = load().kv_attend8(ctypes.byref(paged.c), step._ref, layer, ctypes.byref(cq), heads,
                               _scale(paged, scale), _ref(cw), ctypes.byref(co), lse.data_ptr(), ws, n_ws, h)
    elif cw is not None:
        rc = load().kv_attend_window(ctypes.byref(paged.c), step._ref, layer, ctypes.byref(cq), heads,
                                     _scale(paged, scale), ctypes.byref(cw), ctypes.byref(co), lse.data_ptr(), ws,
                                     n_ws, h)
    else:
        rc = load().kv_attend(ctypes.byref(paged.c), step._ref, layer, ctypes.byref(cq), heads, _scale(paged, scale),
                              ctypes.byref(co), lse.data_ptr(), ws, n_ws, h)
    if rc != KV_OK:
        _check(rc)
    return out, lse


def _sums(inp, out, n, heads, what):
    torch = _t()
    if out is None:
        out = inp
    if out is None:
        return None, None
    for t in (inp, out):
        if t is not None and (t.dtype != torch.float32 or not t.is_contiguous() or t.dim() != 3
                              or t.shape[:2] != (n, heads) or t.shape != out.shape):
            raise KvError(KV_EINVAL,
                          f"{what} must be contiguous float32 device tensors [{n}, {heads}, slots] of one shape")
    return _KvSums(inp.data_ptr() if inp is not None else None, out.data_ptr(), out.shape[2]), out


def add_weights(paged: Paged, step: Step, layer: int, q, lse, weights=None, prefix_weights=None, scale=None,
                out=None, prefix_out=None, stream=None):
    """Add the attention weights of the new tokens' q to every cached token's
    running sum (kv_add_weights): ``weights`` [sequences, H, slots] for the
    own pages, ``prefix_weights`` [groups, H, slots] for the shared prefixes
    (either may be None: not computed), in place, or into ``out`` /
    ``prefix_out`` (with weights None: from zero).  ``lse``: what attend
    returned.  Returns (own sums, prefix sums)."""
    _bf16_pool(paged, "add_weights")
    if layer >> 31:
        _int32("layer", layer)
    torch = _t()
    cq, heads = _q(paged, step, q)
    if lse.dtype != torch.float32 or not lse.is_contiguous() or lse.shape != (step.n_rows, heads):
        raise KvError(KV_EINVAL, f"lse must be a contiguous float32 device tensor [{step.n_rows}, {heads}]")
    co, out = _sums(weights, out, step.own.n, paged.num_kv_heads, "weights")
    cp, prefix_out = _sums(prefix_weights, prefix_out, step.prefix.n if step.prefix is not None else 0,
                           paged.num_kv_heads, "prefix weights")
    h = step._call(paged, stream, q, lse, weights, prefix_weights, out, prefix_out)
    rc = load().kv_add_weights(ctypes.byref(paged.c), step._ref, layer, ctypes.byref(cq), lse.data_ptr(), heads,
                               _scale(paged, scale), _ref(co), _ref(cp), h)
    if rc != KV_OK:
        _check(rc)
    return out, prefix_out


def evict(paged: Paged, tables: Tables, layer_begin: int, layer_end: int, weights, positions, keep: int,
          recent: int = 0, out_weights=None, out_positions=None, out_lens=None, workspace=None, stream=None):
    """Evict each (layer, sequence, head) down to ``keep`` tokens by weight,
    the ``recent`` newest protected, and move what stays into the first slots
    (kv_evict).  ``weights`` float32 and ``positions`` int32 [layers, sequences,
    H or 1, slots], updated in place unless out_weights / out_positions
    [layers, sequences, H or 1, >= keep] are given.  ``workspace``: a device
    uint8 tensor of tables.evict_workspace_bytes(...) (None: allocated for the
    call).  Returns the new lengths, an int32 tensor [sequences]."""
    _bf16_pool(paged, "evict")
    if (layer_begin | layer_end | keep | recent) >> 31:
        _int32("layer, keep or recent", layer_begin, layer_end, keep, recent)
    torch = _t()
    shape = (layer_end - layer_begin, tables.n)
    ci = _slots(weights, positions, shape, "evict:")
    if out_weights is None and out_positions is None:
        out_weights, out_positions, co = weights, positions, ci
    else:
        co = _slots(out_weights, out_positions, shape, "evict: out")
    tables._check(paged)
    if out_lens is None:
        out_lens = _empty((tables.n,), torch.int32, tables.table.device, stream)
    if out_lens.dtype != torch.int32 or not out_lens.is_contiguous() or out_lens.shape != (tables.n,):
        raise KvError(KV_EINVAL, f"out_lens must be a contiguous int32 device tensor [{tables.n}]")
    if workspace is None:
        workspace = _empty(tables.evict_workspace_bytes(paged, shape[0], ci.heads, keep), torch.uint8,
                           tables.table.device, stream)
    ws, n_ws = _workspace(workspace)
    used = (paged.k_addrs, paged.v_addrs, tables.table, tables.lens, weights, positions, out_weights, out_positions,
            out_lens, workspace)
    dev = _here(*used)
    if stream is None:
        h = torch._C._cuda_getCurrentRawStream(dev) or None
        if (h or 0) not in paged._on_streams:
            _used_on_current((paged.k_addrs, paged.v_addrs), paged._on_streams)
    else:
        _used_on(stream, used)
        h = _stream_handle(stream)
    rc = load().kv_evict(ctypes.byref(paged.c), ctypes.byref(tables.c), layer_begin, layer_end, ctypes.byref(ci),
                         ctypes.byref(co), keep, recent, out_lens.data_ptr(), ws, n_ws, h)
    if rc != KV_OK:
        _check(rc)
    return out_lens


def _pack(call, source, tables, target, to_table, layer_begin, layer_end, stream) -> None:
    torch = _t()
    if layer_end is None:
        layer_end = source.num_layers
    if (layer_begin | layer_end) >> 31:
        _int32("layer", layer_begin, layer_end)
    tables._check(source)
    table, stride = None, 0
    if to_table is not None:
        if to_table.dtype != torch.int32 or to_table.dim() != 2 or to_table.size(0) != tables.n or not (
                to_table.stride(1) == 1 or to_table.size(1) <= 1):
            raise KvError(KV_EINVAL, f"to_table must be an int32 device tensor [{tables.n}, entries], entries contiguous")
        if tables.max_len > to_table.size(1) * source.page_size:
            raise KvError(KV_ERANGE, f"max_len {tables.max_len} beyond to_table ({to_table.size(1)} pages of "
                                     f"{source.page_size})")
        _need(tables.n <= 1 or to_table.stride(0) >= to_table.size(1), "to_table's rows must not overlap")
        table, stride = to_table.data_ptr(), to_table.stride(0) if tables.n > 1 else to_table.size(1)
    used = (*source._arrays, *target._arrays, tables.table, tables.lens, to_table)
    dev = _here(*used)
    if stream is None:
        h = torch._C._cuda_getCurrentRawStream(dev) or None
        for p in (source, target):
            if (h or 0) not in p._on_streams:
                _used_on_current(p._arrays, p._on_streams)
    else:
        _used_on(stream, used)
        h = _stream_handle(stream)
    rc = call(ctypes.byref(source.c), ctypes.byref(tables.c), ctypes.byref(target.c), table, stride, layer_begin,
              layer_end, h)
    if rc != KV_OK:
        _check(rc)


def pack8(paged: Paged, tables: Tables, paged8: Paged8, to_table=None, layer_begin: int = 0,
          layer_end: int | None = None, stream=None) -> None:
    """The cached tokens of ``tables``' sequences from the bf16 pool's pages into
    the 8-bit pool's (kv_pack8), of layers [layer_begin, layer_end) (all unless
    given): into the pages of ``to_table``, int32 [sequences, entries], or
    those of the same ids.  Each block's scale is made from the tokens it
    holds.  After retrieve it brings chunks into an 8-bit pool."""
    _bf16_pool(paged, "pack8's source")
    _need(isinstance(paged8, Paged8), "pack8 needs a Paged8 to write to")
    _pack(load().kv_pack8, paged, tables, paged8, to_table, layer_begin, layer_end, stream)


def unpack8(paged8: Paged8, tables: Tables, paged: Paged, to_table=None, layer_begin: int = 0,
            layer_end: int | None = None, stream=None) -> None:
    """The reverse of pack8 (kv_unpack8): byte * scale as bf16, exactly, into the
    bf16 pool's pages, for store, add_weights or evict."""
    _bf16_pool(paged, "unpack8's target")
    _need(isinstance(paged8, Paged8), "unpack8 needs a Paged8 to read from")
    _pack(load().kv_unpack8, paged8, tables, paged, to_table, layer_begin, layer_end, stream)
