"""ctypes binding of libtd.so: argument marshalling and buffer checks only."""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import torch

MODE_FULL = 0
MODE_FULL_SELECT = 1
MODE_SPARSE = 2
FLAG_INDEX_OUT_OF_RANGE = 0x1
FLAG_SEQ_LEN_OUT_OF_RANGE = 0x2
FLAG_WAIT_TIMEOUT = 0x4
FLAG_TREE_OUT_OF_RANGE = 0x8
FLAG_PAGE_OUT_OF_RANGE = 0x10
FLAG_PAGES_EXHAUSTED = 0x20
MAX_TREE = 128                   # TD_MAX_TREE: drafted tokens per request of a tree call
NOALLOC_SCRATCH_BYTES = 8 << 20  # TD_NOALLOC_SCRATCH_BYTES: td_sparse_attn_noalloc's fixed scratch

_HERE = os.path.dirname(os.path.abspath(__file__))


def lib_path() -> str:
    return os.path.join(_HERE, "libtd.so")


class TdError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {td_status_string(status)} ({status})")


class Shape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("max_seq_len", ctypes.c_int32), ("scale", ctypes.c_float)]

    @property
    def group(self) -> int:
        return self.num_q_heads // self.num_kv_heads


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("block_table", ctypes.c_void_p),
                ("max_blocks", ctypes.c_int32)]


class _Q4Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("block_table", ctypes.c_void_p), ("max_blocks", ctypes.c_int32)]


def default_scale(head_dim: int) -> float:
    """The library's scale when Shape.scale == 0: 1/sqrtf(head_dim) in fp32."""
    import numpy as np
    return float(np.float32(1.0) / np.sqrt(np.float32(head_dim)))


def make_shape(batch, num_q_heads, num_kv_heads, max_seq_len, head_dim=128, scale=0.0) -> Shape:
    return Shape(batch, num_q_heads, num_kv_heads, head_dim, max_seq_len, scale)


_lib = None


def lib():
    """Load libtd.so; raise if it has not been built (no fallback exists)."""
    global _lib
    if _lib is not None:
        return _lib
    path = lib_path()
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -c \"import __graft_entry__ "
                          f"as g; g.build()\"` (or sparse_attention_td_gb300/build.py)")
    L = ctypes.CDLL(path)
    vp, sz, i32, u32p = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.POINTER(ctypes.c_uint32)
    shp = ctypes.POINTER(Shape)
    vpp = ctypes.POINTER(ctypes.c_void_p)
    L.td_status_string.restype = ctypes.c_char_p
    L.td_status_string.argtypes = [ctypes.c_int]
    L.td_workspace_size.restype = sz
    L.td_workspace_size.argtypes = [shp, i32]
    L.td_workspace_init.restype = ctypes.c_int
    L.td_workspace_init.argtypes = [vp, sz, vp]
    L.td_workspace_status.restype = ctypes.c_int
    L.td_workspace_status.argtypes = [vp, sz, u32p, vp]
    L.td_full_attn_select.restype = ctypes.c_int
    L.td_full_attn_select.argtypes = [shp, vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, sz, vp]
    L.td_topk_select.restype = ctypes.c_int
    L.td_topk_select.argtypes = [shp, vp, vp, i32, vp, vp, sz, vp]
    L.td_full_attn_select_coverage.restype = ctypes.c_int
    L.td_full_attn_select_coverage.argtypes = [shp, vp, vp, vp, vp, ctypes.c_float, i32, vp, vp,
                                               vp, vp, vp, vp, sz, vp]
    L.td_probe_layer_reads.restype = ctypes.c_int
    L.td_probe_layer_reads.argtypes = [shp, vp, vp, vp, vp, i32, vp, i32, vp]
    L.td_kv_append.restype = ctypes.c_int
    L.td_kv_append.argtypes = [shp, vp, vp, vp, vp, vp, vp]
    L.td_decode_step_append.restype = ctypes.c_int
    L.td_decode_step_append.argtypes = [shp, i32, vp, vpp, vpp, vpp, vpp, vpp, vp, i32, vp, i32,
                                        vpp, vpp, vp, sz, vp, vpp]
    L.td_plan_create_append.restype = ctypes.c_int
    L.td_plan_create_append.argtypes = [ctypes.POINTER(vp), shp, i32, vp, vpp, vpp, vpp, vpp, vpp,
                                        vp, i32, vp, i32, vpp, vpp, vp, sz]
    L.td_plan_create_host.restype = ctypes.c_int
    L.td_plan_create_host.argtypes = [ctypes.POINTER(vp), shp, i32, vp, vp, vp, vpp, vpp, vp,
                                      i32, vp, i32, vp, vpp, vp, vp, sz]
    L.td_index_overlap.restype = ctypes.c_int
    L.td_index_overlap.argtypes = [shp, vp, vp, i32, vp, vp]
    cch, i64 = ctypes.POINTER(_Cache), ctypes.c_int64
    L.td_tree_workspace_size.restype = sz
    L.td_tree_workspace_size.argtypes = [shp, i32]
    L.td_tree_attn.restype = ctypes.c_int
    L.td_tree_attn.argtypes = [shp, cch, i32, vp, vp, vp, vp, vp, vp, sz, vp]
    L.td_tree_sparse_attn.restype = ctypes.c_int
    L.td_tree_sparse_attn.argtypes = [shp, cch, i32, vp, vp, vp, vp, vp, i32, vp, vp, sz, vp]
    L.td_tree_commit.restype = ctypes.c_int
    L.td_tree_commit.argtypes = [shp, i32, cch, i32, vp, vp, vp, vp, vp, vp, sz, vp]
    L.td_kv_append_slots.restype = ctypes.c_int
    L.td_kv_append_slots.argtypes = [shp, cch, i32, vp, vp, i64, vp, vp]
    L.td_block_tables.restype = ctypes.c_int
    L.td_block_tables.argtypes = [i32, i32, i32, i32] + [vp] * 10 + [i32, vp, sz, vp]
    q4 = ctypes.POINTER(_Q4Cache)
    L.td_cache_workspace_size.restype = sz
    L.td_cache_workspace_size.argtypes = [shp]
    for call, cache in ((L.td_window_attn, cch), (L.td_q4_attn, q4)):
        call.restype = ctypes.c_int
        call.argtypes = [shp, cache, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
    L.td_q4_sparse_attn.restype = ctypes.c_int
    L.td_q4_sparse_attn.argtypes = [shp, q4, vp, vp, vp, i32, vp, vp, sz, vp]
    L.td_q4_append.restype = ctypes.c_int
    L.td_q4_append.argtypes = [shp, q4, i32, vp, vp, i64, vp, vp]
    L.td_weights_attn.restype = ctypes.c_int
    L.td_weights_attn.argtypes = [shp, cch, i32, vp, vp, vp, vp, vp, vp, sz, vp]
    L.td_evict.restype = ctypes.c_int
    L.td_evict.argtypes = [shp, cch, cch, i32, i32, i32, vp, vp, i32, vp, vp, vp, vp, sz, vp]
    L.td_sparse_attn.restype = ctypes.c_int
    L.td_sparse_attn.argtypes = [shp, vp, vp, vp, vp, vp, i32, vp, vp, vp, sz, vp]
    L.td_sparse_attn_noalloc.restype = ctypes.c_int
    L.td_sparse_attn_noalloc.argtypes = [shp, vp, vp, vp, vp, vp, i32, vp, vp, vp]
    L.td_decode_step.restype = ctypes.c_int
    L.td_decode_step.argtypes = [shp, i32, vp, vpp, vpp, vpp, vp, i32, vp, i32, vpp, vpp, vp, sz,
                                 vp, vpp]
    L.td_plan_create.restype = ctypes.c_int
    L.td_plan_create.argtypes = [ctypes.POINTER(vp), shp, i32, vp, vpp, vpp, vpp, vp, i32, vp, i32,
                                 vpp, vpp, vp, sz]
    L.td_plan_launch.restype = ctypes.c_int
    L.td_plan_launch.argtypes = [vp, vp]
    L.td_plan_destroy.restype = None
    L.td_plan_destroy.argtypes = [vp]
    L.td_set_tuning.restype = ctypes.c_int
    L.td_set_tuning.argtypes = [ctypes.c_char_p, i32]
    L.td_query_splits.restype = i32
    L.td_query_splits.argtypes = [shp, i32, i32]
    L.td_kernel_name.restype = ctypes.c_char_p
    L.td_kernel_name.argtypes = [shp, i32, i32]
    _lib = L
    return L


def td_status_string(status: int) -> str:
    return lib().td_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != 0:
        raise TdError(status, where)


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _torch_stream(stream):
    if stream is None:
        return torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(stream))


def _dev(t: Optional[torch.Tensor], name: str, dtype, numel: Optional[int] = None,
         optional=False) -> Optional[int]:
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name} holds {t.numel()} elements, needs {numel}")
    return t.data_ptr()


def td_workspace_size(shape: Shape, top_k: int) -> int:
    return int(lib().td_workspace_size(ctypes.byref(shape), int(top_k)))


def td_workspace_init(ws: torch.Tensor, stream=None):
    _check(lib().td_workspace_init(_dev(ws, "ws", torch.uint8), ws.numel(), _stream(stream)),
           "td_workspace_init")


def td_workspace_status(ws: torch.Tensor, stream=None) -> int:
    flags = ctypes.c_uint32(0)
    _check(lib().td_workspace_status(_dev(ws, "ws", torch.uint8), ws.numel(),
                                     ctypes.byref(flags), _stream(stream)),
           "td_workspace_status")
    return flags.value


def td_tree_workspace_size(shape: Shape, tree_size: int) -> int:
    return int(lib().td_tree_workspace_size(ctypes.byref(shape), int(tree_size)))


def td_cache_workspace_size(shape: Shape) -> int:
    return int(lib().td_cache_workspace_size(ctypes.byref(shape)))


class Workspace:
    """A zero-initialised device workspace of td_workspace_size bytes; with
    tree_size also td_tree_workspace_size bytes, for the tree calls.  Those write
    the buffer's last bytes, which the other calls must find as they left them: the
    tree calls take only a workspace with a tree part of their size, the others see
    the buffer without it.  cache_calls adds td_cache_workspace_size bytes, between
    the two, for the calls on small caches (td_window_attn and those behind it), which
    likewise take only a workspace with a part large enough and write no other."""

    def __init__(self, shape: Shape, top_k: int, device=None, stream=None, tree_size: int = 0,
                 cache_calls: bool = False):
        n = td_workspace_size(shape, top_k)
        if n == 0:
            raise TdError(1, "td_workspace_size")
        self.cache_bytes = (td_cache_workspace_size(shape) + 255) // 256 * 256 if cache_calls else 0
        self._cache_shapes = set()   # (batch, query heads, KV heads) known to fit
        n = (n + 255) // 256 * 256 + self.cache_bytes if cache_calls else n
        self.tree_bytes = 0
        if tree_size:
            self.tree_bytes = td_tree_workspace_size(shape, tree_size)
            if self.tree_bytes == 0:
                raise TdError(1, "td_tree_workspace_size")
        self._trees = set()          # (query heads, KV heads, tree size) known to fit
        self.tensor = torch.empty(n + self.tree_bytes, dtype=torch.uint8, device=device or "cuda")
        td_workspace_init(self.tensor, stream)

    @property
    def ptr(self) -> int:
        return self.tensor.data_ptr()

    @property
    def nbytes(self) -> int:
        """Bytes without the parts of the tree calls and of the calls on small caches."""
        return self.tensor.numel() - self.tree_bytes - self.cache_bytes

    def check_cache(self, shape: Shape):
        key = (shape.batch, shape.num_q_heads, shape.num_kv_heads)
        if key in self._cache_shapes:
            return
        need = td_cache_workspace_size(shape)
        if need > self.cache_bytes:
            raise ValueError(f"ws has {self.cache_bytes} bytes for calls on small caches, needs {need} "
                             f"(Workspace(..., cache_calls=True))")
        if need:                     # (0: the call refuses the shape)
            self._cache_shapes.add(key)

    def check_tree(self, shape: Shape, tree_size: int):
        key = (shape.num_q_heads, shape.num_kv_heads, tree_size)
        if key in self._trees:
            return
        need = td_tree_workspace_size(shape, tree_size)
        if need > self.tree_bytes:
            raise ValueError(f"ws has {self.tree_bytes} bytes for tree calls, needs {need} "
                             f"(Workspace(..., tree_size={tree_size}))")
        if need:                     # (0: the call refuses the shape or tree_size)
            self._trees.add(key)

    def status(self, stream=None) -> int:
        return td_workspace_status(self.tensor, stream)


def _sizes(shape: Shape):
    B, Hq, Hkv, d, N = (shape.batch, shape.num_q_heads, shape.num_kv_heads, shape.head_dim,
                        shape.max_seq_len)
    return B * Hq * d, B * Hkv * N * d, B


def td_full_attn_select(shape: Shape, q, k_cache, v_cache, seq_lens, top_k, idx_out, out,
                        out_f32=None, scores_out=None, ws: Workspace = None, stream=None):
    nq, nkv, nb = _sizes(shape)
    st = lib().td_full_attn_select(
        ctypes.byref(shape), _dev(q, "q", torch.bfloat16, nq),
        _dev(k_cache, "k_cache", torch.bfloat16, nkv), _dev(v_cache, "v_cache", torch.bfloat16, nkv),
        _dev(seq_lens, "seq_lens", torch.int32, nb), int(top_k),
        _dev(idx_out, "idx_out", torch.int32, nb * shape.num_kv_heads * top_k, optional=top_k == 0),
        _dev(out, "out", torch.bfloat16, nq), _dev(out_f32, "out_f32", torch.float32, nq, True),
        _dev(scores_out, "scores_out", torch.float32, nkv // shape.head_dim, True),
        ws.ptr, ws.nbytes, _stream(stream))
    _check(st, "td_full_attn_select")


def td_full_attn_select_coverage(shape: Shape, q, k_cache, v_cache, seq_lens, tau, k_max, idx_out,
                                 counts_out, out, out_f32=None, scores_out=None,
                                 ws: Workspace = None, stream=None):
    nq, nkv, nb = _sizes(shape)
    st = lib().td_full_attn_select_coverage(
        ctypes.byref(shape), _dev(q, "q", torch.bfloat16, nq),
        _dev(k_cache, "k_cache", torch.bfloat16, nkv), _dev(v_cache, "v_cache", torch.bfloat16, nkv),
        _dev(seq_lens, "seq_lens", torch.int32, nb), float(tau), int(k_max),
        _dev(idx_out, "idx_out", torch.int32, nb * shape.num_kv_heads * k_max),
        _dev(counts_out, "counts_out", torch.int32, nb * shape.num_kv_heads, True),
        _dev(out, "out", torch.bfloat16, nq), _dev(out_f32, "out_f32", torch.float32, nq, True),
        _dev(scores_out, "scores_out", torch.float32, nkv // shape.head_dim, True),
        ws.ptr, ws.nbytes, _stream(stream))
    _check(st, "td_full_attn_select_coverage")


def td_topk_select(shape: Shape, scores, seq_lens, top_k, idx_out, ws: Workspace = None,
                   stream=None):
    nq, nkv, nb = _sizes(shape)
    st = lib().td_topk_select(
        ctypes.byref(shape), _dev(scores, "scores", torch.float32, nkv // shape.head_dim),
        _dev(seq_lens, "seq_lens", torch.int32, nb), int(top_k),
        _dev(idx_out, "idx_out", torch.int32, nb * shape.num_kv_heads * top_k),
        ws.ptr, ws.nbytes, _stream(stream))
    _check(st, "td_topk_select")


def td_index_overlap(shape: Shape, idx_a, idx_b, top_k, counts, stream=None):
    n = shape.batch * shape.num_kv_heads
    st = lib().td_index_overlap(
        ctypes.byref(shape), _dev(idx_a, "idx_a", torch.int32, n * top_k),
        _dev(idx_b, "idx_b", torch.int32, n * top_k), int(top_k),
        _dev(counts, "counts", torch.int32, n), _stream(stream))
    _check(st, "td_index_overlap")


def td_sparse_attn(shape: Shape, q, k_cache, v_cache, seq_lens, idx, top_k, out, out_f32=None,
                   ws: Workspace = None, stream=None):
    nq, nkv, nb = _sizes(shape)
    st = lib().td_sparse_attn(
        ctypes.byref(shape), _dev(q, "q", torch.bfloat16, nq),
        _dev(k_cache, "k_cache", torch.bfloat16, nkv), _dev(v_cache, "v_cache", torch.bfloat16, nkv),
        _dev(seq_lens, "seq_lens", torch.int32, nb),
        _dev(idx, "idx", torch.int32, nb * shape.num_kv_heads * top_k), int(top_k),
        _dev(out, "out", torch.bfloat16, nq), _dev(out_f32, "out_f32", torch.float32, nq, True),
        ws.ptr, ws.nbytes, _stream(stream))
    _check(st, "td_sparse_attn")


def td_sparse_attn_noalloc(shape: Shape, q, k_cache, v_cache, seq_lens, idx, top_k, out,
                           out_f32=None, stream=None):
    """td_sparse_attn without a workspace, for callers that cannot allocate
    device memory (scratch lives in a fixed array in the library)."""
    nq, nkv, nb = _sizes(shape)
    st = lib().td_sparse_attn_noalloc(
        ctypes.byref(shape), _dev(q, "q", torch.bfloat16, nq),
        _dev(k_cache, "k_cache", torch.bfloat16, nkv), _dev(v_cache, "v_cache", torch.bfloat16, nkv),
        _dev(seq_lens, "seq_lens", torch.int32, nb),
        _dev(idx, "idx", torch.int32, nb * shape.num_kv_heads * top_k), int(top_k),
        _dev(out, "out", torch.bfloat16, nq), _dev(out_f32, "out_f32", torch.float32, nq, True),
        _stream(stream))
    _check(st, "td_sparse_attn_noalloc")


def _ptr_array(tensors, name, dtype, numel, optional=False):
    ptrs = [_dev(t, f"{name}[{i}]", dtype, numel, optional) or 0 for i, t in enumerate(tensors)]
    return (ctypes.c_void_p * max(len(ptrs), 1))(*ptrs)


# The calls below run once or more per layer, so their marshalling is kept short:
# one look at each tensor (_on), the raw stream handle.

def _launch(stream):
    """(device, raw stream): a call launches on the current device."""
    dev = torch._C._cuda_getDevice()
    if stream is None:
        return dev, torch._C._cuda_getCurrentRawStream(dev)
    if isinstance(stream, torch.cuda.Stream) and stream.device_index != dev:
        raise ValueError(f"the stream is on cuda:{stream.device_index}, the current device is cuda:{dev}")
    return dev, _stream(stream)


def _on(dev, t, name, dtype, numel):
    """Pointer of a contiguous tensor of at least numel values on device dev."""
    if t is not None and t.get_device() == dev and t.dtype is dtype and t.is_contiguous() and \
            t.numel() >= numel:
        return t.data_ptr()
    _dev(t, name, dtype, numel)
    raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")


def _ws(dev, ws):
    if ws is None:
        raise ValueError("ws is required")
    t = ws.tensor
    if t.get_device() != dev:
        raise ValueError(f"ws is on {t.device}, the current device is cuda:{dev}")
    return t.data_ptr(), t.numel()


def _tree_ws(dev, ws, shape, tree_size):
    where = _ws(dev, ws)
    ws.check_tree(shape, tree_size)
    return where


class Cache:
    """One layer's K/V rows (td_cache): k, v [pages][Hkv][page_size][128] and a
    block table [B][max_blocks], or without a table a contiguous cache
    [B][Hkv][max_seq_len][128]."""

    def __init__(self, k, v, block_table=None):
        for name, t in (("k", k), ("v", v)):
            if t.dim() != 4 or t.shape[3] != 128:
                raise ValueError(f"{name} must be [pages][kv heads][page size][128], got {tuple(t.shape)}")
        if k.shape != v.shape:
            raise ValueError(f"k and v differ: {tuple(k.shape)} and {tuple(v.shape)}")
        if block_table is not None and block_table.dim() != 2:
            raise ValueError("block_table must be [batch][max_blocks]")
        self.k, self.v, self.block_table = k, v, block_table
        self.num_pages, self.kv_heads, self.page_size = (int(x) for x in k.shape[:3])
        self.c = _Cache(_dev(k, "k", torch.bfloat16), _dev(v, "v", torch.bfloat16), self.num_pages,
                        self.page_size, _dev(block_table, "block_table", torch.int32, optional=True),
                        0 if block_table is None else int(block_table.shape[1]))
        self.device = k.get_device()
        for name, t in (("v", v), ("block_table", block_table)):
            if t is not None and t.get_device() != self.device:
                raise ValueError(f"k is on {k.device}, {name} on {t.device}")
        self.ref = ctypes.byref(self.c)
        self.raw = bytes(self.c)
        # what a call has to agree with: device, KV heads, requests (None: any)
        self.fits = (self.device, self.kv_heads, None if block_table is None else int(block_table.shape[0]))

    def check(self, shape: Shape, dev: int):
        _fits(self.fits, shape, dev)
        return self.ref


def _fits(fits, shape, dev):
    device, heads, rows = fits
    if device != dev:
        raise ValueError(f"the cache is on cuda:{device}, the current device is cuda:{dev}")
    if heads != shape.num_kv_heads:
        raise ValueError(f"the cache has {heads} KV heads, the shape {shape.num_kv_heads}")
    if rows is not None and rows < shape.batch:
        raise ValueError(f"block_table has {rows} rows, needs {shape.batch}")


def make_cache(k, v, block_table=None) -> Cache:
    return Cache(k, v, block_table)


_BF16, _I32, _F32 = torch.bfloat16, torch.int32, torch.float32


def td_tree_attn(shape: Shape, cache: Cache, tree_size, tree_lens, tree_mask, q, seq_lens, out,
                 ws: Workspace = None, stream=None):
    """Attention of tree_size drafted tokens per request over the cache;
    tree_mask int32 words [B][T][ceil(T / 32)] (None: a chain)."""
    dev, st = _launch(stream)
    nb, T = shape.batch, int(tree_size)
    wp, wn = _tree_ws(dev, ws, shape, T)
    n = nb * T * shape.num_q_heads * 128
    rc = lib().td_tree_attn(
        shape, cache.check(shape, dev), T,
        None if tree_lens is None else _on(dev, tree_lens, "tree_lens", _I32, nb),
        None if tree_mask is None else _on(dev, tree_mask, "tree_mask", _I32, nb * T * ((T + 31) // 32)),
        _on(dev, q, "q", _BF16, n), _on(dev, seq_lens, "seq_lens", _I32, nb),
        _on(dev, out, "out", _BF16, n), wp, wn, st)
    if rc:
        _check(rc, "td_tree_attn")


def td_tree_sparse_attn(shape: Shape, cache: Cache, tree_size, tree_lens, tree_mask, q, seq_lens,
                        idx, top_k, out, ws: Workspace = None, stream=None):
    """td_tree_attn over the persisted index set of a PPSA layer and the tree."""
    dev, st = _launch(stream)
    nb, T, k = shape.batch, int(tree_size), int(top_k)
    wp, wn = _tree_ws(dev, ws, shape, T)
    n = nb * T * shape.num_q_heads * 128
    rc = lib().td_tree_sparse_attn(
        shape, cache.check(shape, dev), T,
        None if tree_lens is None else _on(dev, tree_lens, "tree_lens", _I32, nb),
        None if tree_mask is None else _on(dev, tree_mask, "tree_mask", _I32, nb * T * ((T + 31) // 32)),
        _on(dev, q, "q", _BF16, n), _on(dev, seq_lens, "seq_lens", _I32, nb),
        _on(dev, idx, "idx", _I32, nb * shape.num_kv_heads * k), k, _on(dev, out, "out", _BF16, n),
        wp, wn, st)
    if rc:
        _check(rc, "td_tree_sparse_attn")


def td_tree_commit(shape: Shape, caches: Sequence[Cache], tree_size, tree_lens, accepted,
                   accepted_lens, seq_lens, seq_lens_out, ws: Workspace = None, stream=None):
    """Move the accepted drafted rows of every layer to the front of their tree."""
    dev, st = _launch(stream)
    wp, wn = _ws(dev, ws)
    nb, T = shape.batch, int(tree_size)
    for fits in {c.fits for c in caches}:
        _fits(fits, shape, dev)
    arr = ctypes.create_string_buffer(b"".join([c.raw for c in caches]))   # the td_cache array
    rc = lib().td_tree_commit(
        shape, len(caches), ctypes.cast(arr, ctypes.POINTER(_Cache)), T,
        None if tree_lens is None else _on(dev, tree_lens, "tree_lens", _I32, nb),
        _on(dev, accepted, "accepted", _I32, nb * T), _on(dev, accepted_lens, "accepted_lens", _I32, nb),
        _on(dev, seq_lens, "seq_lens", _I32, nb), _on(dev, seq_lens_out, "seq_lens_out", _I32, nb),
        wp, wn, st)
    if rc:
        _check(rc, "td_tree_commit")


def _token_rows(dev, t, name, heads):
    """A [tokens][heads][128] tensor whose token rows may lie apart (a column
    block of a packed projection): its pointer, tokens and token stride."""
    if t.get_device() != dev or t.dtype is not _BF16:
        raise ValueError(f"{name} must be a bfloat16 tensor on cuda:{dev}")
    size, step = t.shape, t.stride()
    if len(size) != 3 or size[1] != heads or size[2] != 128 or step[2] != 1 or \
            (heads > 1 and step[1] != 128):
        raise ValueError(f"{name} must be [tokens][{heads}][128] with whole token rows")
    return t.data_ptr(), size[0], step[0] if size[0] > 1 else heads * 128


def td_kv_append_slots(shape: Shape, cache: Cache, k_new, v_new, slot_map, stream=None):
    """New K/V rows [tokens][Hkv][128] into the cache at slot_map [tokens]."""
    dev, st = _launch(stream)
    heads = shape.num_kv_heads
    ref = cache.ref
    if cache.device != dev or cache.kv_heads != heads:
        cache.check(shape, dev)
    pk, n, sk = _token_rows(dev, k_new, "k_new", heads)
    pv, nv, sv = _token_rows(dev, v_new, "v_new", heads)
    if n != nv or sk != sv:
        raise ValueError("k_new and v_new must have the same tokens and token stride")
    rc = lib().td_kv_append_slots(shape, ref, n, pk, pv, sk, _on(dev, slot_map, "slot_map", _I32, n), st)
    if rc:
        _check(rc, "td_kv_append_slots")


def td_block_tables(seq_lens, new_lens, page_size, block_table, num_blocks, num_blocks_out,
                    free_pages, free_count, free_count_out, cu_new, slot_map,
                    ws: Workspace = None, stream=None):
    """Block tables and slot map of a batch from its lengths; sizes come from
    block_table [B][max_blocks], free_pages [num_pages] and slot_map [max_new]."""
    dev, st = _launch(stream)
    wp, wn = _ws(dev, ws)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [batch][max_blocks]")
    B, blocks = block_table.shape
    pages, slots = free_pages.numel(), slot_map.numel()
    rc = lib().td_block_tables(
        B, int(page_size), blocks, pages, _on(dev, seq_lens, "seq_lens", _I32, B),
        _on(dev, new_lens, "new_lens", _I32, B), _on(dev, block_table, "block_table", _I32, 0),
        _on(dev, num_blocks, "num_blocks", _I32, B),
        _on(dev, num_blocks_out, "num_blocks_out", _I32, B),
        _on(dev, free_pages, "free_pages", _I32, 0), _on(dev, free_count, "free_count", _I32, 1),
        _on(dev, free_count_out, "free_count_out", _I32, 1), _on(dev, cu_new, "cu_new", _I32, B + 1),
        _on(dev, slot_map, "slot_map", _I32, 0), slots, wp, wn, st)
    if rc:
        _check(rc, "td_block_tables")


def _cache_ws(dev, ws, shape):
    """The buffer up to the end of the part for calls on small caches."""
    p, n = _ws(dev, ws)
    ws.check_cache(shape)
    return p, n - ws.tree_bytes


class Q4Cache:
    """One layer's K/V rows in 4 bits (td_q4_cache): k, v uint8 [pages][Hkv][page_size][64],
    scales uint8 [pages][Hkv][page_size][16] (K's 8 e4m3 scales of a token, then V's) and a
    block table [B][max_blocks], or without a table a contiguous cache."""

    def __init__(self, k, v, scales, block_table=None):
        for name, t, width in (("k", k, 64), ("v", v, 64), ("scales", scales, 16)):
            if t.dim() != 4 or t.shape[3] != width:
                raise ValueError(f"{name} must be [pages][kv heads][page size][{width}], got {tuple(t.shape)}")
            if t.shape[:3] != k.shape[:3]:
                raise ValueError(f"k and {name} differ: {tuple(k.shape)} and {tuple(t.shape)}")
        if block_table is not None and block_table.dim() != 2:
            raise ValueError("block_table must be [batch][max_blocks]")
        self.k, self.v, self.scales, self.block_table = k, v, scales, block_table
        self.num_pages, self.kv_heads, self.page_size = (int(x) for x in k.shape[:3])
        self.c = _Q4Cache(_dev(k, "k", torch.uint8), _dev(v, "v", torch.uint8),
                          _dev(scales, "scales", torch.uint8), self.num_pages, self.page_size,
                          _dev(block_table, "block_table", torch.int32, optional=True),
                          0 if block_table is None else int(block_table.shape[1]))
        self.device = k.get_device()
        for name, t in (("v", v), ("scales", scales), ("block_table", block_table)):
            if t is not None and t.get_device() != self.device:
                raise ValueError(f"k is on {k.device}, {name} on {t.device}")
        self.ref = ctypes.byref(self.c)
        self.fits = (self.device, self.kv_heads, None if block_table is None else int(block_table.shape[0]))

    check = Cache.check


def make_q4_cache(k, v, scales, block_table=None) -> Q4Cache:
    return Q4Cache(k, v, scales, block_table)


def _kind(cache, cls, call):
    if not isinstance(cache, cls):
        raise ValueError(f"{call} takes a {cls.__name__}, got {type(cache).__name__}")


def _new_tokens(name, kind, shape, cache, window, sinks, cu_new, q, seq_lens, out, ws, stream):
    dev, st = _launch(stream)
    _kind(cache, kind, name)
    wp, wn = _cache_ws(dev, ws, shape)
    if q.dim() != 3 or q.shape[1] != shape.num_q_heads or q.shape[2] != 128:
        raise ValueError(f"q must be [tokens][{shape.num_q_heads}][128], got {tuple(q.shape)}")
    nb, tokens = shape.batch, int(q.shape[0])
    n = tokens * shape.num_q_heads * 128
    rc = getattr(lib(), name)(
        shape, cache.check(shape, dev), int(window), int(sinks), tokens,
        None if cu_new is None else _on(dev, cu_new, "cu_new", _I32, nb + 1),
        _on(dev, q, "q", _BF16, n), _on(dev, seq_lens, "seq_lens", _I32, nb),
        _on(dev, out, "out", _BF16, n), wp, wn, st)
    if rc:
        _check(rc, name)


def td_window_attn(shape: Shape, cache: Cache, window, sinks, cu_new, q, seq_lens, out,
                   ws: Workspace = None, stream=None):
    """Attention of the new tokens q [tokens][Hq][128] over the cache with a sliding window
    (0: none) and the first `sinks` tokens; request b's rows are cu_new[b] .. cu_new[b + 1] - 1
    (None: one new token per request)."""
    _new_tokens("td_window_attn", Cache, shape, cache, window, sinks, cu_new, q, seq_lens, out, ws, stream)


def td_q4_attn(shape: Shape, cache: Q4Cache, window, sinks, cu_new, q, seq_lens, out,
               ws: Workspace = None, stream=None):
    """td_window_attn over a 4-bit cache."""
    _new_tokens("td_q4_attn", Q4Cache, shape, cache, window, sinks, cu_new, q, seq_lens, out, ws, stream)


def td_q4_sparse_attn(shape: Shape, cache: Q4Cache, q, seq_lens, idx, top_k, out,
                      ws: Workspace = None, stream=None):
    """One PPSA layer over a 4-bit cache: the persisted set idx [B][Hkv][top_k]."""
    dev, st = _launch(stream)
    _kind(cache, Q4Cache, "td_q4_sparse_attn")
    wp, wn = _cache_ws(dev, ws, shape)
    nb, k = shape.batch, int(top_k)
    n = nb * shape.num_q_heads * 128
    rc = lib().td_q4_sparse_attn(
        shape, cache.check(shape, dev), _on(dev, q, "q", _BF16, n),
        _on(dev, seq_lens, "seq_lens", _I32, nb),
        _on(dev, idx, "idx", _I32, nb * shape.num_kv_heads * k), k, _on(dev, out, "out", _BF16, n),
        wp, wn, st)
    if rc:
        _check(rc, "td_q4_sparse_attn")


def td_q4_append(shape: Shape, cache: Q4Cache, k_new, v_new, slot_map, stream=None):
    """New K/V rows [tokens][Hkv][128] into the 4-bit cache at slot_map [tokens]."""
    dev, st = _launch(stream)
    _kind(cache, Q4Cache, "td_q4_append")
    heads = shape.num_kv_heads
    ref = cache.ref
    if cache.device != dev or cache.kv_heads != heads:
        cache.check(shape, dev)
    pk, n, sk = _token_rows(dev, k_new, "k_new", heads)
    pv, nv, sv = _token_rows(dev, v_new, "v_new", heads)
    if n != nv or sk != sv:
        raise ValueError("k_new and v_new must have the same tokens and token stride")
    rc = lib().td_q4_append(shape, ref, n, pk, pv, sk, _on(dev, slot_map, "slot_map", _I32, n), st)
    if rc:
        _check(rc, "td_q4_append")


def td_weights_attn(shape: Shape, cache: Cache, fresh, q, seq_lens, weights, logits, out,
                    ws: Workspace = None, stream=None):
    """Full attention of one token per request that adds its probabilities, summed over each KV
    head's query heads, to weights [B][Hkv][max_seq_len] (the last `fresh` positions are set)."""
    dev, st = _launch(stream)
    _kind(cache, Cache, "td_weights_attn")
    wp, wn = _cache_ws(dev, ws, shape)
    nb, nq, N = shape.batch, shape.num_q_heads, shape.max_seq_len
    rc = lib().td_weights_attn(
        shape, cache.check(shape, dev), int(fresh), _on(dev, q, "q", _BF16, nb * nq * 128),
        _on(dev, seq_lens, "seq_lens", _I32, nb),
        _on(dev, weights, "weights", _F32, nb * shape.num_kv_heads * N),
        _on(dev, logits, "logits", _F32, nb * nq * N), _on(dev, out, "out", _BF16, nb * nq * 128),
        wp, wn, st)
    if rc:
        _check(rc, "td_weights_attn")


def td_evict(shape: Shape, cache: Cache, to: Cache, budget, sinks, recent, weights, weights_out,
             seq_lens, seq_lens_out, kept, ws: Workspace = None, stream=None):
    """Each KV head of a request with more than budget positions keeps its first `sinks`, its last
    `recent` and the heaviest others, as rows 0 .. budget - 1 of `to` (which may be cache);
    weights_out [B][Hkv][row], kept int32 [B][Hkv][budget]."""
    dev, st = _launch(stream)
    _kind(cache, Cache, "td_evict")
    _kind(to, Cache, "td_evict")
    wp, wn = _ws(dev, ws)
    nb, units, budget = shape.batch, shape.batch * shape.num_kv_heads, int(budget)
    if weights_out.dim() != 3:
        raise ValueError("weights_out must be [batch][kv heads][positions]")
    row = int(weights_out.shape[2])
    rc = lib().td_evict(
        shape, cache.check(shape, dev), to.check(shape, dev), budget, int(sinks), int(recent),
        _on(dev, weights, "weights", _F32, units * shape.max_seq_len),
        _on(dev, weights_out, "weights_out", _F32, units * row), row,
        _on(dev, seq_lens, "seq_lens", _I32, nb), _on(dev, seq_lens_out, "seq_lens_out", _I32, nb),
        _on(dev, kept, "kept", _I32, units * max(budget, 0)), wp, wn, st)
    if rc:
        _check(rc, "td_evict")


class _StepArgs:
    """Marshalled arguments of one decode step (kept alive while in use)."""

    def __init__(self, shape, modes, q, k_caches, v_caches, seq_lens, top_k, idx_buf, outs,
                 outs_f32, k_new=None, v_new=None):
        nq, nkv, nb = _sizes(shape)
        L = len(modes)
        if not (len(q) == len(k_caches) == len(v_caches) == len(outs) == L):
            raise ValueError("per-layer lists must have one entry per mode")
        if outs_f32 is not None and len(outs_f32) != L:
            raise ValueError("outs_f32 must have one entry per mode")
        self.L = L
        self.modes = (ctypes.c_int32 * max(L, 1))(*[int(m) for m in modes])
        self.q = _ptr_array(q, "q", torch.bfloat16, nq)
        self.k = _ptr_array(k_caches, "k_caches", torch.bfloat16, nkv)
        self.v = _ptr_array(v_caches, "v_caches", torch.bfloat16, nkv)
        self.outs = _ptr_array(outs, "outs", torch.bfloat16, nq)
        self.outs_f32 = (_ptr_array(outs_f32, "outs_f32", torch.float32, nq, optional=True)
                         if outs_f32 is not None else None)
        self.seq = _dev(seq_lens, "seq_lens", torch.int32, nb)
        needs_idx = any(int(m) != MODE_FULL for m in modes)
        self.idx = _dev(idx_buf, "idx_buf", torch.int32, nb * shape.num_kv_heads * top_k,
                        optional=not needs_idx)
        self.top_k = int(top_k)
        if (k_new is None) != (v_new is None):
            raise ValueError("k_new and v_new go together")
        self.append = k_new is not None
        if self.append:
            if not (len(k_new) == len(v_new) == L):
                raise ValueError("k_new / v_new need one entry per mode")
            n_new = nb * shape.num_kv_heads * shape.head_dim
            self.k_new = _ptr_array(k_new, "k_new", torch.bfloat16, n_new)
            self.v_new = _ptr_array(v_new, "v_new", torch.bfloat16, n_new)


def td_probe_layer_reads(shape: Shape, k_cache, v_cache, seq_lens, idx, top_k, sink,
                         stream=None):
    """Measurement aid: the K/V reads of one full (idx None) or sparse layer only."""
    nq, nkv, nb = _sizes(shape)
    st = lib().td_probe_layer_reads(
        ctypes.byref(shape), _dev(k_cache, "k_cache", torch.bfloat16, nkv),
        _dev(v_cache, "v_cache", torch.bfloat16, nkv), _dev(seq_lens, "seq_lens", torch.int32, nb),
        _dev(idx, "idx", torch.int32, nb * shape.num_kv_heads * max(int(top_k), 1), True),
        int(top_k), _dev(sink, "sink", torch.int32, 1), int(sink.numel()), _stream(stream))
    _check(st, "td_probe_layer_reads")


def td_kv_append(shape: Shape, k_cache, v_cache, k_new, v_new, seq_lens, stream=None):
    nq, nkv, nb = _sizes(shape)
    n_new = nb * shape.num_kv_heads * shape.head_dim
    st = lib().td_kv_append(
        ctypes.byref(shape), _dev(k_cache, "k_cache", torch.bfloat16, nkv),
        _dev(v_cache, "v_cache", torch.bfloat16, nkv), _dev(k_new, "k_new", torch.bfloat16, n_new),
        _dev(v_new, "v_new", torch.bfloat16, n_new), _dev(seq_lens, "seq_lens", torch.int32, nb),
        _stream(stream))
    _check(st, "td_kv_append")


def td_decode_step(shape: Shape, modes: Sequence[int], q, k_caches, v_caches, seq_lens, top_k,
                   idx_buf, outs, outs_f32=None, ws: Workspace = None, idx_valid=False,
                   stream=None, layer_events: Optional[Sequence] = None, k_new=None, v_new=None):
    """One decode step; with k_new / v_new (per-layer [B][Hkv][128] rows) the
    step also appends the new token to each layer's cache (td_decode_step_append)."""
    a = _StepArgs(shape, modes, q, k_caches, v_caches, seq_lens, top_k, idx_buf, outs, outs_f32,
                  k_new, v_new)
    ev = None
    if layer_events is not None:
        if len(layer_events) != a.L + 1:
            raise ValueError("layer_events needs num_layers + 1 events")
        for e in layer_events:
            if int(e.cuda_event) == 0:   # torch creates the CUDA event on first record
                e.record(_torch_stream(stream))
        ev =(ctypes.c_void_p * (a.L + 1))(*[int(e.cuda_event) for e in layer_events])
    if a.append:
        st = lib().td_decode_step_append(ctypes.byref(shape), a.L, a.modes, a.q, a.k, a.v, a.k_new,
                                         a.v_new, a.seq, a.top_k, a.idx, int(bool(idx_valid)),
                                         a.outs, a.outs_f32, ws.ptr, ws.nbytes, _stream(stream), ev)
        _check(st, "td_decode_step_append")
        return
    st = lib().td_decode_step(ctypes.byref(shape), a.L, a.modes, a.q, a.k, a.v, a.seq, a.top_k,
                              a.idx, int(bool(idx_valid)), a.outs, a.outs_f32, ws.ptr, ws.nbytes,
                              _stream(stream), ev)
    _check(st, "td_decode_step")


def _one_buffer(ts, name, n):
    """Device pointer of per-layer tensors that are consecutive slices of one
    buffer (layer l at the start + l * n values)."""
    base = ts[0].data_ptr()
    for l, t in enumerate(ts):
        if not t.is_cuda or t.dtype != torch.bfloat16 or t.numel() != n or \
                t.data_ptr() != base + 2 * n * l:
            raise ValueError(f"{name}: the layers must be consecutive slices of one bf16 buffer")
    return base


def _host_buffer(t, name, n):
    if t is None or t.is_cuda or t.dtype != torch.bfloat16 or t.numel() != n or \
            not t.is_contiguous():
        raise ValueError(f"{name}: one contiguous bf16 host tensor of {n} values expected")
    if not t.is_pinned():
        raise ValueError(f"{name}: the host tensor must be page-locked (pin_memory())")
    return t.data_ptr()


class Plan:
    """A decode step captured once into a CUDA graph (td_plan_create).  With
    q_host / out_host (page-locked host tensors of all layers' rows, [L][B][Hq][128])
    the step also copies the q rows in and the outputs back
    (td_plan_create_host); q and outs must then be slices of one device
    buffer each."""

    def __init__(self, shape: Shape, modes, q, k_caches, v_caches, seq_lens, top_k, idx_buf, outs,
                 outs_f32=None, ws: Workspace = None, idx_valid=False, k_new=None, v_new=None,
                 q_host=None, out_host=None):
        self._args = _StepArgs(shape, modes, q, k_caches, v_caches, seq_lens, top_k, idx_buf,
                               outs, outs_f32, k_new, v_new)
        self._keep = (q, k_caches, v_caches, seq_lens, idx_buf, outs, outs_f32, ws, k_new, v_new,
                      q_host, out_host)
        self._plan = ctypes.c_void_p(0)
        a = self._args
        if q_host is not None or out_host is not None:
            if a.append:
                raise ValueError("host q/out and KV append are separate plans")
            n = shape.batch * shape.num_q_heads * shape.head_dim
            qh = _host_buffer(q_host, "q_host", a.L * n)
            oh = _host_buffer(out_host, "out_host", a.L * n)
            st = lib().td_plan_create_host(
                ctypes.byref(self._plan), ctypes.byref(shape), a.L, a.modes, qh,
                _one_buffer(q, "q", n), a.k, a.v, a.seq, a.top_k, a.idx, int(bool(idx_valid)),
                _one_buffer(outs, "outs", n), a.outs_f32, oh, ws.ptr, ws.nbytes)
            _check(st, "td_plan_create_host")
            return
        if a.append:
            st = lib().td_plan_create_append(
                ctypes.byref(self._plan), ctypes.byref(shape), a.L, a.modes, a.q, a.k, a.v,
                a.k_new, a.v_new, a.seq, a.top_k, a.idx, int(bool(idx_valid)), a.outs, a.outs_f32,
                ws.ptr, ws.nbytes)
            _check(st, "td_plan_create_append")
            return
        st = lib().td_plan_create(ctypes.byref(self._plan), ctypes.byref(shape), a.L, a.modes,
                                  a.q, a.k, a.v, a.seq, a.top_k, a.idx, int(bool(idx_valid)),
                                  a.outs, a.outs_f32, ws.ptr, ws.nbytes)
        _check(st, "td_plan_create")

    def launch(self, stream=None):
        _check(lib().td_plan_launch(self._plan, _stream(stream)), "td_plan_launch")

    def close(self):
        if self._plan:
            lib().td_plan_destroy(self._plan)
            self._plan = ctypes.c_void_p(0)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def td_set_tuning(key: str, value: int):
    _check(lib().td_set_tuning(key.encode(), int(value)), f"td_set_tuning({key})")


def td_query_splits(shape: Shape, top_k: int, sparse: bool) -> int:
    return int(lib().td_query_splits(ctypes.byref(shape), int(top_k), int(bool(sparse))))


def td_kernel_name(shape: Shape, top_k: int, sparse: bool) -> str:
    return lib().td_kernel_name(ctypes.byref(shape), int(top_k), int(bool(sparse))).decode()
