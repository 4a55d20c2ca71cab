"""Python binding of libpagedkv (include/pagedkv.h): paged decode attention
and its cache-maintenance calls on B200 (sm_100a).

Argument marshalling only: tensors are passed to the C ABI as raw device
pointers with the current CUDA stream; every step of the computation runs in
the library's kernels. There is no fallback: importing this module fails if
the library has not been built (``python paged_kv_cache_417_b200/build.py``).

Cache tensors are [num_blocks, num_heads, block_size, head_dim] fp16/bf16
(see the header for the full contract).
"""
from __future__ import annotations

import array
import ctypes
import functools
import operator
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpagedkv.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python paged_kv_cache_417_b200/build.py` "
        "(nvcc, sm_100a). There is no non-CUDA fallback.")

_lib = ctypes.CDLL(LIB_PATH)

PA_OK, PA_ERR_INVALID_ARG, PA_ERR_UNSUPPORTED, PA_ERR_WORKSPACE, PA_ERR_CUDA = range(5)
PA_F16, PA_BF16, PA_F32, PA_FP8_E4M3 = 0, 1, 2, 3
PA_DEVERR_BLOCK_ID = 1
PA_DEVERR_CONTEXT_LEN = 2
PA_DEVERR_SLOT = 4
PA_DEVERR_TIMEOUT = 8
PA_DEVERR_COPY_PAIR = 16
PA_DEVERR_TREE = 32
PA_TREE_MAX_NODES = 1024
PA_MAX_LAYERS = 256

_DTYPE = {torch.float16: PA_F16, torch.bfloat16: PA_BF16, torch.float32: PA_F32}


class CacheDesc(ctypes.Structure):
    _fields_ = [("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int), ("io_dtype", ctypes.c_int)]


class Fp8Cache:
    """An fp8 (e4m3) K or V cache: a uint8 tensor [num_blocks, num_heads,
    block_size*head_dim + 4*block_size] whose (block, head) tiles hold
    block_size rows of head_dim codes and then one fp32 scale per row.
    ``io_dtype`` is the dtype of the query/key/value rows used with it."""

    def __init__(self, data, block_size, head_dim, io_dtype=torch.float16):
        if data.dtype != torch.uint8 or data.dim() != 3:
            raise ValueError("fp8 cache data must be uint8 [num_blocks, heads, tile bytes]")
        if data.shape[2] != block_size * head_dim + 4 * block_size:
            raise ValueError("tile bytes must be block_size*head_dim + 4*block_size")
        if io_dtype not in (torch.float16, torch.bfloat16):
            raise ValueError("io_dtype must be float16 or bfloat16")
        self.data, self.block_size, self.head_dim, self.io_dtype = data, block_size, head_dim, \
            io_dtype

    @classmethod
    def empty(cls, num_blocks, num_heads, block_size, head_dim, io_dtype=torch.float16,
              device="cuda"):
        data = torch.empty(num_blocks, num_heads, block_size * head_dim + 4 * block_size,
                           dtype=torch.uint8, device=device)
        return cls(data, block_size, head_dim, io_dtype)

    def data_ptr(self):
        return self.data.data_ptr()

    def is_contiguous(self):
        return self.data.is_contiguous()

    def is_pinned(self):
        return self.data.is_pinned()

    @property
    def is_cuda(self):
        return self.data.is_cuda

    @property
    def device(self):
        return self.data.device

    @property
    def shape(self):
        return self.data.shape


_P = ctypes.c_void_p
_i32 = ctypes.c_int32
_lib.pa_write_kv.restype = ctypes.c_int
_lib.pa_write_kv.argtypes = [_P, _P, _i32, _i32, _P, _P, _P, ctypes.POINTER(CacheDesc), _P, _P]
_lib.pa_decode_workspace_size.restype = ctypes.c_size_t
_lib.pa_decode_workspace_size.argtypes = [_i32, _i32, _i32, _i32, _i32]
_lib.pa_decode_partition_size.restype = _i32
_lib.pa_decode_partition_size.argtypes = [_i32, _i32, ctypes.POINTER(CacheDesc), _i32, _i32]
_lib.pa_decode.restype = ctypes.c_int
_lib.pa_decode.argtypes = [_P, ctypes.c_int, _P, _i32, _i32, _P, _P, ctypes.POINTER(CacheDesc),
                           _P, _i32, _P, _i32, ctypes.c_float, _i32, _P, ctypes.c_size_t, _P, _P]
_lib.pa_write_kv_decode.restype = ctypes.c_int
_lib.pa_write_kv_decode.argtypes = [_P, ctypes.c_int, _P, _P, _P, _i32, _i32, _P, _P,
                                    ctypes.POINTER(CacheDesc), _P, _i32, _P, _i32,
                                    ctypes.c_float, _i32, _P, ctypes.c_size_t, _P, _P]
_lib.pa_decode_noalloc.restype = ctypes.c_int
_lib.pa_decode_noalloc.argtypes = [_P, ctypes.c_int, _P, _i32, _i32, _P, _P,
                                   ctypes.POINTER(CacheDesc), _P, _i32, _P, _i32,
                                   ctypes.c_float, _i32, _P, _P]
_lib.pa_copy_blocks.restype = ctypes.c_int
_lib.pa_copy_blocks.argtypes = [ctypes.POINTER(_P), ctypes.POINTER(_P), _i32, _P, _i32,
                                ctypes.POINTER(CacheDesc), _P, _P]
_lib.pa_swap_blocks.restype = ctypes.c_int
_lib.pa_swap_blocks.argtypes = [ctypes.POINTER(_P), ctypes.POINTER(_P), ctypes.POINTER(CacheDesc),
                                ctypes.POINTER(_P), ctypes.POINTER(_P), ctypes.POINTER(CacheDesc),
                                _i32, _P, _i32, _P, _P]
_lib.pa_tree_mask.restype = ctypes.c_int
_lib.pa_tree_mask.argtypes = [_P, _P, _P, _P, _i32, _i32, _i32, _P, _P]
_lib.pa_tree_decode_workspace_size.restype = ctypes.c_size_t
_lib.pa_tree_decode_workspace_size.argtypes = [ctypes.POINTER(CacheDesc)]
_lib.pa_tree_decode.restype = ctypes.c_int
_lib.pa_tree_decode.argtypes = [_P, ctypes.c_int, _P, _i32, _i32, _i32, _P, _P,
                                ctypes.POINTER(CacheDesc), _P, _i32, _P, _P, _P, _i32,
                                ctypes.c_float, _P, ctypes.c_size_t, _P, _P]
_lib.pa_tree_accept.restype = ctypes.c_int
_lib.pa_tree_accept.argtypes = [_P, _P, _P, _P, _P, _P, _P, _i32, _i32, _i32, _P, _P]
_lib.pa_tree_compact.restype = ctypes.c_int
_lib.pa_tree_compact.argtypes = [_P, _P, _i32, ctypes.POINTER(CacheDesc), _P, _i32, _P, _P, _P,
                                 _i32, _i32, _P, _P]
_lib.pa_selftest_wait_timeout.restype = ctypes.c_int
_lib.pa_selftest_wait_timeout.argtypes = [_P, ctypes.c_uint32, _P]
_lib.pa_status_string.restype = ctypes.c_char_p
_lib.pa_status_string.argtypes = [ctypes.c_int]
_lib.pa_last_error.restype = ctypes.c_char_p
_lib.pa_last_error.argtypes = []
_lib.pa_version.restype = _i32
_lib.pa_version.argtypes = []

SIZE_MAX = ctypes.c_size_t(-1).value


class PagedKVError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        super().__init__(f"{_lib.pa_status_string(status).decode()}: {detail}")


def _check(status: int) -> None:
    if status != PA_OK:
        raise PagedKVError(status, _lib.pa_last_error().decode())


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def cache_desc(key_cache) -> CacheDesc:
    if isinstance(key_cache, Fp8Cache):
        nb, h, _ = key_cache.data.shape
        return CacheDesc(nb, key_cache.block_size, h, key_cache.head_dim, PA_FP8_E4M3,
                         _DTYPE[key_cache.io_dtype])
    if key_cache.dim() != 4:
        raise ValueError("cache must be [num_blocks, num_heads, block_size, head_dim]")
    nb, h, bs, d = key_cache.shape
    if key_cache.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError("cache dtype must be float16 or bfloat16")
    return CacheDesc(nb, bs, h, d, _DTYPE[key_cache.dtype], _DTYPE[key_cache.dtype])


def io_dtype(cache) -> torch.dtype:
    """dtype of the query/key/value rows used with a cache."""
    return cache.io_dtype if isinstance(cache, Fp8Cache) else cache.dtype


def _need(t, name: str, dtype=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _need_cache(c, name: str, like=None):
    if isinstance(c, Fp8Cache):
        _need(c.data, name)
        if like is not None and (not isinstance(like, Fp8Cache) or c.shape != like.shape):
            raise ValueError(f"{name} does not match the other cache")
        return
    _need(c, name)
    if like is not None and (isinstance(like, Fp8Cache) or c.dtype != like.dtype or
                             c.shape != like.shape):
        raise ValueError(f"{name} does not match the other cache")


def version() -> int:
    return int(_lib.pa_version())


def write_kv(key, value, slot_mapping, key_cache, value_cache, dev_err=None):
    """Store new tokens' K/V ([T, H, D]) at ``slot_mapping`` (int64 [T]) in
    the caches; negative slots are skipped."""
    _need_cache(key_cache, "key_cache")
    _need_cache(value_cache, "value_cache", key_cache)
    for t, n in ((key, "key"), (value, "value")):
        _need(t, n, io_dtype(key_cache))
    _need(slot_mapping, "slot_mapping", torch.int64)
    if key.shape != value.shape:
        raise ValueError("shape mismatch")
    desc = cache_desc(key_cache)
    _check(_lib.pa_write_kv(_ptr(key), _ptr(value), key.shape[0], key.shape[1],
                            _ptr(slot_mapping), _ptr(key_cache), _ptr(value_cache),
                            ctypes.byref(desc), _ptr(dev_err), _stream(key_cache)))


def decode_workspace_size(num_seqs, num_heads, head_dim, max_context_len, partition_size=0):
    n = _lib.pa_decode_workspace_size(num_seqs, num_heads, head_dim, max_context_len,
                                      partition_size)
    if n == SIZE_MAX:
        raise ValueError("invalid arguments to decode_workspace_size")
    return int(n)


def decode_partition_size(num_seqs, num_heads, cache, max_context_len, partition_size=0):
    """``cache``: a key cache (tensor or Fp8Cache) or a CacheDesc."""
    desc = cache if isinstance(cache, CacheDesc) else cache_desc(cache)
    n = _lib.pa_decode_partition_size(num_seqs, num_heads, ctypes.byref(desc),
                                      max_context_len, partition_size)
    if n < 0:
        raise ValueError("invalid arguments to decode_partition_size")
    return int(n)


def alloc_workspace(num_seqs, num_heads, head_dim, max_context_len, partition_size=0,
                    device="cuda"):
    """A decode workspace, zero-filled (its counter region must start at
    zero; every call leaves it so)."""
    n = decode_workspace_size(num_seqs, num_heads, head_dim, max_context_len, partition_size)
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=device)


def decode(out, query, key_cache, value_cache, block_tables, context_lens, max_context_len,
           scale, partition_size=0, workspace=None, dev_err=None):
    """out[s,h,:] = softmax(scale * q K^T) V over each sequence's cached
    tokens. ``out`` may be fp16, bf16 or fp32; ``workspace`` is allocated
    here when not given."""
    _need_cache(key_cache, "key_cache")
    _need_cache(value_cache, "value_cache", key_cache)
    _need(query, "query", io_dtype(key_cache))
    _need(block_tables, "block_tables", torch.int32)
    _need(context_lens, "context_lens", torch.int32)
    _need(out, "out")
    if out.dtype not in _DTYPE:
        raise ValueError("out dtype must be float16, bfloat16 or float32")
    if out.shape != query.shape:
        raise ValueError("shape mismatch")
    desc = cache_desc(key_cache)
    S, H, D = query.shape
    if workspace is None:
        workspace = alloc_workspace(S, H, D, int(max_context_len), partition_size,
                                    query.device)
    mb = block_tables.shape[1] if block_tables.dim() == 2 else 0
    _check(_lib.pa_decode(_ptr(out), _DTYPE[out.dtype], _ptr(query), S, H, _ptr(key_cache),
                          _ptr(value_cache), ctypes.byref(desc), _ptr(block_tables), mb,
                          _ptr(context_lens), int(max_context_len), float(scale),
                          int(partition_size), _ptr(workspace),
                          workspace.numel() * workspace.element_size(), _ptr(dev_err),
                          _stream(query)))
    return out


def write_kv_decode(out, query, key, value, key_cache, value_cache, block_tables,
                    context_lens, max_context_len, scale, partition_size=0, workspace=None,
                    dev_err=None):
    """:func:`write_kv` + :func:`decode` in one launch for a batch where
    every sequence appends one token: ``key``/``value`` [S, H, D] are the new
    rows, stored at position ``context_lens[s] - 1`` of each sequence (the
    slot its block table gives), and attention covers every token including
    them."""
    _need_cache(key_cache, "key_cache")
    _need_cache(value_cache, "value_cache", key_cache)
    _need(query, "query", io_dtype(key_cache))
    _need(key, "key", io_dtype(key_cache))
    _need(value, "value", io_dtype(key_cache))
    _need(block_tables, "block_tables", torch.int32)
    _need(context_lens, "context_lens", torch.int32)
    _need(out, "out")
    if out.dtype not in _DTYPE:
        raise ValueError("out dtype must be float16, bfloat16 or float32")
    if out.shape != query.shape or key.shape != value.shape or key.shape[0] != query.shape[0] \
            or key.shape[2] != query.shape[2]:
        raise ValueError("shape mismatch")
    desc = cache_desc(key_cache)
    S, H, D = query.shape
    if workspace is None:
        workspace = alloc_workspace(S, H, D, int(max_context_len), partition_size,
                                    query.device)
    mb = block_tables.shape[1] if block_tables.dim() == 2 else 0
    _check(_lib.pa_write_kv_decode(_ptr(out), _DTYPE[out.dtype], _ptr(query), _ptr(key),
                                   _ptr(value), S, H, _ptr(key_cache), _ptr(value_cache),
                                   ctypes.byref(desc), _ptr(block_tables), mb,
                                   _ptr(context_lens), int(max_context_len), float(scale),
                                   int(partition_size), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(),
                                   _ptr(dev_err), _stream(query)))
    return out


NOALLOC_SCRATCH_BYTES = 32 << 20


def decode_noalloc(out, query, key_cache, value_cache, block_tables, context_lens,
                   max_context_len, scale, partition_size=0, dev_err=None):
    """Like :func:`decode`, for callers that must not allocate device memory
    while decoding (for example an engine that has handed almost all device
    memory to its KV block pool): partial results of split contexts go to a
    fixed 32 MiB array inside the library instead of a workspace. A split
    call first clears the array's arrival counters on the current stream.
    Calls that overlap on the GPU share the array and race (their outputs are
    wrong, with no error); serialised calls are unaffected. The first call on
    a device looks up the array's address and should come before any stream
    capture."""
    _need_cache(key_cache, "key_cache")
    _need_cache(value_cache, "value_cache", key_cache)
    _need(query, "query", io_dtype(key_cache))
    _need(block_tables, "block_tables", torch.int32)
    _need(context_lens, "context_lens", torch.int32)
    _need(out, "out")
    if out.dtype not in _DTYPE:
        raise ValueError("out dtype must be float16, bfloat16 or float32")
    if out.shape != query.shape:
        raise ValueError("shape mismatch")
    desc = cache_desc(key_cache)
    S, H, D = query.shape
    mb = block_tables.shape[1] if block_tables.dim() == 2 else 0
    _check(_lib.pa_decode_noalloc(_ptr(out), _DTYPE[out.dtype], _ptr(query), S, H,
                                  _ptr(key_cache), _ptr(value_cache), ctypes.byref(desc),
                                  _ptr(block_tables), mb, _ptr(context_lens),
                                  int(max_context_len), float(scale), int(partition_size),
                                  _ptr(dev_err), _stream(query)))
    return out


def copy_blocks(key_caches, value_caches, block_mapping, dev_err=None):
    """Copy whole blocks (src, dst) = block_mapping[i] in every layer's K
    and V cache (copy-on-write)."""
    if len(key_caches) != len(value_caches) or not key_caches:
        raise ValueError("need the same, non-zero number of K and V caches")
    _need(block_mapping, "block_mapping", torch.int64)
    for c in list(key_caches) + list(value_caches):
        _need_cache(c, "cache", key_caches[0])
    desc = cache_desc(key_caches[0])
    L = len(key_caches)
    kp = (_P * L)(*[c.data_ptr() for c in key_caches])
    vp = (_P * L)(*[c.data_ptr() for c in value_caches])
    n = block_mapping.shape[0] if block_mapping.numel() else 0
    _check(_lib.pa_copy_blocks(kp, vp, L, _ptr(block_mapping), n, ctypes.byref(desc),
                               _ptr(dev_err), _stream(key_caches[0])))


def swap_blocks(src_key_caches, src_value_caches, dst_key_caches, dst_value_caches,
                block_mapping, dev_err=None):
    """Copy block ``block_mapping[i][0]`` of every source layer's K/V cache to
    block ``block_mapping[i][1]`` of the destination caches. Pools may be CUDA
    tensors or pinned CPU tensors (swap out / swap in); pageable CPU memory
    is refused. Runs on the current CUDA stream."""
    L = len(src_key_caches)
    groups = (src_key_caches, src_value_caches, dst_key_caches, dst_value_caches)
    if L == 0 or any(len(g) != L for g in groups):
        raise ValueError("need the same, non-zero number of caches in every list")
    for g in groups:
        for c in g:
            if not c.is_contiguous():
                raise ValueError("caches must be contiguous")
    if block_mapping.dtype != torch.int64 or not block_mapping.is_contiguous():
        raise ValueError("block_mapping must be a contiguous int64 tensor")
    sd, dd = cache_desc(src_key_caches[0]), cache_desc(dst_key_caches[0])
    arr = lambda cs: (_P * L)(*[c.data_ptr() for c in cs])  # noqa: E731
    n = block_mapping.shape[0] if block_mapping.numel() else 0
    dev = next((c.device for g in groups for c in g if c.is_cuda), None)
    stream = torch.cuda.current_stream(dev).cuda_stream
    _check(_lib.pa_swap_blocks(arr(src_key_caches), arr(src_value_caches), ctypes.byref(sd),
                               arr(dst_key_caches), arr(dst_value_caches), ctypes.byref(dd),
                               L, _ptr(block_mapping), n, _ptr(dev_err), stream))


# The tree calls are made once a layer or once a step on little data, so their
# checks are written for speed: device indices instead of device objects, the
# raw stream, no context manager unless the tensors are on another device than
# the current one.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda device: torch.cuda.current_stream(device).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_dtype_of, _shape_of = operator.attrgetter("dtype"), operator.attrgetter("shape")


def _call(fn, device: int, *args):
    """``fn(*args, stream)`` on the tensors' own device and its current stream."""
    if device == _current_device():
        status = fn(*args, _raw_stream(device))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _raw_stream(device))
    if status:
        _check(status)


def _refuse(t, name, dtype, device, shape):
    """The error for a tensor that is not what the two checks below want."""
    if not t.is_cuda:
        return ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        return ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        return ValueError(f"{name} must be contiguous")
    if device is not None and t.get_device() != device:
        return ValueError(f"{name} is on {t.device}, not cuda:{device}")
    return ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")


def _sized(t, name, dtype, device, shape):
    """A contiguous tensor of a type and shape on CUDA device `device`."""
    if t.dtype != dtype or t.shape != shape or t.get_device() != device or \
            not t.is_contiguous():
        raise _refuse(t, name, dtype, device, shape)


def _matrix(t, name, dtype, device, rows):
    """The same with two dimensions and any number of columns, which it returns."""
    shape = t.shape
    if len(shape) != 2 or shape[0] != rows or t.dtype != dtype or t.get_device() != device or \
            not t.is_contiguous():
        raise _refuse(t, name, dtype, device, (rows, "*"))
    return shape[1]


def _first(t, name, dtype, dim):
    """A contiguous CUDA tensor of a type and number of dimensions, the first
    of its call: its shape and device."""
    shape = t.shape
    if t.dtype != dtype or len(shape) != dim or not t.is_cuda or not t.is_contiguous():
        raise _refuse(t, name, dtype, None, ("*",) * dim)
    return shape, t.get_device()


def _err_ptr(dev_err, device):
    if dev_err is None:
        return None
    _need(dev_err, "dev_err", torch.int32)
    if dev_err.numel() < 1 or dev_err.get_device() != device:
        raise ValueError(f"dev_err must be an int32 word on cuda:{device}")
    return dev_err.data_ptr()


def _num_trees(tree_start, device):
    n = tree_start.numel()
    if n < 1:
        raise ValueError("tree_start must have one entry more than there are sequences")
    _sized(tree_start, "tree_start", torch.int32, device, (n,))
    return n - 1


def tree_mask(mask, depth, parents, tree_start, dev_err=None):
    """Ancestor bits and depths of drafted trees: ``parents`` int32 [N] (-1:
    a root) and ``tree_start`` int32 [S + 1] give ``mask`` int32 [N, W] (bit
    j % 32 of word j // 32: node j is the row's node or an ancestor of it)
    and ``depth`` int32 [N] (or None). Trees have at most 32 * W nodes. Rows
    of no tree are left as they were."""
    i32 = torch.int32
    (N,), dev = _first(parents, "parents", i32, 1)
    S = _num_trees(tree_start, dev)
    words = _matrix(mask, "mask", i32, dev, N)
    if depth is not None:
        _sized(depth, "depth", i32, dev, (N,))
    _call(_lib.pa_tree_mask, dev, mask.data_ptr(), _ptr(depth), parents.data_ptr(),
          tree_start.data_ptr(), S, N, words, _err_ptr(dev_err, dev))
    return mask, depth


def tree_decode_workspace_size(cache):
    """Bytes of workspace :func:`tree_decode` needs on the current device.
    ``cache``: a key cache (tensor or Fp8Cache) or a CacheDesc."""
    desc = cache if isinstance(cache, CacheDesc) else cache_desc(cache)
    n = _lib.pa_tree_decode_workspace_size(ctypes.byref(desc))
    if n == SIZE_MAX:
        raise ValueError("invalid arguments to tree_decode_workspace_size")
    return int(n)


def alloc_tree_workspace(cache):
    """A workspace for :func:`tree_decode` over ``cache`` (and any other cache
    of its head dimension), on its device. Needs no initialisation."""
    with torch.cuda.device(cache.device):
        return torch.empty(tree_decode_workspace_size(cache), dtype=torch.uint8,
                           device=cache.device)


@functools.lru_cache(maxsize=64)
def _desc_of(num_blocks, num_kv_heads, block_size, head_dim, code):
    """The descriptor of a 16-bit cache of these sizes, which nothing changes."""
    return CacheDesc(num_blocks, block_size, num_kv_heads, head_dim, code, code)


def tree_decode(out, query, key_cache, value_cache, block_tables, context_lens, tree_start, mask,
                scale, workspace=None, dev_err=None):
    """Attention of every node of every drafted tree: ``query`` and ``out``
    [N, H, D], nodes of sequence s at rows tree_start[s] .. tree_start[s+1]-1.
    Node i attends to the ``context_lens[s]`` cached tokens and to those nodes
    j of its own tree whose bit is set in ``mask`` [N, W] (see
    :func:`tree_mask`); node j's K/V are at position context_lens[s] + j.
    ``out`` may be fp16, bf16 or fp32; ``workspace`` is allocated here when
    not given."""
    i32 = torch.int32
    if isinstance(key_cache, Fp8Cache):
        _need_cache(key_cache, "key_cache")
        _need_cache(value_cache, "value_cache", key_cache)
        desc, row = cache_desc(key_cache), key_cache.io_dtype
        dev = key_cache.data.get_device()
        if value_cache.io_dtype != row or value_cache.data.get_device() != dev or \
                value_cache.block_size != key_cache.block_size:
            raise ValueError("value_cache does not match the other cache")
    else:
        row = key_cache.dtype
        if row not in (torch.float16, torch.bfloat16):
            raise ValueError("cache dtype must be float16 or bfloat16")
        shape, dev = _first(key_cache, "key_cache", row, 4)
        if isinstance(value_cache, Fp8Cache):
            raise ValueError("value_cache does not match the other cache")
        _sized(value_cache, "value_cache", row, dev, shape)
        code = _DTYPE[row]
        desc = _desc_of(*shape, code)
    (N, H, D), on = _first(query, "query", row, 3)
    if on != dev:
        raise ValueError(f"query is on {query.device}, not cuda:{dev}")
    kind = _DTYPE.get(out.dtype)
    if kind is None:
        raise ValueError("out dtype must be float16, bfloat16 or float32")
    _sized(out, "out", out.dtype, dev, (N, H, D))
    if D != desc.head_dim:
        raise ValueError(f"query and out must be [N, H, {desc.head_dim}]")
    S = _num_trees(tree_start, dev)
    _sized(context_lens, "context_lens", i32, dev, (S,))
    width = _matrix(block_tables, "block_tables", i32, dev, S)
    words = _matrix(mask, "mask", i32, dev, N)
    if workspace is None:
        workspace = alloc_tree_workspace(key_cache)
    elif not workspace.is_cuda or not workspace.is_contiguous() or workspace.get_device() != dev:
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    _call(_lib.pa_tree_decode, dev, out.data_ptr(), kind, query.data_ptr(), S, N, H,
          key_cache.data_ptr(), value_cache.data_ptr(), desc, block_tables.data_ptr(), width,
          context_lens.data_ptr(), tree_start.data_ptr(), mask.data_ptr(), words, float(scale),
          workspace.data_ptr(), workspace.nbytes, _err_ptr(dev_err, dev))
    return out


def tree_accept(accepted, accepted_lens, next_token, parents, tree_start, draft_tokens,
                target_tokens, dev_err=None):
    """The path of each tree that the model agrees with: from node 0 on to
    the lowest child whose token (``draft_tokens`` int64 [N]) is the one the
    model picked at the node (``target_tokens`` int64 [N]). Writes
    ``accepted`` int32 [S, max_path] (-1 past the path), ``accepted_lens``
    int32 [S] and ``next_token`` int64 [S], the model's token at the path's
    last node. A path is cut at max_path nodes."""
    i32, i64 = torch.int32, torch.int64
    (N,), dev = _first(parents, "parents", i32, 1)
    S = _num_trees(tree_start, dev)
    _sized(draft_tokens, "draft_tokens", i64, dev, (N,))
    _sized(target_tokens, "target_tokens", i64, dev, (N,))
    room = _matrix(accepted, "accepted", i32, dev, S)
    _sized(accepted_lens, "accepted_lens", i32, dev, (S,))
    _sized(next_token, "next_token", i64, dev, (S,))
    _call(_lib.pa_tree_accept, dev, accepted.data_ptr(), accepted_lens.data_ptr(),
          next_token.data_ptr(), parents.data_ptr(), tree_start.data_ptr(),
          draft_tokens.data_ptr(), target_tokens.data_ptr(), S, N, room,
          _err_ptr(dev_err, dev))
    return accepted, accepted_lens, next_token


def tree_compact(key_caches, value_caches, block_tables, context_lens, accepted, accepted_lens,
                 dev_err=None):
    """Move the accepted nodes' K/V rows behind the context, in place and in
    every layer: position context_lens[s] + accepted[s, k] to position
    context_lens[s] + k for k < accepted_lens[s]. A cache that layers share is
    moved once."""
    L = len(key_caches)
    if len(value_caches) != L or not L:
        raise ValueError("need the same, non-zero number of K and V caches")
    i32 = torch.int32
    like = key_caches[0]
    _need_cache(like, "cache")
    desc = cache_desc(like)
    caches = [*key_caches, *value_caches]
    if isinstance(like, Fp8Cache):
        if any(not isinstance(c, Fp8Cache) or c.block_size != like.block_size for c in caches):
            raise ValueError("cache does not match the other cache")
        caches, like = [c.data for c in caches], like.data
    elif any(isinstance(c, Fp8Cache) for c in caches):
        raise ValueError("cache does not match the other cache")
    # A list at a time: with 32 layers these checks are most of the call.
    T, dev = torch.Tensor, like.get_device()
    if set(map(_dtype_of, caches)) != {like.dtype} or set(map(T.get_device, caches)) != {dev} or \
            list(map(_shape_of, caches)).count(like.shape) != 2 * L:
        raise ValueError("cache does not match the other cache")
    if not all(map(T.is_contiguous, caches)):
        raise ValueError("cache must be contiguous")
    pointers = array.array("Q", map(T.data_ptr, caches))
    S = accepted.shape[0] if accepted.dim() else 0
    room = _matrix(accepted, "accepted", i32, dev, S)
    _sized(accepted_lens, "accepted_lens", i32, dev, (S,))
    _sized(context_lens, "context_lens", i32, dev, (S,))
    width = _matrix(block_tables, "block_tables", i32, dev, S)
    at = pointers.buffer_info()[0]
    _call(_lib.pa_tree_compact, dev, at, at + 8 * L, L, desc, block_tables.data_ptr(), width,
          context_lens.data_ptr(), accepted.data_ptr(), accepted_lens.data_ptr(), S, room,
          _err_ptr(dev_err, dev))


def selftest_wait_timeout(limit_us: int = 1000, device="cuda") -> int:
    """Run the bounded-wait self-test and return the device error bits it
    produced (PA_DEVERR_TIMEOUT expected)."""
    err = torch.zeros(1, dtype=torch.int32, device=device)
    _check(_lib.pa_selftest_wait_timeout(_ptr(err), int(limit_us),
                                         torch.cuda.current_stream(err.device).cuda_stream))
    torch.cuda.synchronize(err.device)
    return int(err.item())
