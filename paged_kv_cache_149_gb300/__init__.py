"""Python binding of libpa.so: paged KV-cache decode attention on GB300 (sm_103a).

Argument marshalling only.  Every computation runs in the library's CUDA kernels (or,
for the block pool, its C++ host code); PyTorch supplies device memory and streams.
The functions take torch tensors, check dtypes/devices/shapes, pass raw pointers and
the current CUDA stream to the C ABI (include/pa.h) and raise ``PagedAttentionError``
on a negative status.  If libpa.so is missing the import of this package still works
but every call raises: there is no fallback path.

Layouts (row-major):
    q, out        [num_seqs, num_q_heads, head_dim]            fp16 / bf16
    k_cache       [num_blocks, num_kv_heads, block_size, head_dim]
    v_cache       [num_blocks, num_kv_heads, block_size, head_dim]
    block_tables  [num_seqs, max_blocks_per_seq] int32
    context_lens  [num_seqs] int32
    key, value    [num_tokens, num_kv_heads, head_dim]
    slot_mapping  [num_tokens] int64
    block_mapping [num_pairs, 2] int32
"""
import ctypes
import functools
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpa.so")

PA_OK = 0
PA_ERR_ARG = -1
PA_ERR_WORKSPACE = -2
PA_ERR_CUDA = -3
PA_ERR_POOL_EXHAUSTED = -4
PA_ERR_UNKNOWN_SEQ = -5
PA_ERR_WRONG_TIER = -6

DEVERR_BAD_BLOCK = 0x1
DEVERR_BAD_CONTEXT = 0x2
DEVERR_BAD_SLOT = 0x4
DEVERR_BAD_PAIR = 0x8
DEVERR_TIMEOUT = 0x10
DEVERR_NO_BLOCKS = 0x20
DEVERR_BAD_PROBS = 0x40

PA_FP16 = 0
PA_BF16 = 1
PA_FP8_E4M3 = 2
PA_FP32 = 3

_c = ctypes
_vp, _i32, _i64, _sz, _f32 = _c.c_void_p, _c.c_int, _c.c_int64, _c.c_size_t, _c.c_float

# name -> (restype, argtypes); mirrors include/pa.h
SIGNATURES = {
    "pa_reshape_and_cache": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _vp]),
    "pa_decode": (_i32, [_vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32, _i32,
                         _f32, _vp, _vp, _sz, _i32, _vp]),
    "pa_decode_append": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32,
                                _i32, _i32, _f32, _vp, _vp, _sz, _i32, _vp]),
    "pa_decode_fp8": (_i32, [_vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32, _i32,
                             _f32, _f32, _f32, _vp, _vp, _sz, _i32, _vp]),
    "pa_decode_append_fp8": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32,
                                    _i32, _i32, _i32, _f32, _f32, _f32, _vp, _vp, _sz, _i32,
                                    _vp]),
    "pa_reshape_and_cache_fp8": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                                        _f32, _f32, _i32, _vp]),
    "pa_reshape_and_cache_int4": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32,
                                         _i32, _i32, _i32, _vp]),
    "pa_decode_int4": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32,
                              _i32, _i32, _f32, _vp, _vp, _sz, _i32, _vp]),
    "pa_decode_append_int4": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32,
                                     _i32, _i32, _i32, _i32, _i32, _f32, _vp, _vp, _sz, _i32,
                                     _vp]),
    "pa_copy_blocks_int4": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp]),
    "pa_swap_blocks_int4": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32,
                                   _i32, _i32, _i32, _vp]),
    "pa_build_step": (_i32, [_vp, _vp, _i32, _vp, _i32, _vp, _vp, _i32, _i32, _i32, _vp, _i32,
                             _vp, _vp, _vp]),
    "pa_append_fp8_block": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _i32, _i32,
                                   _i32, _i32, _i32, _i32, _i32, _vp]),
    "pa_decode_fp8_block": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32,
                                   _i32, _i32, _i32, _f32, _vp, _vp, _sz, _i32, _vp]),
    "pa_prefill_fp8_block": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _i32, _i32,
                                    _i32, _i32, _i32, _i32, _i32, _i32, _f32, _vp, _i32, _vp]),
    "pa_copy_blocks_fp8_block": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                                        _vp]),
    "pa_swap_blocks_fp8_block": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32,
                                        _i32, _i32, _i32, _i32, _vp]),
    "pa_prefill": (_i32, [_vp, _vp, _vp, _vp, _i32, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                          _i32, _i32, _f32, _vp, _i32, _vp]),
    "pa_rotary_frequencies": (_i32, [_vp, _i32, _vp]),
    "pa_rotary": (_i32, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i32, _i32, _f32,
                         _i32, _i32, _i32, _i32, _i32, _i32, _vp]),
    "pa_rotary_append": (_i32, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i32,
                                _vp, _vp, _vp, _i32, _i32, _f32, _i32, _i32, _i32, _i32, _i32, _i32,
                                _i32, _i32, _vp]),
    "pa_decode_drafts": (_i32, [_vp, _vp, _vp, _vp, _i32, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                                _i32, _i32, _f32, _vp, _vp, _sz, _i32, _vp]),
    "pa_cross": (_i32, [_vp, _vp, _vp, _vp, _i32, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32,
                        _i32, _f32, _vp, _vp, _sz, _i32, _vp]),
    "pa_split_workspace_size": (_sz, [_i32, _i32, _i32]),
    "pa_verify_drafts": (_i32, [_vp, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i32, _i32, _i32, _vp,
                                _vp, _vp, _i32, _vp]),
    "pa_decode_workspace_size": (_sz, [_i32, _i32, _i32]),
    "pa_decode_timeline": (_i32, [_vp, _sz]),
    "pa_decode_fixed_scratch": (_i32, [_vp, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _i32,
                                       _i32, _f32, _vp, _i32, _vp]),
    "pa_copy_blocks": (_i32, [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _vp]),
    "pa_swap_blocks": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
                              _vp]),
    "pa_check_block_mapping": (_i32, [_vp, _i32, _i32]),
    "pa_get_device_error": (_i32, [_vp, _c.POINTER(_c.c_uint32)]),
    "pa_status_string": (_c.c_char_p, [_i32]),
    "pa_pool_create": (_vp, [_i32, _i32, _vp]),
    "pa_pool_create_tiered": (_vp, [_i32, _i32, _vp, _i32, _vp]),
    "pa_pool_destroy": (None, [_vp]),
    "pa_pool_allocate": (_i32, [_vp, _i64, _i32]),
    "pa_pool_append_slot": (_i32, [_vp, _i64, _c.POINTER(_i64), _c.POINTER(_c.c_int32),
                                   _c.POINTER(_c.c_int32)]),
    "pa_pool_fork": (_i32, [_vp, _i64, _i64]),
    "pa_pool_truncate": (_i32, [_vp, _i64, _i32]),
    "pa_pool_free": (_i32, [_vp, _i64]),
    "pa_pool_block_table": (_i32, [_vp, _i64, _vp, _i32]),
    "pa_pool_context_len": (_i32, [_vp, _i64]),
    "pa_pool_slots": (_i32, [_vp, _i64, _i32, _i32, _vp]),
    "pa_pool_num_free": (_i32, [_vp]),
    "pa_pool_free_list": (_i32, [_vp, _vp, _i32]),
    "pa_pool_refcount": (_i32, [_vp, _c.c_int32]),
    "pa_pool_swap_out": (_i32, [_vp, _vp, _i32, _vp, _i32]),
    "pa_pool_swap_in": (_i32, [_vp, _vp, _i32, _vp, _i32]),
    "pa_pool_is_swapped": (_i32, [_vp, _i64]),
    "pa_pool_num_free_cpu": (_i32, [_vp]),
    "pa_pool_cpu_free_list": (_i32, [_vp, _vp, _i32]),
    "pa_pool_cpu_refcount": (_i32, [_vp, _c.c_int32]),
    "pa_pool_allocate_prefix": (_i32, [_vp, _i64, _vp, _i32, _vp, _i32, _c.POINTER(_c.c_int)]),
    "pa_pool_num_cached": (_i32, [_vp]),
    "pa_pool_table_width": (_i32, [_vp, _i32, _vp]),
    "pa_pool_allocate_prefix_batch": (_i32, [_vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                             _i32, _c.POINTER(_c.c_int)]),
    "pa_pool_allocate_hashed_batch": (_i32, [_vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i32,
                                             _c.POINTER(_c.c_int)]),
    "pa_pool_free_batch": (_i32, [_vp, _vp, _i32]),
    "pa_pool_block_digest": (_i32, [_vp, _c.c_int32, _vp]),
    "pa_prefix_block_hashes": (_i32, [_vp, _i32, _i32, _vp, _i32, _vp, _i32]),
    "pa_sha256": (_i32, [_vp, _sz, _vp]),
}

_lib = None


class PagedAttentionError(RuntimeError):
    def __init__(self, status, what=""):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})" if what else status_string(status))


class PoolExhausted(PagedAttentionError):
    pass


class UnknownSequence(PagedAttentionError):
    pass


class WrongTier(PagedAttentionError):
    pass


def lib():
    """The loaded libpa.so (ctypes), with argument types set.  Raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build it with `python -m paged_kv_cache_149_gb300.build` "
                "(nvcc, sm_103a).  There is no CPU or PyTorch fallback.")
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(l, name)
            f.restype = res
            f.argtypes = args
        _lib = l
    return _lib


def status_string(status):
    return lib().pa_status_string(int(status)).decode()


def _check(status, what):
    if status < 0:
        if status == PA_ERR_POOL_EXHAUSTED:
            raise PoolExhausted(status, what)
        if status == PA_ERR_UNKNOWN_SEQ:
            raise UnknownSequence(status, what)
        if status == PA_ERR_WRONG_TIER:
            raise WrongTier(status, what)
        raise PagedAttentionError(status, what)
    return status


def _switch_to(dev):
    """The device to make current for a call on tensors of `dev`, or None when it already
    is (the library works on the current device: its SM count, error word and scratch)."""
    import torch
    if dev is None or dev.type != "cuda" or dev.index is None:
        return None
    return None if dev.index == torch.cuda.current_device() else dev


def _runs_on(pick):
    """Decorator: run the call with the device `pick(*args, **kw)` current."""
    def deco(fn):
        @functools.wraps(fn)
        def wrapped(*args, **kw):
            dev = _switch_to(pick(*args, **kw))
            if dev is None:
                return fn(*args, **kw)
            import torch
            with torch.cuda.device(dev):
                return fn(*args, **kw)
        return wrapped
    return deco


# the device of the call's first tensor argument
_on_first = _runs_on(lambda t, *args, **kw: t.device)


def _pool_device(src, dst, *args, device=None, **kw):
    """The device of a copy between pools that may be pinned CPU memory."""
    import torch
    if device is not None:
        return torch.device(device)
    firsts = (src[0], dst[0]) if isinstance(src, (tuple, list)) else (src, dst)
    return next((t.device for t in firsts if t.is_cuda), None)


class Launch:
    """A library call whose arguments were checked and marshalled once (``plan=True`` on
    the decode step functions, decode_fp8_block, the prefills, reshape_and_cache,
    append_fp8_block, build_step, rotary, rotary_append, decode_drafts, cross and verify_drafts): ``run(stream)`` issues it again on ``stream`` over the
    same buffers, whose contents may change between runs.  For serving loops that launch
    the same step shape many times; the per-call cost is one foreign call.  The marshalled
    arguments are raw device addresses, so the Launch holds a reference to every tensor
    they point into (a workspace the call created included): none is freed, and its
    memory reused, while the Launch can still run.  Drop the Launch only after its last
    run has finished, or ordered before later work on the stream it ran on.  A run makes
    the planned tensors' device current if another one is."""

    def __init__(self, name, args, out, keep=()):
        self._fn = getattr(lib(), name)
        self._name = name
        self._args = args
        self._keep = tuple(keep)
        self.out = out
        self.device = out.device

    def run(self, stream):
        dev = _switch_to(self.device)
        if dev is None:
            st = self._fn(*self._args, stream.cuda_stream)
        else:
            import torch
            with torch.cuda.device(dev):
                st = self._fn(*self._args, stream.cuda_stream)
        if st < 0:
            _check(st, self._name)
        return self.out


# ----------------------------------------------------------------- device calls

def _dtype_code(t):
    import torch
    if t.dtype == torch.float16:
        return PA_FP16
    if t.dtype == torch.bfloat16:
        return PA_BF16
    raise TypeError(f"unsupported dtype {t.dtype}; expected float16 or bfloat16")


def _cache_code(t):
    """dtype code of a K/V cache tensor: 16-bit floats, or FP8 E4M3 codes (uint8 or
    torch.float8_e4m3fn)."""
    import torch
    if t.dtype in (torch.uint8, getattr(torch, "float8_e4m3fn", torch.uint8)):
        return PA_FP8_E4M3
    return _dtype_code(t)


def _stream_ptr(stream, device):
    import torch
    s = torch.cuda.current_stream(device) if stream is None else stream
    return s.cuda_stream


def _need(cond, msg):
    if not cond:
        raise ValueError(msg)


def _host_out(arr, dtype, size, name):
    """A caller's host array the library writes `size` elements of: a writeable C-contiguous
    NumPy array of `dtype` with room for them."""
    import numpy as np
    # (messages are formatted only on failure: these checks run on every serving step)
    if not (isinstance(arr, np.ndarray) and arr.dtype == dtype and arr.flags.c_contiguous
            and arr.flags.writeable):
        raise ValueError(f"{name} must be a writeable C-contiguous {np.dtype(dtype).name} array")
    if arr.size < size:
        raise ValueError(f"{name} holds {arr.size} entries, {size} needed")
    return arr


def _dev(t, name, dtype=None):
    if not (t.is_cuda and t.is_contiguous() and (dtype is None or t.dtype == dtype)):
        _need(t.is_cuda, f"{name} must be a CUDA tensor")
        _need(t.is_contiguous(), f"{name} must be contiguous")
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


@_on_first
def reshape_and_cache(key, value, k_cache, v_cache, slot_mapping, stream=None, plan=False):
    """k_cache[slot // B, h, slot % B] = key[i, h] (and V) for every slot >= 0.  plan=True
    returns a Launch (whose run writes the rows the buffers hold then) instead of writing."""
    import torch
    n, hkv, d = key.shape
    nb, hkv2, bs, d2 = k_cache.shape
    _need(value.shape == key.shape and v_cache.shape == k_cache.shape, "shape mismatch")
    _need(hkv == hkv2 and d == d2 and slot_mapping.shape == (n,), "shape mismatch")
    _need(key.dtype == value.dtype == k_cache.dtype == v_cache.dtype, "dtype mismatch")
    args = (_dev(key, "key"), _dev(value, "value"), _dev(k_cache, "k_cache"),
            _dev(v_cache, "v_cache"), _dev(slot_mapping, "slot_mapping", torch.int64), n, nb, hkv,
            d, bs, _dtype_code(key))
    if plan:
        return Launch("pa_reshape_and_cache", args, k_cache,
                      keep=(key, value, v_cache, slot_mapping))
    st = lib().pa_reshape_and_cache(*args, _stream_ptr(stream, key.device))
    _check(st, "pa_reshape_and_cache")


def decode_workspace_size(num_q_heads, num_kv_heads, head_dim):
    """Bytes of workspace pa_decode needs on the current device."""
    n = lib().pa_decode_workspace_size(num_q_heads, num_kv_heads, head_dim)
    if n == 0:
        raise PagedAttentionError(PA_ERR_ARG, "pa_decode_workspace_size")
    return n


def decode_timeline(buffer=None):
    """Diagnostics (pa_decode_timeline): while `buffer` is set -- a device int64 tensor of
    at least SM count x 8 x 3 entries -- every 16-bit decode launch from this thread writes
    its warps' phase stamps into it, [cta][warp][k]; None clears the setting."""
    if buffer is None:
        _check(lib().pa_decode_timeline(None, 0), "pa_decode_timeline")
        return
    import torch
    if buffer.dtype != torch.int64 or not buffer.is_cuda or not buffer.is_contiguous():
        raise PagedAttentionError(PA_ERR_ARG, "pa_decode_timeline: a contiguous device int64 tensor")
    _check(lib().pa_decode_timeline(buffer.data_ptr(), buffer.numel() * 8), "pa_decode_timeline")


def make_workspace(num_q_heads, num_kv_heads, head_dim, device=None):
    import torch
    return torch.empty(decode_workspace_size(num_q_heads, num_kv_heads, head_dim),
                       dtype=torch.uint8, device=device or "cuda")


def _scratch(num_q_heads, num_kv_heads, head_dim, device, stream):
    """A workspace for one call launched on `stream`, allocated on that stream: the caching
    allocator then reuses its memory, once the call returns and the tensor is dropped, only
    for work ordered after the call on that stream."""
    import torch
    if stream is None:
        return make_workspace(num_q_heads, num_kv_heads, head_dim, device)
    with torch.cuda.stream(stream):
        return make_workspace(num_q_heads, num_kv_heads, head_dim, device)


@_on_first
def decode(q, k_cache, v_cache, block_tables, context_lens, scale, out=None, workspace=None,
           stream=None):
    """Paged decode attention; returns ``out`` [num_seqs, num_q_heads, head_dim]."""
    import torch
    n, hq, d = q.shape
    nb, hkv, bs, d2 = k_cache.shape
    _need(v_cache.shape == k_cache.shape and d == d2, "shape mismatch")
    _need(block_tables.dim() == 2 and block_tables.shape[0] == n, "block_tables must be [num_seqs, T]")
    _need(context_lens.shape == (n,), "context_lens must be [num_seqs]")
    _need(q.dtype == k_cache.dtype == v_cache.dtype, "dtype mismatch")
    if out is None:
        out = torch.empty_like(q)
    _need(out.shape == q.shape and out.dtype == q.dtype, "out must match q")
    if workspace is None:
        workspace = _scratch(hq, hkv, d, q.device, stream)
    st = lib().pa_decode(
        _dev(q, "q"), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
        _dev(block_tables, "block_tables", torch.int32), block_tables.shape[1],
        _dev(context_lens, "context_lens", torch.int32), n, hq, hkv, d, bs, nb, float(scale),
        _dev(out, "out"), _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _dtype_code(q), _stream_ptr(stream, q.device))
    _check(st, "pa_decode")
    return out


@_on_first
def decode_append(q, key_new, value_new, k_cache, v_cache, block_tables, context_lens, scale,
                  out=None, workspace=None, stream=None, plan=False):
    """One decode step in one kernel: writes each sequence's newest token (``key_new`` /
    ``value_new`` [num_seqs, num_kv_heads, head_dim], at position context_lens[s] - 1) into
    the caches and returns attention over contexts that include it.  Same results as
    reshape_and_cache into those slots followed by decode.  plan=True returns a Launch
    instead of launching."""
    import torch
    n, hq, d = q.shape
    nb, hkv, bs, d2 = k_cache.shape
    _need(v_cache.shape == k_cache.shape and d == d2, "shape mismatch")
    _need(key_new.shape == (n, hkv, d) and value_new.shape == (n, hkv, d),
          "key_new / value_new must be [num_seqs, num_kv_heads, head_dim]")
    _need(block_tables.dim() == 2 and block_tables.shape[0] == n, "block_tables must be [num_seqs, T]")
    _need(context_lens.shape == (n,), "context_lens must be [num_seqs]")
    _need(q.dtype == k_cache.dtype == v_cache.dtype == key_new.dtype == value_new.dtype,
          "dtype mismatch")
    if out is None:
        out = torch.empty_like(q)
    _need(out.shape == q.shape and out.dtype == q.dtype, "out must match q")
    if workspace is None:
        workspace = _scratch(hq, hkv, d, q.device, stream)
    args = (_dev(q, "q"), _dev(key_new, "key_new"), _dev(value_new, "value_new"),
            _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
            _dev(block_tables, "block_tables", torch.int32), block_tables.shape[1],
            _dev(context_lens, "context_lens", torch.int32), n, hq, hkv, d, bs, nb, float(scale),
            _dev(out, "out"), _dev(workspace, "workspace"),
            workspace.numel() * workspace.element_size(), _dtype_code(q))
    if plan:
        return Launch("pa_decode_append", args, out,
                      keep=(q, key_new, value_new, k_cache, v_cache, block_tables,
                            context_lens, out, workspace))
    _check(lib().pa_decode_append(*args, _stream_ptr(stream, q.device)), "pa_decode_append")
    return out


def _fp8_cache(t, name):
    import torch
    if t.dtype not in (torch.uint8, getattr(torch, "float8_e4m3fn", torch.uint8)):
        raise ValueError(f"{name} must hold E4M3 codes (uint8 or float8_e4m3fn), got {t.dtype}")
    return _dev(t, name)


@_on_first
def reshape_and_cache_fp8(key, value, k_cache, v_cache, slot_mapping, k_scale, v_scale,
                          stream=None):
    """FP8 cache write: k_cache[slot // B, h, slot % B] = E4M3(key[i, h] / k_scale) (and V)."""
    import torch
    n, hkv, d = key.shape
    nb, hkv2, bs, d2 = k_cache.shape
    _need(value.shape == key.shape and v_cache.shape == k_cache.shape, "shape mismatch")
    _need(hkv == hkv2 and d == d2 and slot_mapping.shape == (n,), "shape mismatch")
    _need(key.dtype == value.dtype, "dtype mismatch")
    st = lib().pa_reshape_and_cache_fp8(
        _dev(key, "key"), _dev(value, "value"), _fp8_cache(k_cache, "k_cache"),
        _fp8_cache(v_cache, "v_cache"), _dev(slot_mapping, "slot_mapping", torch.int64), n, nb,
        hkv, d, bs, float(k_scale), float(v_scale), _dtype_code(key),
        _stream_ptr(stream, key.device))
    _check(st, "pa_reshape_and_cache_fp8")


@_on_first
def decode_fp8(q, k_cache, v_cache, block_tables, context_lens, scale, k_scale, v_scale,
               out=None, workspace=None, stream=None):
    """Paged decode over FP8 E4M3 blocks (codes times k_scale / v_scale); q and out are
    fp16 or bf16."""
    import torch
    n, hq, d = q.shape
    nb, hkv, bs, d2 = k_cache.shape
    _need(v_cache.shape == k_cache.shape and d == d2, "shape mismatch")
    _need(block_tables.dim() == 2 and block_tables.shape[0] == n, "block_tables must be [num_seqs, T]")
    _need(context_lens.shape == (n,), "context_lens must be [num_seqs]")
    if out is None:
        out = torch.empty_like(q)
    _need(out.shape == q.shape and out.dtype == q.dtype, "out must match q")
    if workspace is None:
        workspace = _scratch(hq, hkv, d, q.device, stream)
    st = lib().pa_decode_fp8(
        _dev(q, "q"), _fp8_cache(k_cache, "k_cache"), _fp8_cache(v_cache, "v_cache"),
        _dev(block_tables, "block_tables", torch.int32), block_tables.shape[1],
        _dev(context_lens, "context_lens", torch.int32), n, hq, hkv, d, bs, nb, float(scale),
        float(k_scale), float(v_scale), _dev(out, "out"), _dev(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _dtype_code(q), _stream_ptr(stream, q.device))
    _check(st, "pa_decode_fp8")
    return out


@_on_first
def decode_append_fp8(q, key_new, value_new, k_cache, v_cache, block_tables, context_lens,
                      scale, k_scale, v_scale, out=None, workspace=None, stream=None, plan=False):
    """One FP8 decode step in one kernel: each sequence's newest K/V row is quantised into
    its slot at position ctx - 1 (read from the block tables) and attended (= bit for bit
    reshape_and_cache_fp8 + decode_fp8).  plan=True returns a Launch instead of launching."""
    import torch
    n, hq, d = q.shape
    nb, hkv, bs, d2 = k_cache.shape
    _need(v_cache.shape == k_cache.shape and d == d2, "shape mismatch")
    _need(key_new.shape == (n, hkv, d) and value_new.shape == key_new.shape, "key_new must be [n, Hkv, d]")
    _need(key_new.dtype == value_new.dtype == q.dtype, "dtype mismatch")
    _need(block_tables.dim() == 2 and block_tables.shape[0] == n, "block_tables must be [num_seqs, T]")
    _need(context_lens.shape == (n,), "context_lens must be [num_seqs]")
    if out is None:
        out = torch.empty_like(q)
    _need(out.shape == q.shape and out.dtype == q.dtype, "out must match q")
    if workspace is None:
        workspace = _scratch(hq, hkv, d, q.device, stream)
    args = (_dev(q, "q"), _dev(key_new, "key_new"), _dev(value_new, "value_new"),
            _fp8_cache(k_cache, "k_cache"), _fp8_cache(v_cache, "v_cache"),
            _dev(block_tables, "block_tables", torch.int32), block_tables.shape[1],
            _dev(context_lens, "context_lens", torch.int32), n, hq, hkv, d, bs, nb, float(scale),
            float(k_scale), float(v_scale), _dev(out, "out"), _dev(workspace, "workspace"),
            workspace.numel() * workspace.element_size(), _dtype_code(q))
    if plan:
        return Launch("pa_decode_append_fp8", args, out,
                      keep=(q, key_new, value_new, k_cache, v_cache, block_tables,
                            context_lens, out, workspace))
    _check(lib().pa_decode_append_fp8(*args, _stream_ptr(stream, q.device)), "pa_decode_append_fp8")
    return out


@_on_first
def prefill(q, k_cache, v_cache, block_tables, context_lens, query_start, scale,
            max_query_len, out=None, stream=None, plan=False):
    """Causal attention of each sequence's newest tokens (q rows query_start[s] ..
    query_start[s+1]-1, at positions ctx - q_len .. ctx - 1, their K/V already in the cache)
    over its paged context; returns ``out`` shaped like q.  plan=True returns a Launch
    instead of launching: its runs read the tables, lengths and offsets the buffers hold
    then, so max_query_len must stay an upper bound of the query counts."""
    import torch
    ntok, hq, d = q.shape
    nb, hkv, bs, d2 = k_cache.shape
    n = context_lens.shape[0]
    _need(v_cache.shape == k_cache.shape and d == d2, "shape mismatch")
    _need(block_tables.dim() == 2 and block_tables.shape[0] == n, "block_tables must be [num_seqs, T]")
    _need(query_start.shape == (n + 1,), "query_start must be [num_seqs + 1]")
    _need(q.dtype == k_cache.dtype == v_cache.dtype, "dtype mismatch")
    if out is None:
        out = torch.empty_like(q)
    _need(out.shape == q.shape and out.dtype == q.dtype, "out must match q")
    args = (_dev(q, "q"), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
            _dev(block_tables, "block_tables", torch.int32), block_tables.shape[1],
            _dev(context_lens, "context_lens", torch.int32),
            _dev(query_start, "query_start", torch.int32), n, int(max_query_len), hq, hkv, d, bs,
            nb, float(scale), _dev(out, "out"), _dtype_code(q))
    if plan:
        return Launch("pa_prefill", args, out,
                      keep=(q, k_cache, v_cache, block_tables, context_lens, query_start))
    st = lib().pa_prefill(*args, _stream_ptr(stream, q.device))
    _check(st, "pa_prefill")
    return out


@_on_first
def decode_fixed_scratch(q, k_cache, v_cache, block_tables, context_lens, scale, out=None,
                         stream=None):
    """Paged decode that allocates nothing on the device: its scratch is a fixed array
    inside the library (see pa_decode_fixed_scratch in include/pa.h).  For callers that
    cannot allocate device memory; calls whose GPU work overlaps race on that scratch."""
    import torch
    n, hq, d = q.shape
    nb, hkv, bs, d2 = k_cache.shape
    _need(v_cache.shape == k_cache.shape and d == d2, "shape mismatch")
    _need(block_tables.dim() == 2 and block_tables.shape[0] == n, "block_tables must be [num_seqs, T]")
    _need(context_lens.shape == (n,), "context_lens must be [num_seqs]")
    _need(q.dtype == k_cache.dtype == v_cache.dtype, "dtype mismatch")
    if out is None:
        out = torch.empty_like(q)
    _need(out.shape == q.shape and out.dtype == q.dtype, "out must match q")
    st = lib().pa_decode_fixed_scratch(
        _dev(q, "q"), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
        _dev(block_tables, "block_tables", torch.int32), block_tables.shape[1],
        _dev(context_lens, "context_lens", torch.int32), n, hq, hkv, d, bs, nb, float(scale),
        _dev(out, "out"), _dtype_code(q), _stream_ptr(stream, q.device))
    _check(st, "pa_decode_fixed_scratch")
    return out


def _int4_cache(codes, scales, name):
    import torch
    if codes.dtype != torch.uint8:
        raise ValueError(f"{name} codes must be uint8 (two 4-bit codes a byte)")
    if scales.dtype != torch.float32:
        raise ValueError(f"{name} scales must be float32")
    if not (codes.dim() == 4 and scales.shape == codes.shape[:3]):
        raise ValueError(f"{name}: codes [NB, Hkv, B, d/2] and scales [NB, Hkv, B]")
    return _dev(codes, name), _dev(scales, name + " scales")


@_on_first
def reshape_and_cache_int4(key, value, k_codes, v_codes, k_scales, v_scales, slot_mapping,
                           stream=None):
    """INT4 cache write: the row key[i, h] gets s = max|x| / 7 and codes rint(x / s) in
    [-7, 7] at slot_mapping[i] (and V likewise)."""
    import torch
    n, hkv, d = key.shape
    nb, hkv2, bs, d2 = k_codes.shape
    _need(value.shape == key.shape and v_codes.shape == k_codes.shape, "shape mismatch")
    _need(hkv == hkv2 and d == 2 * d2 and slot_mapping.shape == (n,), "shape mismatch")
    _need(key.dtype == value.dtype, "dtype mismatch")
    kc, ks = _int4_cache(k_codes, k_scales, "k")
    vc, vs = _int4_cache(v_codes, v_scales, "v")
    st = lib().pa_reshape_and_cache_int4(
        _dev(key, "key"), _dev(value, "value"), kc, vc, ks, vs,
        _dev(slot_mapping, "slot_mapping", torch.int64), n, nb, hkv, d, bs, _dtype_code(key),
        _stream_ptr(stream, key.device))
    _check(st, "pa_reshape_and_cache_int4")


@_on_first
def decode_int4(q, k_codes, v_codes, k_scales, v_scales, block_tables, context_lens, scale,
                out=None, workspace=None, stream=None):
    """Paged decode over INT4 blocks (codes [NB, Hkv, B, d/2] uint8, scales [NB, Hkv, B])."""
    import torch
    n, hq, d = q.shape
    nb, hkv, bs, d2 = k_codes.shape
    _need(v_codes.shape == k_codes.shape and d == 2 * d2, "shape mismatch")
    _need(block_tables.dim() == 2 and block_tables.shape[0] == n, "block_tables must be [num_seqs, T]")
    _need(context_lens.shape == (n,), "context_lens must be [num_seqs]")
    kc, ks = _int4_cache(k_codes, k_scales, "k")
    vc, vs = _int4_cache(v_codes, v_scales, "v")
    if out is None:
        out = torch.empty_like(q)
    _need(out.shape == q.shape and out.dtype == q.dtype, "out must match q")
    if workspace is None:
        workspace = _scratch(hq, hkv, d, q.device, stream)
    st = lib().pa_decode_int4(
        _dev(q, "q"), kc, vc, ks, vs, _dev(block_tables, "block_tables", torch.int32),
        block_tables.shape[1], _dev(context_lens, "context_lens", torch.int32), n, hq, hkv, d, bs,
        nb, float(scale), _dev(out, "out"), _dev(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _dtype_code(q), _stream_ptr(stream, q.device))
    _check(st, "pa_decode_int4")
    return out


@_on_first
def decode_append_int4(q, key_new, value_new, k_codes, v_codes, k_scales, v_scales, block_tables,
                       context_lens, scale, out=None, workspace=None, stream=None, plan=False):
    """One INT4 decode step in one kernel: each sequence's newest K/V row is quantised into
    its slot at position ctx - 1 and attended (= bit for bit reshape_and_cache_int4 +
    decode_int4).  plan=True returns a Launch instead of launching."""
    import torch
    n, hq, d = q.shape
    nb, hkv, bs, d2 = k_codes.shape
    _need(v_codes.shape == k_codes.shape and d == 2 * d2, "shape mismatch")
    _need(key_new.shape == (n, hkv, d) and value_new.shape == key_new.shape, "key_new must be [n, Hkv, d]")
    _need(key_new.dtype == value_new.dtype == q.dtype, "dtype mismatch")
    _need(block_tables.dim() == 2 and block_tables.shape[0] == n, "block_tables must be [num_seqs, T]")
    _need(context_lens.shape == (n,), "context_lens must be [num_seqs]")
    kc, ks = _int4_cache(k_codes, k_scales, "k")
    vc, vs = _int4_cache(v_codes, v_scales, "v")
    if out is None:
        out = torch.empty_like(q)
    _need(out.shape == q.shape and out.dtype == q.dtype, "out must match q")
    if workspace is None:
        workspace = _scratch(hq, hkv, d, q.device, stream)
    args = (_dev(q, "q"), _dev(key_new, "key_new"), _dev(value_new, "value_new"), kc, vc, ks, vs,
            _dev(block_tables, "block_tables", torch.int32), block_tables.shape[1],
            _dev(context_lens, "context_lens", torch.int32), n, hq, hkv, d, bs, nb, float(scale),
            _dev(out, "out"), _dev(workspace, "workspace"),
            workspace.numel() * workspace.element_size(), _dtype_code(q))
    if plan:
        return Launch("pa_decode_append_int4", args, out,
                      keep=(q, key_new, value_new, k_codes, v_codes, k_scales, v_scales,
                            block_tables, context_lens, out, workspace))
    _check(lib().pa_decode_append_int4(*args, _stream_ptr(stream, q.device)), "pa_decode_append_int4")
    return out


@_on_first
def copy_blocks_int4(k_codes, v_codes, k_scales, v_scales, block_mapping, stream=None):
    """copy_blocks for INT4 blocks: codes and scales of each (src, dst) pair."""
    import torch
    nb, hkv, bs, d2 = k_codes.shape
    _need(v_codes.shape == k_codes.shape, "shape mismatch")
    _need(block_mapping.dim() == 2 and block_mapping.shape[1] == 2, "block_mapping must be [n, 2]")
    kc, ks = _int4_cache(k_codes, k_scales, "k")
    vc, vs = _int4_cache(v_codes, v_scales, "v")
    st = lib().pa_copy_blocks_int4(kc, vc, ks, vs, _dev(block_mapping, "block_mapping", torch.int32),
                                   block_mapping.shape[0], nb, hkv, 2 * d2, bs,
                                   _stream_ptr(stream, k_codes.device))
    _check(st, "pa_copy_blocks_int4")


@_runs_on(_pool_device)
def swap_blocks_int4(src, dst, block_mapping, stream=None, device=None):
    """swap_blocks for INT4 blocks; src and dst are (k_codes, v_codes, k_scales, v_scales)
    pools, CUDA tensors or pinned CPU tensors."""
    import torch
    nbs, hkv, bs, d2 = src[0].shape
    nbd = dst[0].shape[0]
    _need(all(t.shape == src[0].shape for t in src[:2]) and all(t.shape == dst[0].shape for t in dst[:2]),
          "shape mismatch")
    _need(dst[0].shape[1:] == src[0].shape[1:], "pools must share Hkv, B, d")
    _need(all(t.dtype == torch.uint8 for t in (src[0], src[1], dst[0], dst[1])) and
          all(t.dtype == torch.float32 and t.shape == c.shape[:3]
              for t, c in ((src[2], src[0]), (src[3], src[0]), (dst[2], dst[0]), (dst[3], dst[0]))),
          "codes uint8 [NB, Hkv, B, d/2], scales float32 [NB, Hkv, B]")
    _need(block_mapping.dim() == 2 and block_mapping.shape[1] == 2, "block_mapping must be [n, 2]")
    if device is None:
        device = next((t.device for t in (src[0], dst[0]) if t.is_cuda), torch.device("cuda"))
    names = ("k", "v", "k scales", "v scales")
    st = lib().pa_swap_blocks_int4(
        *[_reachable(t, "src " + nm) for t, nm in zip(src, names)],
        *[_reachable(t, "dst " + nm) for t, nm in zip(dst, names)],
        _reachable(block_mapping, "block_mapping", torch.int32), block_mapping.shape[0], nbs, nbd,
        hkv, 2 * d2, bs, _stream_ptr(stream, device))
    _check(st, "pa_swap_blocks_int4")


# ---- FP8 blocks with a scale per (block, kv head), and the step's bookkeeping ----
# A serving step makes these calls back to back, several of them shorter on the GPU than in
# Python, so their checks touch each tensor as little as possible, and what they need of torch
# is looked up once.

class _Torch:
    """What the calls below need of torch (their first call imports it)."""

    def __init__(self):
        import torch
        self.i32, self.i64, self.f32, self.u8 = torch.int32, torch.int64, torch.float32, torch.uint8
        self.f8, self.f16, self.bf16 = torch.float8_e4m3fn, torch.float16, torch.bfloat16
        self.module, self.empty_like, self.device = torch, torch.empty_like, torch.cuda.device
        # torch's private shortcuts, which spare a call its checks; the public calls where a torch
        # has none of them
        self.current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        self.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                                  lambda dev: torch.cuda.current_stream(dev).cuda_stream)


_T = None


def _torch():
    global _T
    if _T is None:
        _T = _Torch()
    return _T


def _ptr(t, name, dtype, dev):
    """Address of a contiguous tensor of `dtype` on CUDA device number `dev`."""
    if t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    return _refuse(t, name, (dtype,), dev)


def _codes_ptr(t, name, dev):
    """The same of E4M3 codes (uint8 or float8_e4m3fn)."""
    T = _T or _torch()
    dt = t.dtype
    if (dt is T.u8 or dt is T.f8) and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    return _refuse(t, name, (T.u8, T.f8), dev)


def _code16(dtype):
    T = _T or _torch()
    if dtype is T.bf16:
        return PA_BF16
    if dtype is T.f16:
        return PA_FP16
    raise TypeError(f"unsupported dtype {dtype}; expected float16 or bfloat16")


def _device_of(t, name):
    """The CUDA device number of a call's first tensor."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def _refuse(t, name, dtypes, dev):
    _need(t.is_cuda, f"{name} must be a CUDA tensor")
    _need(t.get_device() == dev, f"{name} is on another device than the call's first tensor")
    _need(t.is_contiguous(), f"{name} must be contiguous")
    raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")


def _on_its_device(fn):
    """Decorator: run the call with the device of its first tensor current."""
    @functools.wraps(fn)
    def wrapped(t, *args, **kw):
        T = _T or _torch()
        dev = t.get_device()
        if dev < 0 or dev == T.current_device():
            return fn(t, *args, **kw)
        with T.device(dev):
            return fn(t, *args, **kw)
    return wrapped


def _raw_stream(stream, dev):
    return (_T or _torch()).raw_stream(dev) if stream is None else stream.cuda_stream


def _empty_like(t, stream):
    """A new tensor like `t`, allocated for the stream that the call runs on."""
    T = _T or _torch()
    if stream is None:
        return T.empty_like(t)
    with T.module.cuda.stream(stream):
        return T.empty_like(t)


def _block_scaled(k_cache, v_cache, k_scales, v_scales, d):
    """(num_blocks, num_kv_heads, block_size) of the caches, checked against each other."""
    nb, hkv, bs, d2 = shape = k_cache.shape
    _need(d2 == d and v_cache.shape == shape, "shape mismatch")
    if k_scales.shape != (nb, hkv) or v_scales.shape != (nb, hkv):
        raise ValueError("k, v: codes [NB, Hkv, B, d] and scales [NB, Hkv]")
    return nb, hkv, bs


@_on_its_device
def build_step(query_lens, context_lens, free_blocks, free_start, block_tables, block_size,
               num_blocks, slot_mapping, query_start=None, free_next=None, stream=None, plan=False):
    """Block tables and slots of one step from request lengths, on the GPU: request s has
    context_lens[s] tokens, query_lens[s] of them new.  Its missing blocks come from
    free_blocks[free_start[0]:] in request order and are written into block_tables;
    slot_mapping gets the slot of every new token (-1 past the last one); returns
    (query_start [num_seqs + 1], free_next [1]).  A step that lacks blocks or slots changes
    no table, sets every slot to -1 and a device error bit.  plan=True returns a Launch whose
    runs return query_start (query_start and free_next must then be given)."""
    T = _T or _torch()
    torch, dev, i32 = T.module, _device_of(query_lens, "query_lens"), T.i32
    n, = query_lens.shape
    tn, width = block_tables.shape
    _need(context_lens.shape == (n,), "query_lens and context_lens must be [num_seqs]")
    _need(tn == n, "block_tables must be [num_seqs, T]")
    nfree, = free_blocks.shape
    slots, = slot_mapping.shape
    _need(free_start.numel() == 1, "free_start must hold one value")
    if query_start is None or free_next is None:
        _need(not plan, "a planned build_step needs query_start and free_next")
        with torch.cuda.stream(stream):  # (allocated for the stream that writes them)
            if query_start is None:
                query_start = torch.empty(n + 1, dtype=i32, device=query_lens.device)
            if free_next is None:
                free_next = torch.empty(1, dtype=i32, device=query_lens.device)
    _need(query_start.shape == (n + 1,), "query_start must be [num_seqs + 1]")
    _need(free_next.numel() == 1, "free_next must hold one value")
    args = (_ptr(query_lens, "query_lens", i32, dev), _ptr(context_lens, "context_lens", i32, dev),
            n, _ptr(free_blocks, "free_blocks", i32, dev), nfree,
            _ptr(free_start, "free_start", i32, dev), _ptr(block_tables, "block_tables", i32, dev),
            width, int(block_size), int(num_blocks), _ptr(slot_mapping, "slot_mapping", T.i64, dev),
            slots, _ptr(query_start, "query_start", i32, dev), _ptr(free_next, "free_next", i32, dev))
    if plan:
        return Launch("pa_build_step", args, query_start,
                      keep=(query_lens, context_lens, free_blocks, free_start, block_tables,
                            slot_mapping, free_next))
    st = lib().pa_build_step(*args, _raw_stream(stream, dev))
    if st < 0:
        _check(st, "pa_build_step")
    return query_start, free_next


@_on_its_device
def append_fp8_block(key, value, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens,
                     query_start, stream=None, plan=False):
    """Cache write of FP8 blocks with a scale per (block, kv head): sequence s's rows
    query_start[s] .. query_start[s+1]-1 of key / value become its positions context_lens[s] -
    q_len .. context_lens[s] - 1.  A block's scale is the smallest power of two that holds
    its rows; where a new row raises it, the block's earlier rows are requantised.  Rows
    behind the last sequence are not read.  plan=True returns a Launch instead of writing."""
    T = _T or _torch()
    dev, i32, dt, f32 = _device_of(key, "key"), T.i32, key.dtype, T.f32
    ntok, heads, d = shape = key.shape
    n, width = block_tables.shape
    nb, hkv, bs = _block_scaled(k_cache, v_cache, k_scales, v_scales, d)
    _need(heads == hkv and value.shape == shape, "shape mismatch")
    _need(context_lens.shape == (n,), "block_tables must be [num_seqs, T], context_lens [num_seqs]")
    _need(query_start.shape == (n + 1,), "query_start must be [num_seqs + 1]")
    args = (_ptr(key, "key", dt, dev), _ptr(value, "value", dt, dev),
            _codes_ptr(k_cache, "k_cache", dev), _codes_ptr(v_cache, "v_cache", dev),
            _ptr(k_scales, "k_scales", f32, dev), _ptr(v_scales, "v_scales", f32, dev),
            _ptr(block_tables, "block_tables", i32, dev), width,
            _ptr(context_lens, "context_lens", i32, dev), _ptr(query_start, "query_start", i32, dev),
            n, ntok, nb, hkv, d, bs, _code16(dt))
    if plan:
        return Launch("pa_append_fp8_block", args, k_cache,
                      keep=(key, value, v_cache, k_scales, v_scales, block_tables, context_lens,
                            query_start))
    st = lib().pa_append_fp8_block(*args, _raw_stream(stream, dev))
    if st < 0:
        _check(st, "pa_append_fp8_block")


@_on_its_device
def decode_fp8_block(q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, scale,
                     out=None, workspace=None, stream=None, plan=False):
    """Paged decode over FP8 blocks with a scale per (block, kv head) (codes [NB, Hkv, B, d],
    scales [NB, Hkv] float32); q and out are fp16 or bf16.  plan=True returns a Launch
    instead of launching."""
    T = _T or _torch()
    dev, i32, dt, f32 = _device_of(q, "q"), T.i32, q.dtype, T.f32
    n, hq, d = shape = q.shape
    tn, width = block_tables.shape
    nb, hkv, bs = _block_scaled(k_cache, v_cache, k_scales, v_scales, d)
    _need(tn == n, "block_tables must be [num_seqs, T]")
    _need(context_lens.shape == (n,), "context_lens must be [num_seqs]")
    if out is None:
        out = _empty_like(q, stream)
    elif out.shape != shape or out.dtype is not dt:
        raise ValueError("out must match q")
    if workspace is None:
        workspace = _scratch(hq, hkv, d, q.device, stream)
    args = (_ptr(q, "q", dt, dev), _codes_ptr(k_cache, "k_cache", dev),
            _codes_ptr(v_cache, "v_cache", dev), _ptr(k_scales, "k_scales", f32, dev),
            _ptr(v_scales, "v_scales", f32, dev), _ptr(block_tables, "block_tables", i32, dev),
            width, _ptr(context_lens, "context_lens", i32, dev), n, hq, hkv, d, bs, nb, float(scale),
            _ptr(out, "out", dt, dev), _ptr(workspace, "workspace", workspace.dtype, dev),
            workspace.numel() * workspace.element_size(), _code16(dt))
    if plan:
        return Launch("pa_decode_fp8_block", args, out,
                      keep=(q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens,
                            workspace))
    st = lib().pa_decode_fp8_block(*args, _raw_stream(stream, dev))
    if st < 0:
        _check(st, "pa_decode_fp8_block")
    return out


@_on_its_device
def prefill_fp8_block(q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens,
                      query_start, scale, max_query_len, out=None, stream=None, plan=False):
    """prefill over FP8 blocks with a scale per (block, kv head): causal attention of each
    sequence's newest tokens over its paged context; the tokens' own rows must already be in
    the cache (append_fp8_block).  scale must be positive.  plan=True returns a Launch
    instead of launching."""
    T = _T or _torch()
    dev, i32, dt, f32 = _device_of(q, "q"), T.i32, q.dtype, T.f32
    ntok, hq, d = shape = q.shape
    n, width = block_tables.shape
    nb, hkv, bs = _block_scaled(k_cache, v_cache, k_scales, v_scales, d)
    _need(context_lens.shape == (n,), "block_tables must be [num_seqs, T], context_lens [num_seqs]")
    _need(query_start.shape == (n + 1,), "query_start must be [num_seqs + 1]")
    if out is None:
        out = _empty_like(q, stream)
    elif out.shape != shape or out.dtype is not dt:
        raise ValueError("out must match q")
    args = (_ptr(q, "q", dt, dev), _codes_ptr(k_cache, "k_cache", dev),
            _codes_ptr(v_cache, "v_cache", dev), _ptr(k_scales, "k_scales", f32, dev),
            _ptr(v_scales, "v_scales", f32, dev), _ptr(block_tables, "block_tables", i32, dev),
            width, _ptr(context_lens, "context_lens", i32, dev),
            _ptr(query_start, "query_start", i32, dev), n, ntok, int(max_query_len), hq, hkv, d, bs, nb,
            float(scale), _ptr(out, "out", dt, dev), _code16(dt))
    if plan:
        return Launch("pa_prefill_fp8_block", args, out,
                      keep=(q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens,
                            query_start))
    st = lib().pa_prefill_fp8_block(*args, _raw_stream(stream, dev))
    if st < 0:
        _check(st, "pa_prefill_fp8_block")
    return out


@_on_its_device
def copy_blocks_fp8_block(k_cache, v_cache, k_scales, v_scales, block_mapping, stream=None):
    """copy_blocks for FP8 blocks with block scales: codes and scales of each (src, dst) pair
    in one launch."""
    T = _T or _torch()
    dev, f32 = _device_of(k_cache, "k_cache"), T.f32
    d = k_cache.shape[3]
    nb, hkv, bs = _block_scaled(k_cache, v_cache, k_scales, v_scales, d)
    pairs, two = block_mapping.shape
    _need(two == 2, "block_mapping must be [n, 2]")
    st = lib().pa_copy_blocks_fp8_block(
        _codes_ptr(k_cache, "k_cache", dev), _codes_ptr(v_cache, "v_cache", dev),
        _ptr(k_scales, "k_scales", f32, dev), _ptr(v_scales, "v_scales", f32, dev),
        _ptr(block_mapping, "block_mapping", T.i32, dev), pairs, nb, hkv, d, bs,
        _raw_stream(stream, dev))
    if st < 0:
        _check(st, "pa_copy_blocks_fp8_block")


@_runs_on(_pool_device)
def swap_blocks_fp8_block(src, dst, block_mapping, stream=None, device=None):
    """swap_blocks for FP8 blocks with block scales; src and dst are (k_cache, v_cache,
    k_scales, v_scales) pools, CUDA tensors or pinned CPU tensors."""
    import torch
    nbs, hkv, bs, d = src[0].shape
    nbd = dst[0].shape[0]
    _need(all(t.shape == src[0].shape for t in src[:2]) and all(t.shape == dst[0].shape for t in dst[:2]),
          "shape mismatch")
    _need(dst[0].shape[1:] == src[0].shape[1:], "pools must share Hkv, B, d")
    _need(all(_cache_code(t) == PA_FP8_E4M3 for t in (src[0], src[1], dst[0], dst[1])) and
          all(t.dtype == torch.float32 and t.shape == c.shape[:2]
              for t, c in ((src[2], src[0]), (src[3], src[0]), (dst[2], dst[0]), (dst[3], dst[0]))),
          "codes E4M3 [NB, Hkv, B, d], scales float32 [NB, Hkv]")
    _need(block_mapping.dim() == 2 and block_mapping.shape[1] == 2, "block_mapping must be [n, 2]")
    if device is None:
        device = next((t.device for t in (src[0], dst[0]) if t.is_cuda), torch.device("cuda"))
    names = ("k_cache", "v_cache", "k_scales", "v_scales")
    st = lib().pa_swap_blocks_fp8_block(
        *[_reachable(t, "src " + nm) for t, nm in zip(src, names)],
        *[_reachable(t, "dst " + nm) for t, nm in zip(dst, names)],
        _reachable(block_mapping, "block_mapping", torch.int32), block_mapping.shape[0], nbs, nbd,
        hkv, d, bs, _stream_ptr(stream, device))
    _check(st, "pa_swap_blocks_fp8_block")


# ---- a decoding step that checks drafted tokens, and attention to an encoder's states ----

def rotary_frequencies(rotary_dim, base=10000.0, scaling=None, device="cuda"):
    """(freqs, amplitude) for rotary and rotary_append: the turns per token of each pair, base **
    (-2 i / rotary_dim) radians, as an int64 tensor [rotary_dim / 2] on `device` in units of 2^-64,
    and the factor on cosines and sines.  `scaling` stretches them for contexts longer than the
    model was trained on (a dict):
      kind="linear", factor: f / factor;
      kind="bands", factor, low, high, trained: f where the trained length holds more than `high`
        turns, f / factor where fewer than `low`, blended by the number of turns between;
      kind="ramp", factor, slow, fast, trained (and amplitude, 0.1 ln(factor) + 1 by default): f /
        factor and f blended linearly in the pair's index between the indexes, rounded outwards,
        whose pairs make `fast` and `slow` turns over the trained length."""
    import math
    import numpy as np
    import torch
    rd = int(rotary_dim)
    _need(rd >= 2 and rd % 2 == 0, "rotary_dim must be even and positive")
    base = float(base)
    _need(math.isfinite(base) and base > 1.0, "base must be above 1")
    f = np.array([base ** (-2.0 * i / rd) for i in range(rd // 2)], dtype=np.float64)
    amplitude = 1.0
    if scaling is not None:
        how = dict(scaling)
        kind, factor = how.pop("kind"), float(how.pop("factor"))
        _need(math.isfinite(factor) and factor > 0.0, "factor must be positive")
        if kind == "linear":
            f = f / factor
        elif kind == "bands":
            low, high, trained = (float(how.pop(k)) for k in ("low", "high", "trained"))
            _need(high > low, "high must be above low")
            a = np.clip((trained * f / (2 * math.pi) - low) / (high - low), 0.0, 1.0)
            f = (1 - a) * f / factor + a * f
        elif kind == "ramp":
            slow, fast, trained = (float(how.pop(k)) for k in ("slow", "fast", "trained"))
            _need(slow > 0 and fast > 0 and trained > 0, "slow, fast and trained must be positive")

            def index(turns):  # of the pair that makes so many turns over the trained length
                return rd * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))
            lo, hi = max(math.floor(index(fast)), 0), min(math.ceil(index(slow)), rd - 1)
            a = np.clip((np.arange(rd // 2) - lo) / max(hi - lo, 0.001), 0.0, 1.0)
            f = a * f / factor + (1 - a) * f
            amplitude = float(how.pop("amplitude", 0.1 * math.log(factor) + 1.0))
        else:
            raise ValueError(f"unknown scaling kind {kind!r}: linear, bands or ramp")
        _need(not how, f"unknown scaling entries {sorted(how)}")
    f = np.ascontiguousarray(f)
    out = np.zeros(rd // 2, dtype=np.int64)
    _check(lib().pa_rotary_frequencies(f.ctypes.data, rd // 2, out.ctypes.data), "pa_rotary_frequencies")
    return torch.from_numpy(out).to(device), amplitude


def _rows_ptr(t, name, heads, d, dtype, dev):
    """(address, values from row to row) of a [rows, heads, d] tensor of `dtype` on CUDA device
    number `dev` whose rows are contiguous, as slices of one projection's output are."""
    if (t.dtype is not dtype or t.get_device() != dev or t.dim() != 3 or t.shape[1] != heads or t.shape[2] != d):
        _need(t.dim() == 3 and t.shape[1] == heads and t.shape[2] == d, f"{name} must be [num_tokens, {heads}, {d}]")
        _refuse(t.contiguous(), name, (dtype,), dev)
    stride, sh, sd = t.stride()
    if not (sd == 1 and (sh == d or heads == 1)):
        raise ValueError(f"the heads of a row of {name} must be contiguous")
    if t.shape[0] <= 1:
        stride = heads * d
    return t.data_ptr(), stride


def _freqs_ptr(freqs, dev):
    T = _T or _torch()
    half, = freqs.shape
    return _ptr(freqs, "freqs", T.i64, dev), 2 * half


@_on_its_device
def rotary(q, key, context_lens, query_start, freqs, interleaved=False, amplitude=1.0, out=None,
           key_out=None, stream=None, plan=False):
    """Rotary positions of a step's new tokens: sequence s's rows query_start[s] ..
    query_start[s+1]-1 of q [num_tokens, num_q_heads, d] and key [num_tokens, num_kv_heads, d] are
    at positions context_lens[s] - q_len .. context_lens[s] - 1.  The first 2 * len(freqs) values
    of each head are turned (rotary_frequencies), as halves or, interleaved, as neighbours.
    Returns (out, key_out), which may be q and key themselves; rows behind the last sequence are left as
    they were.  For caches that rotary_append does not write.  plan=True returns a Launch whose
    runs return out (key_out must then be given)."""
    T = _T or _torch()
    dev, dt, i32 = _device_of(q, "q"), q.dtype, T.i32
    ntok, hq, d = q.shape
    hkv = key.shape[1]
    n, = context_lens.shape
    _need(key.shape[0] == ntok, "q and key must have as many rows")
    _need(query_start.shape == (n + 1,), "query_start must be [num_seqs + 1]")
    _need(not (plan and key_out is None), "a planned rotary needs key_out")
    if out is None:
        out = _new_rows(q, stream)
    if key_out is None:
        key_out = _new_rows(key, stream)
    _need(out.shape == q.shape and key_out.shape == key.shape, "out must match q, key_out key")
    fptr, rd = _freqs_ptr(freqs, dev)
    args = (*_rows_ptr(q, "q", hq, d, dt, dev), *_rows_ptr(key, "key", hkv, d, dt, dev),
            *_rows_ptr(out, "out", hq, d, dt, dev), *_rows_ptr(key_out, "key_out", hkv, d, dt, dev),
            _ptr(context_lens, "context_lens", i32, dev), _ptr(query_start, "query_start", i32, dev),
            fptr, rd, int(bool(interleaved)), float(amplitude), n, ntok, hq, hkv, d, _code16(dt))
    if plan:
        return Launch("pa_rotary", args, out, keep=(q, key, key_out, context_lens, query_start, freqs))
    st = lib().pa_rotary(*args, _raw_stream(stream, dev))
    if st < 0:
        _check(st, "pa_rotary")
    return out, key_out


def _new_rows(t, stream):
    """A new contiguous tensor of t's shape, allocated for the stream that the call runs on."""
    T = _T or _torch()
    if stream is None:
        return T.module.empty(t.shape, dtype=t.dtype, device=t.device)
    with T.module.cuda.stream(stream):
        return T.module.empty(t.shape, dtype=t.dtype, device=t.device)


@_on_its_device
def rotary_append(q, key, value, k_cache, v_cache, block_tables, context_lens, query_start, freqs,
                  interleaved=False, amplitude=1.0, out=None, stream=None, plan=False):
    """rotary with the cache write, in one launch: the turned keys and the values go through the
    block tables into the caches.  q, key and value may be slices of one projection's output
    (heads contiguous, any distance from row to row that is a multiple of 8 values).  Returns the
    turned q (out, which may be q itself).  plan=True returns a Launch instead of launching."""
    T = _T or _torch()
    dev, dt, i32 = _device_of(q, "q"), q.dtype, T.i32
    ntok, hq, d = shape = q.shape
    n, width = block_tables.shape
    nb, hkv, bs, d2 = cache = k_cache.shape
    kv = (ntok, hkv, d)
    if out is None:
        out = _new_rows(q, stream)
    half, = freqs.shape
    if not (key.shape == kv and value.shape == kv and out.shape == shape and d2 == d and v_cache.shape == cache
            and context_lens.shape == (n,) and query_start.shape == (n + 1,)):
        _need(key.shape == kv and value.shape == kv, "key and value must be [num_tokens, num_kv_heads, head_dim]")
        _need(out.shape == shape, "out must match q")
        _need(d2 == d and v_cache.shape == cache, "shape mismatch")
        _need(context_lens.shape == (n,), "block_tables must be [num_seqs, T], context_lens [num_seqs]")
        _need(False, "query_start must be [num_seqs + 1]")
    q0, q1, q2 = q.stride()
    k0, k1, k2 = key.stride()
    v0, v1, v2 = value.stride()
    o0, o1, o2 = out.stride()
    i64 = T.i64
    if (q2 == k2 == v2 == o2 == 1 and q1 == k1 == v1 == o1 == d and ntok > 1 and key.dtype is dt
            and value.dtype is dt and out.dtype is dt and k_cache.dtype is dt and v_cache.dtype is dt
            and block_tables.dtype is i32 and context_lens.dtype is i32 and query_start.dtype is i32
            and freqs.dtype is i64 and key.get_device() == dev and value.get_device() == dev
            and out.get_device() == dev and k_cache.get_device() == dev and v_cache.get_device() == dev
            and block_tables.get_device() == dev and context_lens.get_device() == dev
            and query_start.get_device() == dev and freqs.get_device() == dev
            and k_cache.is_contiguous() and v_cache.is_contiguous() and block_tables.is_contiguous()
            and context_lens.is_contiguous() and query_start.is_contiguous() and freqs.is_contiguous()):
        args = (q.data_ptr(), q0, key.data_ptr(), k0, value.data_ptr(), v0, out.data_ptr(), o0,
                k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(), width, context_lens.data_ptr(),
                query_start.data_ptr(), freqs.data_ptr(), 2 * half, 1 if interleaved else 0, amplitude, n, ntok, nb, hq,
                hkv, d, bs, _code16(dt))
    else:  # (one row, one head, or something to refuse)
        args = (*_rows_ptr(q, "q", hq, d, dt, dev), *_rows_ptr(key, "key", hkv, d, dt, dev),
                *_rows_ptr(value, "value", hkv, d, dt, dev), *_rows_ptr(out, "out", hq, d, dt, dev),
                _ptr(k_cache, "k_cache", dt, dev), _ptr(v_cache, "v_cache", dt, dev),
                _ptr(block_tables, "block_tables", i32, dev), width, _ptr(context_lens, "context_lens", i32, dev),
                _ptr(query_start, "query_start", i32, dev), _ptr(freqs, "freqs", i64, dev), 2 * half,
                1 if interleaved else 0, amplitude, n, ntok, nb, hq, hkv, d, bs, _code16(dt))
    if plan:
        return Launch("pa_rotary_append", args, out,
                      keep=(q, key, value, k_cache, v_cache, block_tables, context_lens, query_start, freqs))
    st = lib().pa_rotary_append(*args, _raw_stream(stream, dev))
    if st < 0:
        _check(st, "pa_rotary_append")
    return out


def split_workspace_size(num_q_heads, num_kv_heads, head_dim):
    """Bytes of workspace decode_drafts and cross need on the current device."""
    n = lib().pa_split_workspace_size(num_q_heads, num_kv_heads, head_dim)
    if n == 0:
        raise PagedAttentionError(PA_ERR_ARG, "pa_split_workspace_size")
    return n


def make_split_workspace(num_q_heads, num_kv_heads, head_dim, device=None):
    import torch
    device = torch.device(device or "cuda")
    with torch.cuda.device(device):
        return torch.empty(split_workspace_size(num_q_heads, num_kv_heads, head_dim),
                           dtype=torch.uint8, device=device)


def _split_attention(name, q, k_cache, v_cache, block_tables, context_lens, query_start, scale, out,
                     workspace, stream, plan):
    T = _T or _torch()
    dev, i32, dt = _device_of(q, "q"), T.i32, q.dtype
    ntok, hq, d = shape = q.shape
    n, width = block_tables.shape
    nb, hkv, bs, d2 = k_cache.shape
    _need(d2 == d and v_cache.shape == k_cache.shape, "shape mismatch")
    _need(context_lens.shape == (n,), "block_tables must be [num_seqs, T], context_lens [num_seqs]")
    _need(query_start.shape == (n + 1,), "query_start must be [num_seqs + 1]")
    if out is None:
        out = _empty_like(q, stream)
    elif out.shape != shape or out.dtype is not dt:
        raise ValueError("out must match q")
    if workspace is None:
        if stream is None:
            workspace = make_split_workspace(hq, hkv, d, q.device)
        else:
            with T.module.cuda.stream(stream):  # (allocated for the stream that the call runs on)
                workspace = make_split_workspace(hq, hkv, d, q.device)
    if (k_cache.dtype is dt and v_cache.dtype is dt and block_tables.dtype is i32 and context_lens.dtype is i32
            and query_start.dtype is i32 and out.dtype is dt
            and k_cache.get_device() == dev and v_cache.get_device() == dev and block_tables.get_device() == dev
            and context_lens.get_device() == dev and query_start.get_device() == dev and out.get_device() == dev
            and workspace.get_device() == dev
            and q.is_contiguous() and k_cache.is_contiguous() and v_cache.is_contiguous()
            and block_tables.is_contiguous() and context_lens.is_contiguous() and query_start.is_contiguous()
            and out.is_contiguous() and workspace.is_contiguous()):
        args = (q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(), width,
                context_lens.data_ptr(), query_start.data_ptr(), n, ntok, hq, hkv, d, bs, nb, scale, out.data_ptr(),
                workspace.data_ptr(), workspace.numel() * workspace.element_size(), _code16(dt))
    else:  # (says which one and why)
        for t, what, kind in ((q, "q", dt), (k_cache, "k_cache", dt), (v_cache, "v_cache", dt),
                              (block_tables, "block_tables", i32), (context_lens, "context_lens", i32),
                              (query_start, "query_start", i32), (out, "out", dt),
                              (workspace, "workspace", workspace.dtype)):
            _ptr(t, what, kind, dev)
        raise ValueError("unsupported arguments")
    if plan:
        return Launch(name, args, out,
                      keep=(q, k_cache, v_cache, block_tables, context_lens, query_start, workspace))
    st = getattr(lib(), name)(*args, _raw_stream(stream, dev))
    if st < 0:
        _check(st, name)
    return out


@_on_its_device
def decode_drafts(q, k_cache, v_cache, block_tables, context_lens, query_start, scale, out=None,
                  workspace=None, stream=None, plan=False):
    """Causal attention of each sequence's newest tokens (rows query_start[s] ..
    query_start[s+1]-1 of q, at positions ctx - q_len .. ctx - 1, their K/V already in the cache)
    over its paged context, the keys of a sequence split over the SMs: for a few tokens a sequence,
    drafts to be checked say, where prefill would leave most SMs idle.  (Up to some 256 rows a
    sequence; whole prompts are prefill's.)  scale must be positive.
    workspace: make_split_workspace.  plan=True returns a Launch instead of launching."""
    return _split_attention("pa_decode_drafts", q, k_cache, v_cache, block_tables, context_lens,
                            query_start, scale, out, workspace, stream, plan)


@_on_its_device
def cross(q, k_cache, v_cache, block_tables, context_lens, query_start, scale, out=None,
          workspace=None, stream=None, plan=False):
    """Attention of each sequence's rows of q to all context_lens[s] cached tokens, without a mask:
    a decoder's tokens over an encoder's states of another length (0 of them: zeros).  Where every
    sequence has one row and some states, decode computes the same and is faster.  Otherwise as
    decode_drafts."""
    return _split_attention("pa_cross", q, k_cache, v_cache, block_tables, context_lens,
                            query_start, scale, out, workspace, stream, plan)


def _probs_ptr(t, name, dtype, dev):
    """(address, values from row to row) of probabilities [rows, vocab]."""
    if t.dtype is not dtype or t.get_device() != dev:
        _refuse(t.contiguous(), name, (dtype,), dev)
    stride, sv = t.stride()
    if sv != 1 and t.shape[1] > 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return t.data_ptr(), (stride if t.shape[0] > 1 else t.shape[1])


@_on_its_device
def verify_drafts(tokens, target_probs, draft_probs, uniforms, query_start, context_lens, out=None,
                  emitted=None, context_next=None, stream=None, plan=False):
    """Which drafted tokens stay, and the token after them.  tokens [num_tokens] int32: sequence
    s's rows query_start[s] .. query_start[s+1]-1 are its last token and its drafts; target_probs
    [num_tokens, vocab] the model's distribution after each row; draft_probs the same of the model
    that drafted (row i is what row i + 1's token was drawn from), or None where each draft was
    certain; uniforms [num_tokens] float32 in [0, 1).  A draft x in row i + 1 is accepted while
    uniforms[i] * draft[i, x] < target[i, x]; then a token is drawn from max(target - draft, 0) of
    the first row refused, or from the last row's target, by inversion with the sequence's last
    uniform.  Probabilities and uniforms below 0 and NaN count as 0, above 1 as 1.  Returns (out
    [num_tokens]: accepted drafts, the drawn token, -1; emitted [num_seqs]: tokens that came out;
    context_next [num_seqs]: context_lens - q_len + emitted, the tokens whose K/V rows stay, which
    may be context_lens itself).  Rows of the probabilities may lie farther apart than vocab.
    plan=True returns a Launch whose runs return out (emitted and context_next must then be
    given)."""
    T = _T or _torch()
    dev, i32 = _device_of(tokens, "tokens"), T.i32
    ntok, = tokens.shape
    n, = context_lens.shape
    rows, vocab = target_probs.shape
    dt = target_probs.dtype
    _need(rows == ntok and uniforms.shape == (ntok,), "tokens, target_probs and uniforms must have as many rows")
    _need(query_start.shape == (n + 1,), "query_start must be [num_seqs + 1]")
    _need(not plan or (emitted is not None and context_next is not None),
          "a planned verify_drafts needs emitted and context_next")
    code = PA_FP32 if dt is T.f32 else _code16(dt)
    if out is None:
        out = _empty_like(tokens, stream)
    if emitted is None:
        emitted = _empty_like(context_lens, stream)
    if context_next is None:
        context_next = _empty_like(context_lens, stream)
    _need(out.shape == (ntok,) and emitted.shape == (n,) and context_next.shape == (n,),
          "out must be [num_tokens], emitted and context_next [num_seqs]")
    if draft_probs is None:
        draft = (None, 0)
    else:
        _need(draft_probs.shape == (rows, vocab), "draft_probs must match target_probs")
        draft = _probs_ptr(draft_probs, "draft_probs", dt, dev)
    f32 = T.f32
    if not (tokens.dtype is i32 and uniforms.dtype is f32 and query_start.dtype is i32 and context_lens.dtype is i32
            and out.dtype is i32 and emitted.dtype is i32 and context_next.dtype is i32
            and uniforms.get_device() == dev and query_start.get_device() == dev and context_lens.get_device() == dev
            and out.get_device() == dev and emitted.get_device() == dev and context_next.get_device() == dev
            and tokens.is_contiguous() and uniforms.is_contiguous() and query_start.is_contiguous()
            and context_lens.is_contiguous() and out.is_contiguous() and emitted.is_contiguous()
            and context_next.is_contiguous()):  # (says which one and why)
        for t, what, kind in ((tokens, "tokens", i32), (uniforms, "uniforms", f32), (query_start, "query_start", i32),
                              (context_lens, "context_lens", i32), (out, "out", i32), (emitted, "emitted", i32),
                              (context_next, "context_next", i32)):
            _ptr(t, what, kind, dev)
    args = (tokens.data_ptr(), *_probs_ptr(target_probs, "target_probs", dt, dev), *draft, uniforms.data_ptr(),
            query_start.data_ptr(), context_lens.data_ptr(), n, ntok, vocab, out.data_ptr(), emitted.data_ptr(),
            context_next.data_ptr(), code)
    if plan:
        return Launch("pa_verify_drafts", args, out,
                      keep=(tokens, target_probs, draft_probs, uniforms, query_start, context_lens, emitted,
                            context_next))
    st = lib().pa_verify_drafts(*args, _raw_stream(stream, dev))
    if st < 0:
        _check(st, "pa_verify_drafts")
    return out, emitted, context_next


@_on_first
def copy_blocks(k_cache, v_cache, block_mapping, stream=None):
    """k_cache[dst] = k_cache[src] and v_cache[dst] = v_cache[src] for each (src, dst)."""
    import torch
    nb, hkv, bs, d = k_cache.shape
    _need(v_cache.shape == k_cache.shape, "shape mismatch")
    _need(block_mapping.dim() == 2 and block_mapping.shape[1] == 2, "block_mapping must be [n, 2]")
    st = lib().pa_copy_blocks(
        _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
        _dev(block_mapping, "block_mapping", torch.int32), block_mapping.shape[0], nb, hkv, d, bs,
        _cache_code(k_cache), _stream_ptr(stream, k_cache.device))
    _check(st, "pa_copy_blocks")


def _reachable(t, name, dtype=None):
    """A CUDA tensor, or a page-locked (pinned) CPU tensor that the GPU can address."""
    if not ((t.is_cuda or t.is_pinned()) and t.is_contiguous()
            and (dtype is None or t.dtype == dtype)):
        _need(t.is_cuda or t.is_pinned(), f"{name} must be a CUDA tensor or a pinned CPU tensor")
        _need(t.is_contiguous(), f"{name} must be contiguous")
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


@_runs_on(_pool_device)
def swap_blocks(src_k, src_v, dst_k, dst_v, block_mapping, stream=None, device=None):
    """dst_k[d] = src_k[s] and dst_v[d] = src_v[s] for each (s, d) of block_mapping, in one
    kernel launch.  Pools and mapping may be CUDA tensors or pinned CPU tensors (swap-out:
    device pool -> pinned CPU pool; swap-in: the reverse)."""
    import torch
    nbs, hkv, bs, d = src_k.shape
    nbd = dst_k.shape[0]
    _need(src_v.shape == src_k.shape and dst_v.shape == dst_k.shape, "shape mismatch")
    _need(dst_k.shape[1:] == src_k.shape[1:], "pools must share Hkv, B, d")
    _need(src_k.dtype == src_v.dtype == dst_k.dtype == dst_v.dtype, "dtype mismatch")
    _need(block_mapping.dim() == 2 and block_mapping.shape[1] == 2, "block_mapping must be [n, 2]")
    if device is None:
        device = next((t.device for t in (src_k, dst_k) if t.is_cuda), torch.device("cuda"))
    st = lib().pa_swap_blocks(
        _reachable(src_k, "src_k"), _reachable(src_v, "src_v"), _reachable(dst_k, "dst_k"),
        _reachable(dst_v, "dst_v"), _reachable(block_mapping, "block_mapping", torch.int32),
        block_mapping.shape[0], nbs, nbd, hkv, d, bs, _cache_code(src_k),
        _stream_ptr(stream, device))
    _check(st, "pa_swap_blocks")


def check_block_mapping(pairs, num_blocks):
    """Host check of a copy_blocks pair list (sequence of (src, dst)); raises on aliasing."""
    import numpy as np
    arr = np.ascontiguousarray(np.asarray(pairs, dtype=np.int32).reshape(-1, 2))
    st = lib().pa_check_block_mapping(arr.ctypes.data, arr.shape[0], num_blocks)
    _check(st, "pa_check_block_mapping")


def get_device_error(stream=None, device=None):
    """Synchronise the stream, then read and clear the error word of `device` (default:
    the stream's device, else the current one)."""
    import torch
    if device is None:
        dev = stream.device if stream is not None else torch.device("cuda", torch.cuda.current_device())
    else:
        dev = torch.device(device)
    sw = _switch_to(dev)
    v = ctypes.c_uint32(0)
    if sw is None:
        st = lib().pa_get_device_error(_stream_ptr(stream, dev), ctypes.byref(v))
    else:
        with torch.cuda.device(sw):
            st = lib().pa_get_device_error(_stream_ptr(stream, dev), ctypes.byref(v))
    _check(st, "pa_get_device_error")
    return v.value


# ------------------------------------------------------------------ block pool

def sha256(data):
    """SHA-256 digest of a bytes object, computed by the library (FIPS 180-4)."""
    buf = ctypes.create_string_buffer(bytes(data), max(len(data), 1))
    out = ctypes.create_string_buffer(32)
    _check(lib().pa_sha256(buf, len(data), out), "pa_sha256")
    return out.raw


def block_hashes(tokens, block_size, extra=b""):
    """The chained digests (list of 32-byte strings) of the full blocks of a token list."""
    import numpy as np
    tok = np.ascontiguousarray(np.asarray(tokens, dtype=np.int32))
    m = len(tok) // int(block_size)
    out = ctypes.create_string_buffer(32 * max(m, 1))
    ex = bytes(extra)
    n = _check(lib().pa_prefix_block_hashes(tok.ctypes.data, len(tok), int(block_size), ex or None,
                                            len(ex), out, m), "pa_prefix_block_hashes")
    return [out.raw[32 * i:32 * (i + 1)] for i in range(n)]


class BlockPool:
    """Host block pool (C++): ordered free list, refcounts, fork, copy-on-write planning,
    and an optional CPU pool for swap-out / swap-in."""

    def __init__(self, num_blocks, block_size, initial_free_order=None, num_cpu_blocks=0,
                 cpu_free_order=None):
        import numpy as np
        self.num_blocks = int(num_blocks)
        self.block_size = int(block_size)
        self.num_cpu_blocks = int(num_cpu_blocks)

        def order_ptr(order, n, name):
            if order is None:
                return None, None
            arr = np.ascontiguousarray(np.asarray(order, dtype=np.int32))
            _need(arr.shape == (n,), f"{name} must have {n} entries")
            return arr, arr.ctypes.data
        self._order, order = order_ptr(initial_free_order, self.num_blocks, "initial_free_order")
        self._cpu_order, cpu_order = order_ptr(cpu_free_order, self.num_cpu_blocks, "cpu_free_order")
        self._h = lib().pa_pool_create_tiered(self.num_blocks, self.block_size, order,
                                              self.num_cpu_blocks, cpu_order)
        if not self._h:
            raise PagedAttentionError(PA_ERR_ARG, "pa_pool_create_tiered")

    def __del__(self):
        h = getattr(self, "_h", None)
        if h and _lib is not None:
            _lib.pa_pool_destroy(h)
            self._h = None

    def allocate(self, seq, n_tokens):
        _check(lib().pa_pool_allocate(self._h, int(seq), int(n_tokens)), "allocate")

    def append_slot(self, seq):
        """Returns (slot, cow) with cow None or the (src, dst) pair to copy before writing."""
        slot = ctypes.c_int64(0)
        src = ctypes.c_int32(-1)
        dst = ctypes.c_int32(-1)
        st = _check(lib().pa_pool_append_slot(self._h, int(seq), ctypes.byref(slot),
                                              ctypes.byref(src), ctypes.byref(dst)), "append_slot")
        return slot.value, ((src.value, dst.value) if st == 1 else None)

    def fork(self, parent, child):
        _check(lib().pa_pool_fork(self._h, int(parent), int(child)), "fork")

    def truncate(self, seq, n_tokens):
        """Keep the sequence's first n_tokens tokens (rejected drafts are given up)."""
        _check(lib().pa_pool_truncate(self._h, int(seq), int(n_tokens)), "truncate")

    def free(self, seq):
        _check(lib().pa_pool_free(self._h, int(seq)), "free")

    def block_table(self, seq):
        import numpy as np
        n = _check(lib().pa_pool_block_table(self._h, int(seq), None, 0), "block_table")
        out = np.zeros(n, dtype=np.int32)
        _check(lib().pa_pool_block_table(self._h, int(seq), out.ctypes.data, n), "block_table")
        return out

    def context_len(self, seq):
        return _check(lib().pa_pool_context_len(self._h, int(seq)), "context_len")

    def slots(self, seq, first, count):
        import numpy as np
        out = np.zeros(count, dtype=np.int64)
        _check(lib().pa_pool_slots(self._h, int(seq), int(first), int(count), out.ctypes.data), "slots")
        return out

    def num_free(self):
        return _check(lib().pa_pool_num_free(self._h), "num_free")

    def free_list(self):
        import numpy as np
        n = self.num_free()
        out = np.zeros(n, dtype=np.int32)
        _check(lib().pa_pool_free_list(self._h, out.ctypes.data, n), "free_list")
        return out

    def refcount(self, block):
        return _check(lib().pa_pool_refcount(self._h, int(block)), "refcount")

    def _move(self, fn, seqs, what):
        import numpy as np
        ids = np.ascontiguousarray(np.asarray(list(seqs), dtype=np.int64))
        cap = sum(len(self.block_table(int(s))) for s in set(ids.tolist())) if ids.size else 0
        pairs = np.zeros((max(cap, 1), 2), dtype=np.int32)
        n = _check(fn(self._h, ids.ctypes.data, ids.size, pairs.ctypes.data, cap), what)
        return pairs[:n]

    def swap_out(self, seqs):
        """Move a group of resident sequences to the CPU pool; returns the (device block,
        CPU block) pairs [n, 2] int32 to copy with swap_blocks."""
        return self._move(lib().pa_pool_swap_out, seqs, "swap_out")

    def swap_in(self, seqs):
        """Bring a group of swapped-out sequences back; returns (CPU block, device block)
        pairs."""
        return self._move(lib().pa_pool_swap_in, seqs, "swap_in")

    def is_swapped(self, seq):
        return bool(_check(lib().pa_pool_is_swapped(self._h, int(seq)), "is_swapped"))

    def num_free_cpu(self):
        return _check(lib().pa_pool_num_free_cpu(self._h), "num_free_cpu")

    def cpu_free_list(self):
        import numpy as np
        n = self.num_free_cpu()
        out = np.zeros(max(n, 1), dtype=np.int32)
        _check(lib().pa_pool_cpu_free_list(self._h, out.ctypes.data, n), "cpu_free_list")
        return out[:n]

    def cpu_refcount(self, block):
        return _check(lib().pa_pool_cpu_refcount(self._h, int(block)), "cpu_refcount")

    def allocate_prefix(self, seq, tokens, extra=b""):
        """Prefill with prefix caching; returns the number of leading tokens whose K/V
        the reused blocks already hold."""
        import numpy as np
        tok = np.ascontiguousarray(np.asarray(tokens, dtype=np.int32))
        ex = bytes(extra)
        cached = ctypes.c_int(0)
        _check(lib().pa_pool_allocate_prefix(self._h, int(seq), tok.ctypes.data, len(tok),
                                             ex or None, len(ex), ctypes.byref(cached)),
               "allocate_prefix")
        return cached.value

    def num_cached(self):
        return _check(lib().pa_pool_num_cached(self._h), "num_cached")

    def block_digest(self, block):
        out = ctypes.create_string_buffer(32)
        st = _check(lib().pa_pool_block_digest(self._h, int(block), out), "block_digest")
        return out.raw if st == 1 else None

    def allocate_prefix_batch(self, seq_ids, tokens, token_start, extras=None, extra_start=None,
                              table_width=None, out=None):
        """Place a batch of prompts through the prefix cache in one call (see
        pa_pool_allocate_prefix_batch).  tokens: int32 [total], token_start: int64 [n + 1].
        Returns (cached [n] int32, slots of the uncached tokens int64, tables [n, width]
        int32).  `out` may pass (cached, slots, tables) arrays to fill."""
        import numpy as np
        ids = np.ascontiguousarray(np.asarray(seq_ids, dtype=np.int64))
        n = ids.size
        tok = np.ascontiguousarray(np.asarray(tokens, dtype=np.int32))
        ts = np.ascontiguousarray(np.asarray(token_start, dtype=np.int64))
        _need(ts.shape == (n + 1,), "token_start must have n + 1 entries")
        lens = np.diff(ts)
        if table_width is None:
            table_width = _check(lib().pa_pool_table_width(self._h, n, ts.ctypes.data),
                                 "pa_pool_table_width")
        _need(n == 0 or (ts[0] >= 0 and ts[-1] <= tok.size and (lens >= 0).all()),
              "token_start must be non-decreasing within tokens")
        if out is None:
            cached = np.zeros(n, dtype=np.int32)
            slots = np.zeros(int(lens.sum()), dtype=np.int64)
            tables = np.zeros((n, table_width), dtype=np.int32)
        else:
            cached, slots, tables = out
            _host_out(cached, np.int32, n, "cached")
            _host_out(slots, np.int64, int(lens.sum()), "slots")
            _host_out(tables, np.int32, n * int(table_width), "tables")
        ex = es = None
        if extras is not None:
            ex = np.ascontiguousarray(np.frombuffer(bytes(extras), dtype=np.uint8)) if not \
                isinstance(extras, np.ndarray) else np.ascontiguousarray(extras, dtype=np.uint8)
            es = np.ascontiguousarray(np.asarray(extra_start, dtype=np.int64))
            _need(es.shape == (n + 1,), "extra_start must have n + 1 entries")
            _need(n == 0 or (es[0] >= 0 and es[-1] <= ex.size and (np.diff(es) >= 0).all()),
                  "extra_start must be non-decreasing within extras")
        done = ctypes.c_int(0)
        _check(lib().pa_pool_allocate_prefix_batch(
            self._h, n, ids.ctypes.data, tok.ctypes.data, ts.ctypes.data,
            None if ex is None else ex.ctypes.data, None if es is None else es.ctypes.data,
            cached.ctypes.data, slots.ctypes.data, tables.ctypes.data, int(table_width),
            ctypes.byref(done)), "allocate_prefix_batch")
        used = int((lens - cached).sum())
        return cached, slots[:used], tables

    def allocate_hashed_batch(self, seq_ids, n_tokens, digests, table_width, out=None):
        """Place a batch from digests computed earlier (bytes or uint8 array holding every
        request's full-block digests in order, as block_hashes returns them joined).
        Returns (cached, slots of the uncached tokens, tables)."""
        import numpy as np
        ids = np.ascontiguousarray(np.asarray(seq_ids, dtype=np.int64))
        n = ids.size
        nt = np.ascontiguousarray(np.asarray(n_tokens, dtype=np.int32))
        dg = np.ascontiguousarray(np.frombuffer(digests, dtype=np.uint8) if isinstance(
            digests, (bytes, bytearray)) else np.asarray(digests, dtype=np.uint8))
        _need(nt.shape == (n,), "n_tokens must have one entry a request")
        _need(dg.size >= 32 * int((np.maximum(nt, 0) // self.block_size).sum()),
              "digests must hold 32 bytes for every full block of every request")
        if out is None:
            cached = np.zeros(n, dtype=np.int32)
            slots = np.zeros(int(nt.sum()), dtype=np.int64)
            tables = np.zeros((n, table_width), dtype=np.int32)
        else:
            cached, slots, tables = out
            _host_out(cached, np.int32, n, "cached")
            _host_out(slots, np.int64, int(nt.sum()), "slots")
            _host_out(tables, np.int32, n * int(table_width), "tables")
        done = ctypes.c_int(0)
        _check(lib().pa_pool_allocate_hashed_batch(
            self._h, n, ids.ctypes.data, nt.ctypes.data, dg.ctypes.data if dg.size else None,
            cached.ctypes.data, slots.ctypes.data, tables.ctypes.data, int(table_width),
            ctypes.byref(done)), "allocate_hashed_batch")
        used = int((nt - cached).sum())
        return cached, slots[:used], tables

    def free_batch(self, seq_ids):
        import numpy as np
        ids = np.ascontiguousarray(np.asarray(seq_ids, dtype=np.int64))
        _check(lib().pa_pool_free_batch(self._h, ids.ctypes.data, ids.size), "free_batch")
