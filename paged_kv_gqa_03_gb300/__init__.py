"""Python binding of libpagedkv.so — paged GQA decode attention for sm_103a.

Argument marshalling only: every step of the decode path runs in the
library's CUDA kernels (or, for the block manager, its native host code).
PyTorch supplies device memory and streams.  Importing this package fails with
ImportError when the library has not been built — there is no fallback.

The function names are those of the C ABI in include/pagedkv.h, whose comments
define each operation, its layouts and its errors.
"""
import ctypes
import os

__all__ = [
    "PagedKVError", "paged_kv_append", "paged_decode_workspace_bytes",
    "paged_decode_attention", "paged_prefill_attention", "paged_decode_status", "paged_decode_merge",
    "paged_decode_attention_static", "paged_decode_static_status",
    "paged_kv4_append", "paged_kv4_pack_blocks", "paged_kv4_expand_blocks", "paged_kv4_copy_blocks",
    "paged_kv4_decode_workspace_bytes", "paged_kv4_decode_attention",
    "RopeTable", "paged_rope", "paged_rope_append", "paged_kv4_rope_append",
    "paged_tree_workspace_bytes", "paged_tree_attention", "paged_tree_verify", "paged_tree_commit",
    "paged_kv_copy_blocks", "pkv_copy", "pkv_status_string", "pkv_version", "pkv_set_route",
    "pkv_get_route", "pkv_test_stall_next", "BlockManager", "Prepared",
    "DTYPE_CODES", "LIB_PATH", "lib",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_build", "libpagedkv.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build the CUDA library first "
        "(python paged_kv_gqa_03_gb300/build.py, or __graft_entry__.build())")

_P, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
_L = ctypes.CDLL(LIB_PATH)


def _sig(name, res, *args):
    fn = getattr(_L, name)
    fn.restype = res
    fn.argtypes = list(args)
    return fn


_sig("paged_kv_append", _i32, _P, _P, _i32, _P, _P, _i32, _P, _P, _P, _i32, _i32, _i32, _i64, _P)
_sig("paged_kv_append_calibrated", _i32, _P, _P, _i32, _P, _P, _i32, _P, _P, _P, _i32, _i32, _i32, _i64, _P)
_sig("paged_decode_workspace_bytes", _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
     ctypes.POINTER(_sz))
_sig("paged_decode_attention", _i32, _P, _P, _i32, _P, _P, _i32, _P, _P, _P, _i32, _P,
     _i32, _i32, _i32, _i32, _i64, ctypes.c_float, _i32, _P, _sz, _P)
_sig("paged_decode_multi_workspace_bytes", _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
     ctypes.POINTER(_sz))
_sig("paged_decode_attention_multi", _i32, _P, _P, _i32, _P, _P, _i32, _P, _P, _P, _i32, _P,
     _i32, _i32, _i32, _i32, _i32, _i32, _i64, ctypes.c_float, _i32, _P, _sz, _P)
_sig("paged_prefill_attention", _i32, _P, _P, _i32, _P, _P, _i32, _P, _i32, _P, _P,
     _i32, _i32, _i32, _i32, _i32, _i64, ctypes.c_float, _i32, _P, _P)
_sig("paged_tree_workspace_bytes", _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, ctypes.POINTER(_sz))
_sig("paged_tree_attention", _i32, _P, _P, _i32, _P, _P, _i32, _P, _P, _P, _i32, _P, _P, _i32, _P,
     _i32, _i32, _i32, _i32, _i32, _i32, _i64, ctypes.c_float, _P, _sz, _P)
_sig("paged_tree_verify", _i32, _P, _P, _P, _P, _P, _i32, _P, _P, _i64, _P, _i64, _i32, _P,
     _i32, _i32, _i32, _P)
_sig("paged_tree_commit", _i32, _P, _P, _i32, _P, _P, _P, _P, _P, _i32, _P, _P, _P,
     _i32, _i32, _i32, _i32, _i64, _P)
_sig("paged_tree_commit_calibrated", _i32, _P, _P, _i32, _P, _P, _P, _P, _P, _i32, _P, _P, _P,
     _i32, _i32, _i32, _i32, _i64, _P)
_sig("paged_decode_status", _i32, _P, _sz, _P, ctypes.POINTER(_i32))
_sig("paged_decode_attention_static", _i32, _P, _P, _i32, _P, _P, _i32, _P, _P, _P, _i32, _P,
     _i32, _i32, _i32, _i32, _i64, ctypes.c_float, _i32, _P)
_sig("paged_decode_static_status", _i32, _P, ctypes.POINTER(_i32))
_sig("paged_decode_merge", _i32, _P, _i32, _P, _P, _i32, _i32, _i32, _i32, _P)
_sig("paged_kv_copy_blocks", _i32, _P, _P, _i32, _P, _P, _P, _i32, _i32, _i32, _i64, _P)
_f32 = ctypes.c_float
_sig("paged_kv4_tile_bytes", _i64, _i32)
_sig("paged_kv4_append", _i32, _P, _i64, _P, _i64, _i32, _P, _P, _i32, _i32, _i32, _i64, _f32, _f32, _P)
_sig("paged_kv4_pack_blocks", _i32, _P, _i64, _P, _P, _i32, _i64, _P, _i32, _i32, _i32, _f32, _f32, _P)
_sig("paged_kv4_expand_blocks", _i32, _P, _P, _i32, _i64, _P, _i64, _P, _i32, _i32, _i32, _f32, _f32, _P)
_sig("paged_kv4_copy_blocks", _i32, _P, _P, _i32, _i32, _i32, _i64, _P)
_sig("paged_kv4_decode_workspace_bytes", _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, ctypes.POINTER(_sz))
_sig("paged_kv4_decode_attention", _i32, _P, _P, _i32, _P, _P, _i32, _P, _i32, _i32, _i32, _i32, _i32, _i32,
     _i64, _f32, _f32, _f32, _i32, _P, _sz, _P)
_sig("pkv_rope_turns", _i32, _P, _P, _i32)
_sig("paged_rope", _i32, _P, _i64, _P, _i64, _P, _i64, _P, _i64, _i32, _P, _P, _i32, _i32, _f32,
     _i32, _i32, _i32, _i32, _P)
_sig("paged_rope_append", _i32, _P, _i64, _P, _i64, _P, _i64, _P, _i64, _i32, _P, _P, _i32, _i32, _f32,
     _P, _P, _P, _i32, _i32, _i32, _i32, _i64, _P)
_sig("paged_kv4_rope_append", _i32, _P, _i64, _P, _i64, _P, _i64, _P, _i64, _i32, _P, _P, _i32, _i32, _f32,
     _P, _P, _i32, _i32, _i32, _i32, _i64, _f32, _f32, _P)
_sig("pkv_copy", _i32, _P, _P, _sz, _P)
_sig("pkv_status_string", ctypes.c_char_p, _i32)
_sig("pkv_last_cuda_error", _i32)
_sig("pkv_version", _i32)
_sig("pkv_set_route", _i32, _i32, _i32)
_sig("pkv_get_route", _i32, _i32)
_sig("pkv_test_stall_next", _i32, _i32, ctypes.c_uint64)
_sig("pkv_bm_create", _P, _i64)
_sig("pkv_bm_destroy", None, _P)
_sig("pkv_bm_allocate", _i32, _P, _i64, _i64)
_sig("pkv_bm_adopt", _i32, _P, _i64, _P, _i32, _i64)
_sig("pkv_bm_fork", _i32, _P, _i64, _i64)
_sig("pkv_bm_free", _i32, _P, _i64)
_sig("pkv_bm_release_window", _i32, _P, _i64, _i64, ctypes.POINTER(_i64))
_sig("pkv_bm_truncate", _i32, _P, _i64, _i64)
_sig("pkv_bm_append_slots", _i32, _P, _P, _i32, _P, _P, ctypes.POINTER(_i32))
_sig("pkv_bm_export", _i32, _P, _P, _i32, _P, _i32, _P)
_sig("pkv_bm_num_free", _i64, _P)
_sig("pkv_bm_refcount", _i32, _P, _i64)
_sig("pkv_bm_num_tokens", _i64, _P, _i64)

PKV_OK, PKV_EINVAL, PKV_EUNSUPPORTED, PKV_EWORKSPACE = 0, -1, -2, -3
PKV_ECUDA, PKV_ETIMEOUT, PKV_EOOM, PKV_ERANGE, PKV_ENOTFOUND = -4, -5, -6, -7, -8
PKV_FLAG_TIMEOUT, PKV_FLAG_BAD_LEN, PKV_FLAG_BAD_BLOCK, PKV_FLAG_RANGE = 1, 2, 4, 8
PKV_STATIC_SCRATCH_BYTES = 16 << 20


def lib():
    """The loaded ctypes library (raw C ABI)."""
    return _L


class PagedKVError(RuntimeError):
    def __init__(self, status, where):
        msg = _L.pkv_status_string(status).decode()
        if status == PKV_ECUDA:
            msg += f" (cudaError {_L.pkv_last_cuda_error()})"
        super().__init__(f"{where}: {msg} [{status}]")
        self.status = status


def _check(status, where):
    if status != PKV_OK:
        raise PagedKVError(status, where)


def pkv_status_string(status):
    return _L.pkv_status_string(status).decode()


def pkv_version():
    return _L.pkv_version()


# Kernel-route decisions that pkv_set_route can force (include/pagedkv.h).
ROUTES = {"multi_query": (0, ("auto", "transposed", "prefill", "units")),
          "prefill": (1, ("auto", "persistent", "tiles")),
          "tree": (2, ("auto", "tiles", "units"))}


def pkv_set_route(which, choice):
    """Forces one kernel-route decision process-wide ("multi_query":
    auto / transposed / prefill / units; "prefill": auto / persistent /
    tiles; "tree": auto / tiles / units); returns the previous choice.  "auto" restores the library's rule."""
    idx, names = ROUTES[which]
    prev = names[_L.pkv_get_route(idx)]
    _check(_L.pkv_set_route(idx, names.index(choice)), "pkv_set_route")
    return prev


def pkv_test_stall_next(which, limit_ns):
    """Failure-path test hook: the next call that launches the "decode" or
    "prefill" kernel family runs out a wait on a barrier nothing completes
    (every wait of that call limited to limit_ns) and reports
    PKV_FLAG_TIMEOUT; see include/pagedkv.h."""
    _check(_L.pkv_test_stall_next({"decode": 0, "prefill": 1}[which], int(limit_ns)),
           "pkv_test_stall_next")


def pkv_get_route(which):
    idx, names = ROUTES[which]
    return names[_L.pkv_get_route(idx)]


_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _dtype_codes():
    torch = _torch()
    return {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2, torch.float8_e4m3fn: 3}


DTYPE_CODES = None


def _code(t):
    global DTYPE_CODES
    if DTYPE_CODES is None:
        DTYPE_CODES = _dtype_codes()
    try:
        return DTYPE_CODES[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}") from None


def _dev(t, name, dtype=None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _out(t):
    """The output pointer of a decode call: a CUDA tensor, or pinned host
    memory that the kernels write directly (see include/pagedkv.h)."""
    if t.is_cuda:
        return _dev(t, "out")
    if not t.is_pinned():
        raise ValueError("out must be a CUDA tensor or pinned host memory")
    if not t.is_contiguous():
        raise ValueError("out must be contiguous")
    return t.data_ptr()


def _stream(stream, device=None):
    """The raw stream: the current one of `device` (None: the current device)
    when none is given."""
    if stream is None:
        torch = _torch()
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if device is None else device)
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _workspace(nbytes, device, stream):
    """A workspace for a call on `stream` (None: the current one), allocated by
    torch as that stream's memory: if the caller drops it while the call runs,
    it is handed out again behind the call."""
    torch = _torch()
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


class Prepared:
    """One C call with its arguments marshalled once (returned by the calls
    below when given prepare=True): calling it issues the call again on the
    same buffers and stream, for a decode loop that runs the same step every
    iteration.  The buffers must stay alive and keep their addresses; a
    workspace that the call allocated itself is kept here (`workspace`)."""

    __slots__ = ("fn", "args", "name", "workspace")

    def __init__(self, fn, args, name, workspace=None):
        self.fn, self.args, self.name, self.workspace = fn, args, name, workspace

    def __call__(self):
        rc = self.fn(*self.args)
        if rc != PKV_OK:
            raise PagedKVError(rc, self.name)


def paged_kv_append(k_new, v_new, k_cache, v_cache, slot_mapping, k_scale=None, v_scale=None,
                    stream=None, calibrated=False, prepare=False):
    """Writes k_new/v_new [B, Hkv, D] into the caches [num_blocks, Hkv, 16, D]
    at slot_mapping[b] (int64; < 0 skips).  calibrated=True: FP8 block scales
    follow the block's running max (paged_kv_append_calibrated)."""
    torch = _torch()
    B, Hkv, D = k_new.shape
    fn = _L.paged_kv_append_calibrated if calibrated else _L.paged_kv_append
    args = (_dev(k_new, "k_new"), _dev(v_new, "v_new"), _code(k_new),
            _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"), _code(k_cache),
            _dev(k_scale, "k_scale", torch.float32), _dev(v_scale, "v_scale", torch.float32),
            _dev(slot_mapping, "slot_mapping", torch.int64), B, Hkv, D, k_cache.shape[0],
            _stream(stream))
    if prepare:
        return Prepared(fn, args, "paged_kv_append")
    _check(fn(*args), "paged_kv_append")


def paged_decode_workspace_bytes(B, Hq, Hkv, D, cache_dtype, q_dtype, num_splits=0, q_len=1):
    """Workspace size for paged_decode_attention (q_len new tokens per
    sequence) on the current device.  dtypes are torch dtypes or C codes."""
    conv = lambda d: d if isinstance(d, int) else _code(_torch().empty(0, dtype=d))
    out = _sz(0)
    if q_len == 1:
        rc = _L.paged_decode_workspace_bytes(B, Hq, Hkv, D, conv(cache_dtype), conv(q_dtype),
                                             num_splits, ctypes.byref(out))
    else:
        rc = _L.paged_decode_multi_workspace_bytes(B, q_len, Hq, Hkv, D, conv(cache_dtype),
                                                   conv(q_dtype), num_splits, ctypes.byref(out))
    _check(rc, "paged_decode_workspace_bytes")
    return out.value


def paged_decode_attention(out, q, k_cache, v_cache, block_table, context_lens, scale,
                           k_scale=None, v_scale=None, num_splits=0, workspace=None, stream=None,
                           window=0, prepare=False):
    """out[b, hq] = softmax(scale * q[b, hq] . K_b^T) V_b over the paged cache.

    q, out [B, Hq, D]: one new token per sequence (paged_decode_attention).
    q, out [B, q_len, Hq, D]: q_len new tokens per sequence, token i seeing
    the cache up to its own position (paged_decode_attention_multi).
    window > 0: each row sees only its `window` most recent positions.
    workspace: a uint8 CUDA tensor of paged_decode_workspace_bytes(...) bytes;
    allocated here (by torch) when None.  prepare=True returns the call as a
    Prepared object, which holds the workspace, instead of issuing it."""
    torch = _torch()
    if q.dim() == 4:
        B, q_len, Hq, D = q.shape
    else:
        (B, Hq, D), q_len = q.shape, 1
    if tuple(out.shape) != tuple(q.shape):
        raise ValueError(f"out shape {tuple(out.shape)} != q shape {tuple(q.shape)}")
    num_blocks, Hkv = k_cache.shape[0], k_cache.shape[1]
    if workspace is None:
        n = paged_decode_workspace_bytes(B, Hq, Hkv, D, _code(k_cache), _code(q), num_splits,
                                         q_len=q_len)
        workspace = _workspace(n, q.device, stream)
    args = (_dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
            _code(k_cache), _dev(k_scale, "k_scale", torch.float32),
            _dev(v_scale, "v_scale", torch.float32), _dev(block_table, "block_table", torch.int32),
            block_table.shape[1], _dev(context_lens, "context_lens", torch.int32))
    tail = (num_blocks, float(scale), num_splits, _dev(workspace, "workspace"),
            workspace.numel() * workspace.element_size(), _stream(stream))
    if q.dim() == 4 or window:
        fn, name = _L.paged_decode_attention_multi, "paged_decode_attention_multi"
        full = (_out(out), _dev(q, "q"), _code(q), *args, B, q_len, int(window), Hq, Hkv, D, *tail)
    else:
        fn, name = _L.paged_decode_attention, "paged_decode_attention"
        full = (_out(out), _dev(q, "q"), _code(q), *args, B, Hq, Hkv, D, *tail)
    if prepare:
        return Prepared(fn, full, name, workspace)
    _check(fn(*full), name)
    return workspace


def paged_prefill_attention(out, q, k_cache, v_cache, block_table, context_lens, q_start, max_q_len,
                            scale, window=0, status=None, stream=None):
    """Causal attention of each sequence's new tokens over its paged cache
    (tensor cores).  q, out [total, Hq, D]; q_start int32 [B+1] row offsets;
    max_q_len >= every sequence's new-token count; status: optional int32
    CUDA tensor that receives the PKV_FLAG_* bits."""
    torch = _torch()
    total, Hq, D = q.shape
    if tuple(out.shape) != tuple(q.shape):
        raise ValueError(f"out shape {tuple(out.shape)} != q shape {tuple(q.shape)}")
    B = q_start.shape[0] - 1
    num_blocks, Hkv = k_cache.shape[0], k_cache.shape[1]
    _check(_L.paged_prefill_attention(
        _out(out), _dev(q, "q"), _code(q), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
        _code(k_cache), _dev(block_table, "block_table", torch.int32), block_table.shape[1],
        _dev(context_lens, "context_lens", torch.int32), _dev(q_start, "q_start", torch.int32),
        B, int(max_q_len), Hq, Hkv, D, num_blocks, float(scale), int(window),
        _dev(status, "status", torch.int32), _stream(stream)), "paged_prefill_attention")


def _arg(t, name, dtype, shape, device):
    """The pointer of a contiguous tensor of this type and shape on CUDA device
    `device` (an index).  One test on the way through; what is wrong is looked
    for only when it fails."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == device:
        return t.data_ptr()
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    _dev(t, name)   # a CUDA tensor, contiguous
    raise ValueError(f"{name} is on {t.device}, expected cuda:{device}")


def _device_of(t, name):
    """The CUDA device a call runs on, from one of its tensors: it must be the
    current device, whose stream and context the call uses."""
    d = t.get_device()
    if d < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if d != _torch().cuda.current_device():
        raise ValueError(f"{name} is on cuda:{d}: make it the current device (torch.cuda.device)")
    return d


def _cache(k_cache, v_cache, k_scale, v_scale, device):
    """Checks a cache's tensors; (k, v, k scale, v scale pointers, num_blocks, Hkv, D)."""
    shape = k_cache.shape
    if len(shape) != 4 or shape[2] != 16:
        raise ValueError(f"k_cache must be [num_blocks, Hkv, 16, D], got {tuple(shape)}")
    dtype, f32, sc = k_cache.dtype, _torch().float32, shape[:2]
    return (_arg(k_cache, "k_cache", dtype, shape, device), _arg(v_cache, "v_cache", dtype, shape, device),
            None if k_scale is None else _arg(k_scale, "k_scale", f32, sc, device),
            None if v_scale is None else _arg(v_scale, "v_scale", f32, sc, device), shape[0], shape[1], shape[3])


def _table(block_table, B, device):
    """(pointer, max_blocks) of an int32 [B, max_blocks] table."""
    if block_table.dim() != 2:
        raise ValueError(f"block_table must be [B, max_blocks], got {tuple(block_table.shape)}")
    mb = block_table.shape[1]
    return _arg(block_table, "block_table", _torch().int32, (B, mb), device), mb


def _tree_mask(tree_mask, B, n, device):
    """(pointer, mask_per_seq) of an int64 [n] or [B, n] mask."""
    if tree_mask.dim() == 1:
        return _arg(tree_mask, "tree_mask", _torch().int64, (n,), device), 0
    return _arg(tree_mask, "tree_mask", _torch().int64, (B, n), device), 1


def paged_tree_workspace_bytes(B, q_len, Hq, Hkv, D, cache_dtype, q_dtype):
    """Workspace size for paged_tree_attention on the current device.  dtypes
    are torch dtypes or C codes."""
    conv = lambda d: d if isinstance(d, int) else _code(_torch().empty(0, dtype=d))
    out = _sz(0)
    _check(_L.paged_tree_workspace_bytes(B, q_len, Hq, Hkv, D, conv(cache_dtype), conv(q_dtype),
                                         ctypes.byref(out)), "paged_tree_workspace_bytes")
    return out.value


def paged_tree_attention(out, q, k_cache, v_cache, block_table, context_lens, tree_mask, scale,
                         tree_lens=None, k_scale=None, v_scale=None, window=0, workspace=None,
                         stream=None, prepare=False):
    """Attention of a tree of drafted tokens over the paged cache.

    q, out [B, q_len, Hq, D]: row i is the tree's node i, the cache's position
    context_lens[b] - n_b + i; it sees the positions before the tree and the
    nodes in its mask.  tree_mask int64 [B, q_len], or [q_len] for one tree
    shared by all sequences; tree_lens int32 [B]: n_b (None: q_len each; rows
    past n_b of out are left as they were).  workspace: a uint8 CUDA tensor of
    paged_tree_workspace_bytes(...) bytes, allocated here (by torch) when None;
    returned for paged_decode_status.  prepare=True returns the call as a
    Prepared object, which holds the workspace, instead of issuing it."""
    torch = _torch()
    shape = q.shape
    if len(shape) != 4:
        raise ValueError(f"q must be [B, q_len, Hq, D], got {tuple(shape)}")
    B, n, Hq, D = shape
    dev, dtype, i32 = _device_of(q, "q"), q.dtype, torch.int32
    k, v, ks, vs, num_blocks, Hkv, Dc = _cache(k_cache, v_cache, k_scale, v_scale, dev)
    if Dc != D:
        raise ValueError(f"q has head dim {D}, the cache {Dc}")
    table, max_blocks = _table(block_table, B, dev)
    mask, per_seq = _tree_mask(tree_mask, B, n, dev)
    if out.is_cuda:
        o = _arg(out, "out", dtype, shape, dev)
    else:   # pinned host memory, as for the other calls that write an output
        o = _out(out)
        if out.shape != shape or out.dtype is not dtype:
            raise ValueError(f"out must be {dtype} of shape {tuple(shape)}")
    qc, kc = _code(q), _code(k_cache)
    if workspace is None:
        workspace = _workspace(paged_tree_workspace_bytes(B, n, Hq, Hkv, D, kc, qc), q.device, stream)
    args = (o, _arg(q, "q", dtype, shape, dev), qc, k, v, kc, ks, vs, table, max_blocks,
            _arg(context_lens, "context_lens", i32, (B,), dev), mask, per_seq,
            None if tree_lens is None else _arg(tree_lens, "tree_lens", i32, (B,), dev), B, n, int(window), Hq, Hkv, D,
            num_blocks, float(scale), _arg(workspace, "workspace", workspace.dtype, workspace.shape, dev),
            workspace.nbytes, _stream(stream, dev))
    if prepare:
        return Prepared(_L.paged_tree_attention, args, "paged_tree_attention", workspace)
    rc = _L.paged_tree_attention(*args)
    if rc != PKV_OK:
        raise PagedKVError(rc, "paged_tree_attention")
    return workspace


def _rows(t, name, dtype, B, n, V, device):
    """(pointer, row distance) of [B, n, V] rows a fixed number of elements
    apart (a slice of a wider vocabulary is such a tensor)."""
    if t.shape != (B, n, V):
        raise ValueError(f"{name} must be [{B}, {n}, {V}], got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}, is on {t.device}")
    if t.is_contiguous():
        return t.data_ptr(), V
    sb, sn, sv = t.stride()
    ld = sn if n > 1 else (sb if B > 1 else V)
    if (V > 1 and sv != 1) or ld < V or (B > 1 and n > 1 and sb != n * sn):
        raise ValueError(f"{name} must have contiguous rows a fixed distance apart, got strides {t.stride()}")
    return t.data_ptr(), ld


def paged_tree_verify(path, path_len, next_token, draft_tokens, tree_mask, target_probs,
                      draft_probs=None, uniforms=None, tree_lens=None, stream=None, prepare=False):
    """Accepts a path of the tree's drafted tokens from the target's
    probabilities (see include/pagedkv.h for the rule) and draws the next token.

    Writes path int32 [B, n] (accepted nodes, then -1), path_len int32 [B] and
    next_token int64 [B].  draft_tokens int64 [B, n]; target_probs, draft_probs
    [B, n, V] fp32 / fp16 / bf16 of one type, rows a fixed distance apart;
    uniforms fp32 [B, n].  With draft_probs: sampled drafts, a node's children
    drawn independently from its row; without: each
    node's deterministic continuations; without uniforms too: greedy."""
    torch = _torch()
    i32, i64 = torch.int32, torch.int64
    shape = draft_tokens.shape
    if len(shape) != 2:
        raise ValueError(f"draft_tokens must be [B, n], got {tuple(shape)}")
    B, n = shape
    if target_probs.dim() != 3:
        raise ValueError(f"target_probs must be [{B}, {n}, V], got {tuple(target_probs.shape)}")
    dev, V, dtype = _device_of(target_probs, "target_probs"), target_probs.shape[2], target_probs.dtype
    mask, per_seq = _tree_mask(tree_mask, B, n, dev)
    target, ld_t = _rows(target_probs, "target_probs", dtype, B, n, V, dev)
    draft, ld_d = (None, 0) if draft_probs is None else _rows(draft_probs, "draft_probs", dtype, B, n, V, dev)
    args = (_arg(path, "path", i32, shape, dev), _arg(path_len, "path_len", i32, (B,), dev),
            _arg(next_token, "next_token", i64, (B,), dev), _arg(draft_tokens, "draft_tokens", i64, shape, dev),
            mask, per_seq, None if tree_lens is None else _arg(tree_lens, "tree_lens", i32, (B,), dev), target, ld_t,
            draft, ld_d, _code(target_probs),
            None if uniforms is None else _arg(uniforms, "uniforms", torch.float32, shape, dev), B, n, V,
            _stream(stream, dev))
    if prepare:
        return Prepared(_L.paged_tree_verify, args, "paged_tree_verify")
    rc = _L.paged_tree_verify(*args)
    if rc != PKV_OK:
        raise PagedKVError(rc, "paged_tree_verify")


def paged_tree_commit(k_cache, v_cache, path, path_len, block_table, context_lens, k_scale=None,
                      v_scale=None, tree_lens=None, new_lens=None, stream=None, prepare=False, calibrated=False):
    """Moves the accepted path's K/V rows together in the paged cache, in
    place: position context_lens[b] - n_b + k takes the row of node path[b, k].
    new_lens (optional int32 [B], memory of its own) receives the lengths that
    remain.  calibrated=True, for caches of the calibrated append: FP8 block
    scales follow the rows moved in, so that none saturates
    (paged_tree_commit_calibrated)."""
    i32 = _torch().int32
    shape = path.shape
    if len(shape) != 2:
        raise ValueError(f"path must be [B, n], got {tuple(shape)}")
    B, n = shape
    dev, one = _device_of(k_cache, "k_cache"), (B,)
    k, v, ks, vs, num_blocks, Hkv, D = _cache(k_cache, v_cache, k_scale, v_scale, dev)
    table, max_blocks = _table(block_table, B, dev)
    rows, row_lens = _arg(path, "path", i32, shape, dev), _arg(path_len, "path_len", i32, one, dev)
    lens = _arg(context_lens, "context_lens", i32, one, dev)
    nodes = None if tree_lens is None else _arg(tree_lens, "tree_lens", i32, one, dev)
    new = None
    if new_lens is not None:   # the call still reads the others when it writes it
        new, per = _arg(new_lens, "new_lens", i32, one, dev), 4 * B
        if (abs(new - lens) < per or abs(new - row_lens) < per or (nodes is not None and abs(new - nodes) < per)
                or rows - per < new < rows + per * n or table - per < new < table + per * max_blocks):
            raise ValueError("new_lens must not share memory with context_lens, tree_lens, path_len, path or block_table")
    args = (k, v, _code(k_cache), ks, vs, rows, row_lens, table, max_blocks, lens, nodes, new, B, n, Hkv, D, num_blocks,
            _stream(stream, dev))
    fn = _L.paged_tree_commit_calibrated if calibrated else _L.paged_tree_commit
    if prepare:
        return Prepared(fn, args, "paged_tree_commit")
    rc = fn(*args)
    if rc != PKV_OK:
        raise PagedKVError(rc, "paged_tree_commit")


def paged_decode_status(workspace, stream=None):
    """Synchronises the stream; returns the PKV_FLAG_* bits the last decode
    recorded in `workspace` (raises on a timeout or range flag)."""
    flags = _i32(0)
    rc = _L.paged_decode_status(_dev(workspace, "workspace"),
                                workspace.numel() * workspace.element_size(), _stream(stream),
                                ctypes.byref(flags))
    if rc not in (PKV_OK, PKV_ETIMEOUT, PKV_ERANGE):
        _check(rc, "paged_decode_status")
    return rc, flags.value


def paged_decode_attention_static(out, q, k_cache, v_cache, block_table, context_lens, scale,
                                  k_scale=None, v_scale=None, num_splits=0, stream=None):
    """paged_decode_attention (one new token per sequence, q, out [B, Hq, D])
    on the scratch array the library keeps on each GPU instead of a caller's
    workspace, for callers that cannot allocate device memory.  Calls on one
    GPU share that array: they must not overlap on the GPU."""
    torch = _torch()
    B, Hq, D = q.shape
    if tuple(out.shape) != tuple(q.shape):
        raise ValueError(f"out shape {tuple(out.shape)} != q shape {tuple(q.shape)}")
    num_blocks, Hkv = k_cache.shape[0], k_cache.shape[1]
    _check(_L.paged_decode_attention_static(
        _out(out), _dev(q, "q"), _code(q), _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"),
        _code(k_cache), _dev(k_scale, "k_scale", torch.float32), _dev(v_scale, "v_scale", torch.float32),
        _dev(block_table, "block_table", torch.int32), block_table.shape[1],
        _dev(context_lens, "context_lens", torch.int32), B, Hq, Hkv, D, num_blocks, float(scale),
        num_splits, _stream(stream)), "paged_decode_attention_static")


def paged_decode_static_status(stream=None):
    """paged_decode_status for the static scratch of the current device:
    (status, PKV_FLAG_* bits) of the last paged_decode_attention_static."""
    flags = _i32(0)
    rc = _L.paged_decode_static_status(_stream(stream), ctypes.byref(flags))
    if rc not in (PKV_OK, PKV_ETIMEOUT, PKV_ERANGE):
        _check(rc, "paged_decode_static_status")
    return rc, flags.value


def paged_decode_merge(out, o_partial, lse, stream=None):
    """out [B, Hq, D] from o_partial [B, Hq, S, D] fp32 and lse [B, Hq, S] fp32."""
    torch = _torch()
    B, Hq, S, D = o_partial.shape
    _check(_L.paged_decode_merge(_dev(out, "out"), _code(out),
                                 _dev(o_partial, "o_partial", torch.float32),
                                 _dev(lse, "lse", torch.float32), B, Hq, D, S, _stream(stream)),
           "paged_decode_merge")


def pkv_copy(dst, src, nbytes=None, stream=None):
    """SM-driven copy of nbytes (default: all of src) between CUDA tensors
    and/or pinned host tensors (see include/pagedkv.h)."""
    for t, name in ((dst, "dst"), (src, "src")):
        if not (t.is_cuda or t.is_pinned()):
            raise ValueError(f"{name} must be a CUDA tensor or pinned host memory")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    n = src.numel() * src.element_size() if nbytes is None else nbytes
    _check(_L.pkv_copy(dst.data_ptr(), src.data_ptr(), n, _stream(stream)), "pkv_copy")


def paged_kv_copy_blocks(k_cache, v_cache, src_dst_pairs, k_scale=None, v_scale=None, stream=None):
    """cache[dst] = cache[src] for each (src, dst) row of the int32 [n, 2] tensor."""
    torch = _torch()
    n = src_dst_pairs.shape[0]
    _check(_L.paged_kv_copy_blocks(
        _dev(k_cache, "k_cache"), _dev(v_cache, "v_cache"), _code(k_cache),
        _dev(k_scale, "k_scale", torch.float32), _dev(v_scale, "v_scale", torch.float32),
        _dev(src_dst_pairs, "src_dst_pairs", torch.int32), n, k_cache.shape[1],
        k_cache.shape[3], k_cache.shape[0], _stream(stream)), "paged_kv_copy_blocks")


def _issue(fn, args, name, prepare, workspace=None):
    if prepare:
        return Prepared(fn, args, name, workspace)
    rc = fn(*args)
    if rc != PKV_OK:
        raise PagedKVError(rc, name)
    return workspace


def _token_rows(t, name, shape, dtype, device):
    """(pointer, elements from a token to the next) of rows [T, heads, D] whose
    heads lie side by side; a token's row may be a part of a wider one."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == device:   # one test on the way through
        ld, sh, sd = t.stride()
        T, heads, D = shape
        if T > 1 and sh == D and sd == 1:
            return t.data_ptr(), ld
        if t.numel() == 0 or (sd == 1 and (sh == D or heads == 1)):
            return t.data_ptr(), (ld if T > 1 else heads * D)
        raise ValueError(f"{name}: the {heads} heads of a token must lie side by side, strides {t.stride()}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} is on {t.device}, expected cuda:{device}")


def _cache4(cache, device):
    """(pointer, num_blocks, Hkv, D) of a 4-bit cache, uint8 [num_blocks, Hkv, 18 D]."""
    shape = cache.shape
    if len(shape) == 3:
        num_blocks, Hkv, tile = shape
        if tile == 18 * 128 or tile == 18 * 64:
            return _arg(cache, "cache", _torch().uint8, shape, device), num_blocks, Hkv, tile // 18
    raise ValueError(f"a 4-bit cache must be [num_blocks, Hkv, 18 * D], D 64 or 128, got {tuple(shape)}")


def paged_kv4_append(k_new, v_new, cache, slot_mapping, k_unit=1.0, v_unit=1.0, stream=None, prepare=False):
    """Quantises k_new / v_new [T, Hkv, D] (f32, f16 or bf16; a token's row may
    be a slice of a wider one) into the 4-bit cache, uint8 [num_blocks, Hkv,
    18 * D], at slot_mapping [T] (int64; < 0 skips)."""
    dev = _device_of(cache, "cache")
    ptr, num_blocks, Hkv, D = _cache4(cache, dev)
    T, dtype = k_new.shape[0], k_new.dtype
    shape = (T, Hkv, D)
    k, ld_k = _token_rows(k_new, "k_new", shape, dtype, dev)
    v, ld_v = _token_rows(v_new, "v_new", shape, dtype, dev)
    args = (k, ld_k, v, ld_v, _code(k_new), ptr, _arg(slot_mapping, "slot_mapping", _torch().int64, (T,), dev),
            T, Hkv, D, num_blocks, float(k_unit), float(v_unit), _stream(stream, dev))
    return _issue(_L.paged_kv4_append, args, "paged_kv4_append", prepare)


def _pages(cache, k_cache, v_cache, pairs):
    dev = _device_of(cache, "cache")
    ptr, num_blocks, Hkv, D = _cache4(cache, dev)
    others, n, dtype = k_cache.shape[0], pairs.shape[0], k_cache.dtype
    shape = (others, Hkv, 16, D)
    k, v = _arg(k_cache, "k_cache", dtype, shape, dev), _arg(v_cache, "v_cache", dtype, shape, dev)
    return dev, ptr, num_blocks, k, v, others, _arg(pairs, "src_dst_pairs", _torch().int32, (n, 2), dev), n, Hkv, D


def paged_kv4_pack_blocks(cache, k_cache, v_cache, src_dst_pairs, k_unit=1.0, v_unit=1.0, stream=None,
                          prepare=False):
    """4-bit block dst of cache = quantised block src of k_cache / v_cache
    [blocks, Hkv, 16, D] (f32, f16, bf16), for each (src, dst) of int32 [n, 2]."""
    dev, ptr, num_blocks, k, v, src, pairs, n, Hkv, D = _pages(cache, k_cache, v_cache, src_dst_pairs)
    args = (ptr, num_blocks, k, v, _code(k_cache), src, pairs, n, Hkv, D, float(k_unit), float(v_unit),
            _stream(stream, dev))
    return _issue(_L.paged_kv4_pack_blocks, args, "paged_kv4_pack_blocks", prepare)


def paged_kv4_expand_blocks(k_cache, v_cache, cache, src_dst_pairs, k_unit=1.0, v_unit=1.0, stream=None,
                            prepare=False):
    """Block dst of k_cache / v_cache [blocks, Hkv, 16, D] (f32, f16, bf16) =
    the values of 4-bit block src of cache, for each (src, dst) of int32 [n, 2]."""
    dev, ptr, num_blocks, k, v, dst, pairs, n, Hkv, D = _pages(cache, k_cache, v_cache, src_dst_pairs)
    args = (k, v, _code(k_cache), dst, ptr, num_blocks, pairs, n, Hkv, D, float(k_unit), float(v_unit),
            _stream(stream, dev))
    return _issue(_L.paged_kv4_expand_blocks, args, "paged_kv4_expand_blocks", prepare)


def paged_kv4_copy_blocks(cache, src_dst_pairs, stream=None, prepare=False):
    """cache[dst] = cache[src] for each (src, dst) row of the int32 [n, 2] tensor (copy on write)."""
    dev = _device_of(cache, "cache")
    ptr, num_blocks, Hkv, D = _cache4(cache, dev)
    n = src_dst_pairs.shape[0]
    args = (ptr, _arg(src_dst_pairs, "src_dst_pairs", _torch().int32, (n, 2), dev), n, Hkv, D, num_blocks,
            _stream(stream, dev))
    return _issue(_L.paged_kv4_copy_blocks, args, "paged_kv4_copy_blocks", prepare)


def paged_kv4_decode_workspace_bytes(B, Hq, Hkv, D, q_dtype, num_splits=0, q_len=1):
    """Workspace size for paged_kv4_decode_attention on the current device.
    q_dtype: a torch dtype or C code."""
    code = q_dtype if isinstance(q_dtype, int) else _code(_torch().empty(0, dtype=q_dtype))
    out = _sz(0)
    _check(_L.paged_kv4_decode_workspace_bytes(B, q_len, Hq, Hkv, D, code, num_splits, ctypes.byref(out)),
           "paged_kv4_decode_workspace_bytes")
    return out.value


def paged_kv4_decode_attention(out, q, cache, block_table, context_lens, scale, k_unit=1.0, v_unit=1.0,
                               num_splits=0, workspace=None, stream=None, window=0, prepare=False):
    """paged_decode_attention over a 4-bit cache, uint8 [num_blocks, Hkv, 18 * D].

    q, out [B, Hq, D]: one new token per sequence; [B, q_len, Hq, D]: q_len of
    them, token i seeing the cache up to its own position (f16 or bf16; out may be
    pinned host memory).  window > 0: each row sees its `window` most recent positions.
    workspace: a uint8 CUDA tensor of paged_kv4_decode_workspace_bytes(...) bytes, allocated
    here (by torch) when None; returned for paged_decode_status.  prepare=True
    returns the call as a Prepared object, which holds the workspace."""
    dev, shape, dtype = _device_of(q, "q"), q.shape, q.dtype
    if len(shape) == 3:
        (B, Hq, D), q_len = shape, 1
    elif len(shape) == 4:
        B, q_len, Hq, D = shape
    else:
        raise ValueError(f"q must be [B, Hq, D] or [B, q_len, Hq, D], got {tuple(shape)}")
    if out.shape != shape or out.dtype is not dtype:
        raise ValueError(f"out must be {tuple(shape)} of {dtype}, got {tuple(out.shape)} of {out.dtype}")
    out_dev = out.get_device()
    if out_dev >= 0 and out_dev != dev:
        raise ValueError(f"out is on {out.device}, expected cuda:{dev}")
    ptr, num_blocks, Hkv, cD = _cache4(cache, dev)
    if cD != D:
        raise ValueError(f"the cache's head dim is {cD}, q's {D}")
    table, max_blocks = _table(block_table, B, dev)
    lens = _arg(context_lens, "context_lens", _torch().int32, (B,), dev)
    code = _code(q)
    if workspace is None:
        workspace = _workspace(paged_kv4_decode_workspace_bytes(B, Hq, Hkv, D, code, num_splits, q_len), q.device, stream)
    args = (_out(out), _arg(q, "q", dtype, shape, dev), code, ptr, table, max_blocks, lens, B, q_len, int(window), Hq, Hkv, D,
            num_blocks, float(scale), float(k_unit), float(v_unit), num_splits, _dev(workspace, "workspace"),
            workspace.nbytes, _stream(stream, dev))
    return _issue(_L.paged_kv4_decode_attention, args, "paged_kv4_decode_attention", prepare, workspace)


class RopeTable:
    """The frequencies of rotary positions, as the rope calls take them.

    Pair i of rot_dim elements turns by position * f_i radians,
    f_i = base ** (-2 i / rot_dim), changed by `scaling` for contexts longer than the
    original_positions the model was trained on:
      "none"    as it is;
      "linear"  f_i / factor (positions interpolated);
      "base"    the base raised by factor ** (rot_dim / (rot_dim - 2)), so that the slowest
                pair is interpolated by the factor and the fastest stays;
      "parts"   by the turns r_i = original_positions * f_i / 2 pi that a pair makes over the
                original context: f_i where r_i >= fast, f_i / factor where r_i <= slow, and
                linear in r_i between.  (Models that go from one to the other linearly in the
                pair's index i: pass their f_i as `frequencies`.)
    frequencies: f_i themselves (float64 [rot_dim / 2]), instead of base and scaling.
    magnitude scales the rotated elements (0.1 ln(factor) + 1 goes with "parts" where the
    model was trained so; 1 leaves them).  interleaved: pairs are elements
    (2 i, 2 i + 1), not (i, i + rot_dim / 2).  `turns` is the device tensor of the table; it
    belongs to one device."""

    def __init__(self, rot_dim, base=10000.0, scaling="none", factor=1.0, original_positions=0, slow=1.0, fast=32.0,
                 magnitude=1.0, interleaved=False, frequencies=None, device=None):
        import numpy as np
        torch = _torch()
        if rot_dim <= 0 or rot_dim % 2:
            raise ValueError(f"rot_dim must be even and positive, got {rot_dim}")
        if frequencies is None:
            if scaling not in ("none", "linear", "base", "parts"):
                raise ValueError(f"unknown scaling {scaling!r}")
            if not (base > 0 and factor > 0):
                raise ValueError("base and factor must be positive")
            if scaling == "base":
                if rot_dim < 4:
                    raise ValueError("scaling by the base needs rot_dim >= 4")
                base = base * factor ** (rot_dim / (rot_dim - 2))
            f = float(base) ** (-np.arange(0, rot_dim, 2, dtype=np.float64) / rot_dim)
            if scaling == "linear":
                f = f / factor
            elif scaling == "parts":
                if not (original_positions > 0 and fast > slow):
                    raise ValueError("scaling by parts needs original_positions > 0 and fast > slow")
                keep = np.clip((original_positions * f / (2 * np.pi) - slow) / (fast - slow), 0.0, 1.0)
                f = f * keep + f / factor * (1 - keep)
        else:
            f = np.ascontiguousarray(np.asarray(frequencies, dtype=np.float64))
            if f.shape != (rot_dim // 2,):
                raise ValueError(f"frequencies must be {rot_dim // 2} numbers, got shape {f.shape}")
        f = np.ascontiguousarray(f)
        host = np.empty(rot_dim // 2, dtype=np.uint64)
        _check(_L.pkv_rope_turns(host.ctypes.data, f.ctypes.data, rot_dim // 2), "pkv_rope_turns")
        self.rot_dim, self.magnitude, self.interleaved, self.frequencies = rot_dim, float(magnitude), bool(interleaved), f
        self.turns = torch.from_numpy(host.view(np.int64)).to("cuda" if device is None else device)
        self._device = self.turns.get_device()
        self._args = (self.turns.data_ptr(), rot_dim, 1 if self.interleaved else 0, self.magnitude)


def _rope_args(table, positions, T, device):
    """positions .. magnitude of a rope call."""
    if table._device != device:
        raise ValueError(f"the table is on {table.turns.device}, expected cuda:{device}")
    return (_arg(positions, "positions", _torch().int64, (T,), device), *table._args)


def paged_rope(q, k, positions, table, q_out=None, k_out=None, stream=None, prepare=False):
    """Rotates q [T, Hq, D] and k [T, Hkv, D] (either may be None) by their
    positions [T] (int64) and the RopeTable, into q_out / k_out (None: in place).  A token's
    row may be a slice of a wider one (one projection's columns)."""
    first = q if q is not None else k
    if first is None:
        raise ValueError("paged_rope needs q or k")
    dev, dtype = _device_of(first, "q" if q is not None else "k"), first.dtype
    T, _, D = first.shape
    side = []
    for x, out, name in ((q, q_out, "q"), (k, k_out, "k")):
        if x is None:
            if out is not None:
                raise ValueError(f"{name}_out without {name}")
            side.append((None, 0, None, 0, 0))
            continue
        heads = x.shape[1]
        p, ld = _token_rows(x, name, (T, heads, D), dtype, dev)
        po, ldo = (p, ld) if out is None else _token_rows(out, name + "_out", (T, heads, D), dtype, dev)
        side.append((po, ldo, p, ld, heads))
    args = (*side[0][:4], *side[1][:4], _code(first), *_rope_args(table, positions, T, dev), T, side[0][4], side[1][4], D,
            _stream(stream, dev))
    return _issue(_L.paged_rope, args, "paged_rope", prepare)


def _rope_rows(q, k_new, v_new, q_out, Hkv, D, dev):
    """q_out .. dtype of a rope append, T and Hq."""
    dtype = q.dtype
    T, Hq, _ = q.shape
    rows, kv = (T, Hq, D), (T, Hkv, D)
    p, ld = _token_rows(q, "q", rows, dtype, dev)
    po, ldo = (p, ld) if q_out is None else _token_rows(q_out, "q_out", rows, dtype, dev)
    k, ld_k = _token_rows(k_new, "k_new", kv, dtype, dev)
    v, ld_v = _token_rows(v_new, "v_new", kv, dtype, dev)
    return (po, ldo, p, ld, k, ld_k, v, ld_v, _code(q)), T, Hq


def paged_rope_append(q, k_new, v_new, positions, table, k_cache, v_cache, slot_mapping, q_out=None, stream=None,
                      prepare=False):
    """Rotates q [T, Hq, D] (into q_out; None: in place) and k_new [T, Hkv, D]
    by their positions [T] (int64), and writes the rotated keys and v_new into the caches
    [num_blocks, Hkv, 16, D] of the same type at slot_mapping [T] (int64; < 0 skips)."""
    dev = _device_of(q, "q")
    shape = k_cache.shape
    if len(shape) != 4 or shape[2] != 16:
        raise ValueError(f"k_cache must be [num_blocks, Hkv, 16, D], got {tuple(shape)}")
    num_blocks, Hkv, _, D = shape
    k, v = _arg(k_cache, "k_cache", q.dtype, shape, dev), _arg(v_cache, "v_cache", q.dtype, shape, dev)
    rows, T, Hq = _rope_rows(q, k_new, v_new, q_out, Hkv, D, dev)
    args = (*rows, *_rope_args(table, positions, T, dev), k, v,
            _arg(slot_mapping, "slot_mapping", _torch().int64, (T,), dev), T, Hq, Hkv, D, num_blocks, _stream(stream, dev))
    return _issue(_L.paged_rope_append, args, "paged_rope_append", prepare)


def paged_kv4_rope_append(q, k_new, v_new, positions, table, cache, slot_mapping, k_unit=1.0, v_unit=1.0, q_out=None,
                          stream=None, prepare=False):
    """paged_rope_append into a 4-bit cache, uint8 [num_blocks, Hkv, 18 * D]."""
    dev = _device_of(q, "q")
    ptr, num_blocks, Hkv, D = _cache4(cache, dev)
    rows, T, Hq = _rope_rows(q, k_new, v_new, q_out, Hkv, D, dev)
    args = (*rows, *_rope_args(table, positions, T, dev), ptr,
            _arg(slot_mapping, "slot_mapping", _torch().int64, (T,), dev), T, Hq, Hkv, D, num_blocks, float(k_unit),
            float(v_unit), _stream(stream, dev))
    return _issue(_L.paged_kv4_rope_append, args, "paged_kv4_rope_append", prepare)


class BlockManager:
    """Host physical-block allocator (native, in libpagedkv.so): allocate /
    adopt / fork / free and per-token slot mapping with copy-on-write."""

    def __init__(self, num_blocks):
        self._destroy = _L.pkv_bm_destroy   # (of the library that makes the handle, whatever _L is in the end)
        self._h = _L.pkv_bm_create(num_blocks)
        if not self._h:
            raise MemoryError("pkv_bm_create failed")
        self.num_blocks = num_blocks

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            self._destroy(h)
            self._h = None

    def allocate(self, seq, num_tokens):
        rc = _L.pkv_bm_allocate(self._h, seq, num_tokens)
        if rc == PKV_EOOM:
            return False
        _check(rc, "allocate")
        return True

    def adopt(self, seq, blocks, num_tokens):
        arr = (ctypes.c_int32 * len(blocks))(*blocks)
        _check(_L.pkv_bm_adopt(self._h, seq, arr, len(blocks), num_tokens), "adopt")

    def fork(self, parent, child):
        rc = _L.pkv_bm_fork(self._h, parent, child)
        if rc == PKV_ENOTFOUND:
            return False
        _check(rc, "fork")
        return True

    def free(self, seq):
        _check(_L.pkv_bm_free(self._h, seq), "free")

    def release_outside_window(self, seq, window):
        """Releases the blocks of seq that no later token sees with this
        sliding window; returns how many table entries were released."""
        n = _i64(0)
        _check(_L.pkv_bm_release_window(self._h, seq, window, ctypes.byref(n)),
               "release_outside_window")
        return n.value

    def truncate(self, seq, num_tokens):
        """Shortens seq to its first num_tokens tokens (rejected drafts)."""
        _check(_L.pkv_bm_truncate(self._h, seq, num_tokens), "truncate")

    def append_slots(self, seqs):
        """One new token per sequence: (slots list, [(src, dst), ...]) or None on OOM."""
        n = len(seqs)
        s = (ctypes.c_int64 * max(n, 1))(*seqs)
        slots = (ctypes.c_int64 * max(n, 1))()
        pairs = (ctypes.c_int32 * max(2 * n, 2))()
        ncow = _i32(0)
        rc = _L.pkv_bm_append_slots(self._h, s, n, slots, pairs, ctypes.byref(ncow))
        if rc == PKV_EOOM:
            return None
        _check(rc, "append_slots")
        return list(slots[:n]), [(pairs[2 * i], pairs[2 * i + 1]) for i in range(ncow.value)]

    def append_slots_into(self, seqs_arr, slots_arr, pairs_arr):
        """Buffer form for hot loops: numpy int64 seqs / int64 slots / int32
        [2n] pairs (host, contiguous); returns the number of copy pairs or -1 on OOM."""
        ncow = _i32(0)
        rc = _L.pkv_bm_append_slots(self._h, seqs_arr.ctypes.data, len(seqs_arr),
                                    slots_arr.ctypes.data, pairs_arr.ctypes.data, ctypes.byref(ncow))
        if rc == PKV_EOOM:
            return -1
        _check(rc, "append_slots")
        return ncow.value

    def export(self, seqs, max_blocks):
        """(table int32 [n, max_blocks] with -1 padding, context_lens int32 [n]) as numpy."""
        import numpy as np
        n = len(seqs)
        s = np.ascontiguousarray(np.asarray(seqs, dtype=np.int64))
        table = np.empty((n, max_blocks), dtype=np.int32)
        lens = np.empty((n,), dtype=np.int32)
        _check(_L.pkv_bm_export(self._h, s.ctypes.data, n, table.ctypes.data, max_blocks,
                                lens.ctypes.data), "export")
        return table, lens

    def num_free(self):
        return _L.pkv_bm_num_free(self._h)

    def refcount(self, block):
        return _L.pkv_bm_refcount(self._h, block)

    def num_tokens(self, seq):
        return _L.pkv_bm_num_tokens(self._h, seq)
