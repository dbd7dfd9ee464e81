"""ctypes binding of include/kda_paged.h: rotary positions, the paged KV cache of a hybrid
stack's full-attention layers, attention over it and the pages' bookkeeping. Argument
marshalling only, as in _binding.py: every step runs in the library's HIP kernels.
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from ._binding import KDA_DTYPE_BF16, KDA_DTYPE_F32, KdaError, _lib

ROPE_INTERLEAVED = 1
ROPE_INVERSE = 2
MAX_POOLS = 8


class _Pool(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("outer_stride", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("page_bytes", ctypes.c_int64),
                ("outer", ctypes.c_int32), ("num_pages", ctypes.c_int32)]


_READY = None


def _api():
    global _READY
    if _READY is None:
        lib = _lib()
        vp, i32, i64, sz, f32 = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t,
                                 ctypes.c_float)
        u32, pool = ctypes.c_uint32, ctypes.POINTER(_Pool)
        st = ctypes.c_int
        for name, res, args in (
                ("kda_rope", st, [vp, vp, vp, vp, i64, i32, i32, i32, i32, i64, i64, st, u32, f32,
                                  vp, vp, vp]),
                ("kda_cache_append", st, [vp, vp, vp, i64, i64, i64, vp, vp, i64, i64, vp, i64, vp, vp,
                                          i32, i64, i32, i32, i32, i32, i32, i32, st, vp, i32, u32,
                                          f32, vp, vp]),
                ("kda_attn_paged_workspace_size", sz, [i32, i64, i32, i32, i32, st]),
                ("kda_attn_paged", st, [vp, i64, vp, vp, i64, i64, vp, i64, vp, vp, i32, i64, i32, i32,
                                        i32, i32, i32, i32, st, f32, i32, vp, vp, vp, sz, vp]),
                ("kda_pages_plan_workspace_size", sz, [i32, i32, i32]),
                ("kda_pages_alloc", st, [vp, vp, i64, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp, sz,
                                         vp]),
                ("kda_pages_fork", st, [pool, i32, vp, vp, i64, vp, vp, vp, i32, i32, i32, i32, i32, vp,
                                        vp, sz, vp]),
                ("kda_pages_free", st, [vp, vp, i64, vp, vp, i32, i32, i32, i32, i32, vp]),
                ("kda_pages_compact_workspace_size", sz, [i32]),
                ("kda_pages_compact", st, [pool, i32, vp, vp, i64, i32, i32, i32, vp, vp, i64, vp, vp,
                                           sz, vp]),
                ("kda_pages_copy", st, [pool, i32, vp, vp, i32, vp])):
            f = getattr(lib, name)
            f.restype, f.argtypes = res, args
        _READY = lib
    return _READY


# ------------------------------------------------------------------ arguments
# A decode step's calls take a few microseconds on the GPU, so what is checked here is checked
# with few and cheap queries of each tensor.
def _code(t, name):
    if t.dtype is torch.bfloat16:
        return KDA_DTYPE_BF16
    if t.dtype is torch.float32:
        return KDA_DTYPE_F32
    raise TypeError("%s must be bfloat16 or float32, got %s" % (name, t.dtype))


def _same(t, name, dtype, index):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.get_device() != index:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, _device(index)))
    if t.dtype is not dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))


def _device(index):
    return torch.device("cuda", index) if index >= 0 else torch.device("cpu")


def _array(t, name, dtype, index, shape):
    _same(t, name, dtype, index)
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), shape))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _rows(t, name, dtype, index, rows, heads, dim):
    """Rows of contiguous heads [rows, heads, dim], any row stride; returns that stride."""
    _same(t, name, dtype, index)
    if t.shape != (rows, heads, dim):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), (rows, heads, dim)))
    s = t.stride()
    if ((s[2] != 1 and dim > 1) or (s[1] != dim and heads > 1)) and t.numel():
        raise ValueError("%s must have contiguous heads (only its rows may be strided)" % name)
    return s[0] if rows > 1 else heads * dim


def _pages(t, name, dtype, index):
    """Pages [P, heads, page_size, dim], contiguous each; returns the page stride."""
    _same(t, name, dtype, index)
    if t.dim() != 4:
        raise ValueError("%s must be [pages, heads, page_size, dim], got shape %s"
                         % (name, tuple(t.shape)))
    P, H, ps, D = t.shape
    s = t.stride()
    if (s[3] != 1 and D > 1) or s[2] != D or (s[1] != ps * D and H > 1):
        raise ValueError("%s must have contiguous pages (only the pages may be strided)" % name)
    return s[0] if P > 1 else H * ps * D


def _table(t, index):
    _same(t, "block_table", torch.int32, index)
    if t.dim() != 2:
        raise ValueError("block_table must be [sequences, pages]")
    n, m = t.shape
    s = t.stride()
    if s[1] != 1 and m > 1:
        raise ValueError("block_table must have contiguous rows")
    return n, m, (s[0] if n > 1 else m)


def _cache(k_cache, v_cache, dtype, index):
    ks, vs = _pages(k_cache, "k_cache", dtype, index), _pages(v_cache, "v_cache", dtype, index)
    if v_cache.shape != k_cache.shape:
        raise ValueError("v_cache has shape %s, expected %s" % (tuple(v_cache.shape),
                                                               tuple(k_cache.shape)))
    return ks, vs


def _batch(block_table, seq_lens, cu_seqlens, index):
    N, M, stride = _table(block_table, index)
    _array(seq_lens, "seq_lens", torch.int32, index, (N,))
    if cu_seqlens is not None:
        _array(cu_seqlens, "cu_seqlens", torch.int32, index, (N + 1,))
    return N, M, stride


def _p(t):
    return None if t is None else t.data_ptr()


def _call(name, index, *args):
    """The entry point ``name``, with the current stream of the tensors' device as its last argument and
    that device current."""
    if index < 0:
        raise ValueError("%s runs on a GPU, its tensors are on the CPU" % name)
    f = getattr(_READY or _api(), name)
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            st = f(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        st = f(*args, torch._C._cuda_getCurrentRawStream(index))
    if st != 0:
        raise KdaError(st, name)


def _workspace(given, need, like, what):
    if need == 0:
        raise KdaError(1, what)
    if given is None:
        return like.new_empty(need, dtype=torch.uint8), need
    if given.get_device() != like.get_device() or not given.is_contiguous():
        raise ValueError("workspace must be a contiguous buffer on %s" % like.device)
    return given, given.numel() * given.element_size()


# workspace sizes, functions of the arguments alone
@functools.lru_cache(maxsize=256)
def _attn_bytes(N, T, Hq, Hk, D, code):
    return int(_api().kda_attn_paged_workspace_size(N, T, Hq, Hk, D, code))


@functools.lru_cache(maxsize=256)
def _plan_bytes(count, N, P):
    return int(_api().kda_pages_plan_workspace_size(count, N, P))


# ------------------------------------------------------------------ rotary positions
def rope_freqs(rot_dim, base=10000.0, scaling=None, factor=1.0, original_length=8192,
               fast_turns=32.0, slow_turns=1.0, device=None):
    """(inv_freq, scale) for rope and cache_append: radians per position of each of the
    rot_dim / 2 pairs, fp64 [rot_dim / 2] on ``device``, and the factor on the turned channels.

    scaling None: base^(-2 i / rot_dim). For a context ``factor`` times the original one:
    'linear' divides every frequency by the factor (positions are interpolated); 'ntk' raises
    the base by factor^(rot_dim / (rot_dim - 2)), which does so for the slowest pair and keeps
    the fastest; 'yarn' divides those of pairs that make fewer than ``slow_turns`` turns over ``original_length``
    tokens, keeps those of pairs that make more than ``fast_turns``, ramps between (linearly in the pair's index),
    and returns scale 0.1 ln(factor) + 1.
    """
    if rot_dim < 2 or rot_dim % 2 != 0:
        raise ValueError("rot_dim must be even, got %d" % rot_dim)
    if not base > 1 or not factor >= 1:
        raise ValueError("base must exceed 1 and factor must be at least 1")
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    scale = 1.0
    if scaling == "ntk":
        if rot_dim < 4:
            raise ValueError("'ntk' needs a rot_dim of at least 4")
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = base ** (-2.0 * i / rot_dim)
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        def pair(turns):  # the pair that makes this many turns over the original context
            return rot_dim * math.log(original_length / (2 * math.pi * turns)) / (2 * math.log(base))
        low = max(0, math.floor(pair(fast_turns)))
        high = min(rot_dim - 1, math.ceil(pair(slow_turns)))
        slow = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        f = f * (1 - slow) + f / factor * slow
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError("scaling must be None, 'linear', 'ntk' or 'yarn', got %r" % (scaling,))
    return f.to(device), scale


def _inv_freq(inv_freq, index):
    _same(inv_freq, "inv_freq", torch.float64, index)
    if inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous vector")
    return 2 * inv_freq.shape[0]


def _rope(q, k, positions, inv_freq, flags, scale, q_out, k_out):
    x = q if q is not None else k
    if x is None:
        raise ValueError("q or k must be given")
    index, dtype, code = x.get_device(), x.dtype, _code(x, "q and k")
    if x.dim() != 3:
        raise ValueError("q and k must be [tokens, heads, dim], got shape %s" % (tuple(x.shape),))
    T, _, D = x.shape
    _array(positions, "positions", torch.int32, index, (T,))
    R = _inv_freq(inv_freq, index)
    Hq, qs, q_out = _turned(q, q_out, "q", dtype, index, T, D)
    Hk, ks, k_out = _turned(k, k_out, "k", dtype, index, T, D)
    if T:
        _call("kda_rope", index, _p(q), _p(k), positions.data_ptr(), inv_freq.data_ptr(), T, Hq, Hk, D, R,
              qs, ks, code, flags, scale, _p(q_out), _p(k_out))
    return q_out, k_out


def _turned(t, out, name, dtype, index, T, D):
    """(heads, row stride, output) of q or k: the output given (t itself, or apart), or a new one."""
    if t is None:
        if out is not None:
            raise ValueError("%s_out is given without %s" % (name, name))
        return 0, 0, None
    H = t.shape[1] if t.dim() == 3 else -1
    stride = _rows(t, name, dtype, index, T, H, D)
    if out is None:
        out = t.new_empty((T, H, D))
    elif out.data_ptr() == t.data_ptr():
        if _rows(out, name + "_out", dtype, index, T, H, D) != stride:
            raise ValueError("%s_out in place of %s must have its strides" % (name, name))
    else:
        _array(out, name + "_out", dtype, index, (T, H, D))
    return H, stride, out


def rope(q, k, positions, inv_freq, interleaved=False, scale=1.0, q_out=None, k_out=None):
    """kda_rope: q [T, Hq, D] and k [T, Hk, D] (either may be None; rows may be strided) turned
    by positions [T] int32 at inv_freq (fp64 [R / 2], see rope_freqs; channels from R on are
    copied). q_out / k_out may be q / k themselves (in place). Returns (q_out, k_out)."""
    return _rope(q, k, positions, inv_freq, ROPE_INTERLEAVED if interleaved else 0, scale, q_out,
                 k_out)


def rope_bwd(d_q, d_k, positions, inv_freq, interleaved=False, scale=1.0, q_out=None, k_out=None):
    """The gradients of rope with respect to its q and k, from those of its outputs (bf16 or
    fp32, whatever rope's inputs were)."""
    return _rope(d_q, d_k, positions, inv_freq,
                 ROPE_INVERSE | (ROPE_INTERLEAVED if interleaved else 0), scale, q_out, k_out)


# ------------------------------------------------------------------ the cache
def cache_append(k, v, k_cache, v_cache, block_table, seq_lens, cu_seqlens=None, q=None,
                 inv_freq=None, interleaved=False, scale=1.0, q_out=None):
    """kda_cache_append: the new tokens' k and v [T, Hk, D] (the last tokens of sequences whose
    lengths seq_lens [N] count them; rows by cu_seqlens [N + 1], or T / N each) go to the pages
    of k_cache, v_cache [P, Hk, page_size, D] that block_table [N, max_pages] names. With
    inv_freq, k is turned by its position on the way, and q [T, Hq, D] too: returns q_out (else
    None)."""
    index, dtype, code = k.get_device(), k.dtype, _code(k, "k")
    if k.dim() != 3:
        raise ValueError("k must be [tokens, heads, dim], got shape %s" % (tuple(k.shape),))
    T, Hk, D = k.shape
    N, M, ts = _batch(block_table, seq_lens, cu_seqlens, index)
    kps, vps = _cache(k_cache, v_cache, dtype, index)
    P, heads, ps, dim = k_cache.shape
    if heads != Hk or dim != D:
        raise ValueError("k_cache has shape %s, expected [pages, %d, page_size, %d]"
                         % (tuple(k_cache.shape), Hk, D))
    ks, vs = _rows(k, "k", dtype, index, T, Hk, D), _rows(v, "v", dtype, index, T, Hk, D)
    R = _inv_freq(inv_freq, index) if inv_freq is not None else 0
    if q is not None and inv_freq is None:
        raise ValueError("q is turned by inv_freq, which is not given")
    Hq, qs, q_out = _turned(q, q_out, "q", dtype, index, T, D)
    if T:
        _call("kda_cache_append", index, _p(q), k.data_ptr(), v.data_ptr(), qs, ks, vs, k_cache.data_ptr(),
              v_cache.data_ptr(), kps, vps, block_table.data_ptr(), ts, seq_lens.data_ptr(), _p(cu_seqlens),
              N, T, Hq, Hk, D, P, M, ps, code, _p(inv_freq), R, ROPE_INTERLEAVED if interleaved else 0,
              scale, _p(q_out))
    return q_out


def attn_workspace_size(num_seqs, total_tokens, num_q_heads, num_kv_heads, head_dim, dtype) -> int:
    """Workspace bytes of attn_paged for this shape."""
    code = KDA_DTYPE_BF16 if dtype == torch.bfloat16 else KDA_DTYPE_F32
    return _attn_bytes(num_seqs, total_tokens, num_q_heads, num_kv_heads, head_dim, code)


def attn_paged(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens=None, scale=None, window=0,
               o=None, lse=None, workspace=None):
    """kda_attn_paged: causal attention of the new tokens' queries q [T, Hq, D] over the pages
    of their sequences, which hold the new tokens' k and v already (layouts as in
    cache_append). ``scale`` defaults to D^-1/2; ``window`` > 0 keeps the last ``window`` keys
    of each row. ``lse`` (fp32 [T, Hq]) receives the log of each row's sum of e^score. Returns
    o [T, Hq, D]; a row with no key is 0, its lse -inf."""
    index, dtype, code = q.get_device(), q.dtype, _code(q, "q")
    if q.dim() != 3:
        raise ValueError("q must be [tokens, heads, dim], got shape %s" % (tuple(q.shape),))
    T, Hq, D = q.shape
    N, M, ts = _batch(block_table, seq_lens, cu_seqlens, index)
    kps, vps = _cache(k_cache, v_cache, dtype, index)
    P, Hk, ps, dim = k_cache.shape
    if dim != D:
        raise ValueError("k_cache has head dim %d, expected %d" % (dim, D))
    qs = _rows(q, "q", dtype, index, T, Hq, D)
    if o is None:
        o = q.new_empty((T, Hq, D))
    else:
        _array(o, "o", dtype, index, (T, Hq, D))
    if lse is not None:
        _array(lse, "lse", torch.float32, index, (T, Hq))
    if T == 0:
        return o
    need = _attn_bytes(N, T, Hq, Hk, D, code)
    if need == 0:
        raise KdaError(2 if D not in (64, 128, 256) else 1, "kda_attn_paged_workspace_size")
    workspace, size = _workspace(workspace, need, q, "kda_attn_paged")
    _call("kda_attn_paged", index, q.data_ptr(), qs, k_cache.data_ptr(), v_cache.data_ptr(), kps, vps,
          block_table.data_ptr(), ts, seq_lens.data_ptr(), _p(cu_seqlens), N, T, Hq, Hk, D, P, M, ps, code,
          D ** -0.5 if scale is None else scale, window, o.data_ptr(), _p(lse), workspace.data_ptr(), size)
    return o


# ------------------------------------------------------------------ pages
@functools.lru_cache(maxsize=256)
def _pool_layout(shape, strides, es, page_dim):
    """(outer_stride, page_stride, page_bytes, outer, num_pages) of a tensor whose dimension page_dim
    counts the pages: what follows it is one page, what precedes it the planes."""
    dims = len(shape)
    if not 0 <= page_dim < dims:
        raise ValueError("page_dim %d of a pool of %d dimensions" % (page_dim, dims))
    if 0 in shape:
        raise ValueError("a pool is empty")
    width = 1
    for j in range(dims - 1, page_dim, -1):
        if shape[j] != 1 and strides[j] != width:
            raise ValueError("a pool's pages must be contiguous")
        width *= shape[j]
    outer, step = 1, 0
    for j in range(page_dim - 1, -1, -1):
        if shape[j] == 1:
            continue
        if outer == 1:
            step = strides[j]
        elif strides[j] != outer * step:
            raise ValueError("the dimensions before a pool's pages must be evenly spaced")
        outer *= shape[j]
    P = shape[page_dim]
    return step * es, strides[page_dim] * es if P > 1 else 0, width * es, outer, P


def _pools(pools, page_dim, index):
    if pools is None:
        return None, 0
    if isinstance(pools, torch.Tensor):
        pools = (pools,)
    if len(pools) > MAX_POOLS:
        raise ValueError("at most %d pools in one call, got %d" % (MAX_POOLS, len(pools)))
    arr = (_Pool * len(pools))()
    for x, t in zip(arr, pools):
        if not isinstance(t, torch.Tensor) or t.get_device() != index:
            raise ValueError("a pool must be a torch.Tensor on %s" % _device(index))
        x.base = t.data_ptr()
        x.outer_stride, x.page_stride, x.page_bytes, x.outer, x.num_pages = _pool_layout(
            t.shape, t.stride(), t.element_size(), page_dim)
    return arr, len(pools)


def _count(t, name, index):
    """Entries of a vector of sequences, pages or token counts."""
    _same(t, name, torch.int32, index)
    if t.dim() != 1 or not t.is_contiguous():
        raise ValueError("%s must be a contiguous vector" % name)
    return t.shape[0]


def _state(page_refs, block_table, seq_lens):
    index = page_refs.get_device()
    P = _count(page_refs, "page_refs", index)
    N, M, ts = _table(block_table, index)
    if seq_lens is not None:
        _array(seq_lens, "seq_lens", torch.int32, index, (N,))
    return index, P, N, M, ts


def _plan(granted, count, workspace, N, P, index, like):
    if granted is None:
        granted = like.new_empty(count)
    else:
        _array(granted, "granted", torch.int32, index, (count,))
    workspace, size = _workspace(workspace, _plan_bytes(count, N, P), like, "kda_pages_plan_workspace_size")
    return granted, workspace, size


def pages_alloc(page_refs, block_table, seq_lens, new_tokens, page_size, seqs=None, granted=None,
                workspace=None):
    """kda_pages_alloc: room for new_tokens[i] more tokens in sequence seqs[i] (default:
    sequence i), from the lowest free pages, in order. page_refs [P], block_table [N,
    max_pages] and seq_lens [N], all int32, change in place. Returns granted [count] int32: 1,
    or 0 where nothing was done."""
    index, P, N, M, ts = _state(page_refs, block_table, seq_lens)
    count = _count(new_tokens, "new_tokens", index)
    if seqs is not None:
        _array(seqs, "seqs", torch.int32, index, (count,))
    elif count != N:
        raise ValueError("new_tokens has %d values for %d sequences" % (count, N))
    granted, workspace, size = _plan(granted, count, workspace, N, P, index, new_tokens)
    _call("kda_pages_alloc", index, page_refs.data_ptr(), block_table.data_ptr(), ts, seq_lens.data_ptr(),
          _p(seqs), new_tokens.data_ptr(), count, N, P, M, page_size, granted.data_ptr(),
          workspace.data_ptr(), size)
    return granted


def pages_fork(pools, page_refs, block_table, seq_lens, parents, children, page_size, page_dim=0,
               granted=None, workspace=None):
    """kda_pages_fork: sequence children[i] (empty) becomes a copy of parents[i]: full pages are
    shared, a page that is not full is copied to the lowest free one in every pool. ``pools``:
    a tensor whose dimension ``page_dim`` counts the pages, up to 8 of them, or None (the
    bookkeeping alone). Returns granted [count] int32."""
    index, P, N, M, ts = _state(page_refs, block_table, seq_lens)
    count = _count(children, "children", index)
    _array(parents, "parents", torch.int32, index, (count,))
    arr, n = _pools(pools, page_dim, index)
    granted, workspace, size = _plan(granted, count, workspace, N, P, index, children)
    _call("kda_pages_fork", index, arr, n, page_refs.data_ptr(), block_table.data_ptr(), ts,
          seq_lens.data_ptr(), parents.data_ptr(), children.data_ptr(), count, N, P, M, page_size,
          granted.data_ptr(), workspace.data_ptr(), size)
    return granted


def pages_free(page_refs, block_table, seq_lens, seqs, page_size):
    """kda_pages_free: the sequences seqs [count] int32 become empty; every page they hold loses
    one reference."""
    index, P, N, M, ts = _state(page_refs, block_table, seq_lens)
    count = _count(seqs, "seqs", index)
    _call("kda_pages_free", index, page_refs.data_ptr(), block_table.data_ptr(), ts, seq_lens.data_ptr(),
          seqs.data_ptr(), count, N, P, M, page_size)


def pages_compact(pools, page_refs, block_table, page_dim=0, out_refs=None, out_table=None,
                  moved=None, workspace=None):
    """kda_pages_compact: the highest live page moves to the lowest free page until the live
    pages are the lowest ones, in every pool (as in pages_fork) and, unless out_refs /
    out_table are given, in page_refs and block_table themselves. Returns moved, int32 [1]."""
    index, P, N, M, ts = _state(page_refs, block_table, None)
    arr, n = _pools(pools, page_dim, index)
    if out_refs is None:
        out_refs = page_refs
    else:
        _array(out_refs, "out_refs", torch.int32, index, (P,))
    No, Mo, ots = N, M, ts
    if out_table is None:
        out_table = block_table
    else:
        No, Mo, ots = _table(out_table, index)
    if (No, Mo) != (N, M):
        raise ValueError("out_table has shape %s, expected %s" % ((No, Mo), (N, M)))
    if moved is None:
        moved = page_refs.new_empty(1)
    else:
        _array(moved, "moved", torch.int32, index, (1,))
    workspace, size = _workspace(workspace, _api().kda_pages_compact_workspace_size(P), page_refs,
                                 "kda_pages_compact_workspace_size")
    _call("kda_pages_compact", index, arr, n, page_refs.data_ptr(), block_table.data_ptr(), ts, N, P, M,
          out_refs.data_ptr(), out_table.data_ptr(), ots, moved.data_ptr(), workspace.data_ptr(), size)
    return moved


def pages_copy(pools, src, dst, page_dim=0):
    """kda_pages_copy: page src[i] to page dst[i] of every pool (any per-slot data: pages of a
    cache, or the states of KDA layers). No page may be a dst twice, or both a src and a dst."""
    index = src.get_device()
    count = _count(src, "src", index)
    _array(dst, "dst", torch.int32, index, (count,))
    arr, n = _pools(pools, page_dim, index)
    _call("kda_pages_copy", index, arr, n, src.data_ptr(), dst.data_ptr(), count)
