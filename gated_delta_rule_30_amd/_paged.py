"""ctypes binding of include/kda_paged.h: rotary positions, the paged KV cache of a hybrid
stack's full-attention layers, attention over it and the pages' bookkeeping. Argument
marshalling only, as in _binding.py: every step runs in the library's HIP kernels.
"""
from __future__ import annotations

import ctypes
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
def _code(t, name):
    if t.dtype == torch.bfloat16:
        return KDA_DTYPE_BF16
    if t.dtype == torch.float32:
        return KDA_DTYPE_F32
    raise TypeError("%s must be bfloat16 or float32, got %s" % (name, t.dtype))


def _same(t, name, dtype, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if t.dtype != dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))


def _array(t, name, dtype, device, shape):
    _same(t, name, dtype, device)
    if tuple(t.shape) != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), shape))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _rows(t, name, dtype, device, rows, heads, dim):
    """Rows of contiguous heads [rows, heads, dim], any row stride; returns that stride."""
    _same(t, name, dtype, device)
    if tuple(t.shape) != (rows, heads, dim):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), (rows, heads, dim)))
    s = t.stride()
    if t.numel() and ((dim > 1 and s[2] != 1) or (heads > 1 and s[1] != dim)):
        raise ValueError("%s must have contiguous heads (only its rows may be strided)" % name)
    return s[0] if rows > 1 else heads * dim


def _pages(t, name, dtype, device):
    """Pages [P, heads, page_size, dim], contiguous each; returns the page stride."""
    _same(t, name, dtype, device)
    if t.dim() != 4:
        raise ValueError("%s must be [pages, heads, page_size, dim], got shape %s"
                         % (name, tuple(t.shape)))
    P, H, ps, D = t.shape
    s = t.stride()
    if (D > 1 and s[3] != 1) or s[2] != D or (H > 1 and s[1] != ps * D):
        raise ValueError("%s must have contiguous pages (only the pages may be strided)" % name)
    return s[0] if P > 1 else H * ps * D


def _table(t, device):
    _same(t, "block_table", torch.int32, device)
    if t.dim() != 2:
        raise ValueError("block_table must be [sequences, pages]")
    n, m = t.shape
    if m > 1 and t.stride(1) != 1:
        raise ValueError("block_table must have contiguous rows")
    return n, m, (t.stride(0) if n > 1 else m)


def _cache(k_cache, v_cache, dtype, device):
    ks, vs = _pages(k_cache, "k_cache", dtype, device), _pages(v_cache, "v_cache", dtype, device)
    if v_cache.shape != k_cache.shape:
        raise ValueError("v_cache has shape %s, expected %s" % (tuple(v_cache.shape),
                                                               tuple(k_cache.shape)))
    return ks, vs


def _batch(block_table, seq_lens, cu_seqlens, device):
    N, M, stride = _table(block_table, device)
    _array(seq_lens, "seq_lens", torch.int32, device, (N,))
    if cu_seqlens is not None:
        _array(cu_seqlens, "cu_seqlens", torch.int32, device, (N + 1,))
    return N, M, stride


def _p(t):
    return None if t is None else t.data_ptr()


class _on:
    """The device of the tensors made current for a call, and that device's current stream."""

    def __init__(self, device):
        if device.type != "cuda":
            raise ValueError("tensors are on %s: the operators run on a GPU" % device)
        self.index = device.index
        self.guard = None

    def __enter__(self):
        if self.index != torch.cuda.current_device():
            self.guard = torch.cuda.device(self.index)
            self.guard.__enter__()
        return torch.cuda.current_stream(self.index).cuda_stream

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _check(st, what):
    if st != 0:
        raise KdaError(st, what)


def _workspace(given, need, device, what):
    if need == 0:
        raise KdaError(1, what)
    if given is None:
        return torch.empty(need, dtype=torch.uint8, device=device), need
    if given.device != device or not given.is_contiguous():
        raise ValueError("workspace must be a contiguous buffer on %s" % device)
    return given, given.numel() * given.element_size()


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


def _inv_freq(inv_freq, device):
    _same(inv_freq, "inv_freq", torch.float64, device)
    if inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous vector")
    return 2 * inv_freq.shape[0]


def _rope(q, k, positions, inv_freq, flags, scale, q_out, k_out):
    x = q if q is not None else k
    if x is None:
        raise ValueError("q or k must be given")
    device, dtype, code = x.device, x.dtype, _code(x, "q and k")
    if x.dim() != 3:
        raise ValueError("q and k must be [tokens, heads, dim], got shape %s" % (tuple(x.shape),))
    T, D = x.shape[0], x.shape[2]
    _array(positions, "positions", torch.int32, device, (T,))
    R = _inv_freq(inv_freq, device)
    strides, heads, outs = [0, 0], [0, 0], [None, None]
    for j, (name, t, out) in enumerate((("q", q, q_out), ("k", k, k_out))):
        if t is None:
            if out is not None:
                raise ValueError("%s_out is given without %s" % (name, name))
            continue
        heads[j] = t.shape[1] if t.dim() == 3 else -1
        strides[j] = _rows(t, name, dtype, device, T, heads[j], D)
        if out is None:
            out = torch.empty((T, heads[j], D), dtype=dtype, device=device)
        elif out.data_ptr() == t.data_ptr():
            if _rows(out, name + "_out", dtype, device, T, heads[j], D) != strides[j]:
                raise ValueError("%s_out in place of %s must have its strides" % (name, name))
        else:
            _array(out, name + "_out", dtype, device, (T, heads[j], D))
        outs[j] = out
    if T == 0:
        return outs[0], outs[1]
    with _on(device) as stream:
        _check(_api().kda_rope(_p(q), _p(k), _p(positions), _p(inv_freq), T, heads[0], heads[1], D, R,
                               strides[0], strides[1], code, flags, scale, _p(outs[0]), _p(outs[1]),
                               stream), "kda_rope")
    return outs[0], outs[1]


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
    device, dtype, code = k.device, k.dtype, _code(k, "k")
    if k.dim() != 3:
        raise ValueError("k must be [tokens, heads, dim], got shape %s" % (tuple(k.shape),))
    T, Hk, D = k.shape
    N, M, ts = _batch(block_table, seq_lens, cu_seqlens, device)
    kps, vps = _cache(k_cache, v_cache, dtype, device)
    if k_cache.shape[1] != Hk or k_cache.shape[3] != D:
        raise ValueError("k_cache has shape %s, expected [pages, %d, page_size, %d]"
                         % (tuple(k_cache.shape), Hk, D))
    ks, vs = _rows(k, "k", dtype, device, T, Hk, D), _rows(v, "v", dtype, device, T, Hk, D)
    R = _inv_freq(inv_freq, device) if inv_freq is not None else 0
    Hq, qs = 0, 0
    if q is not None:
        if inv_freq is None:
            raise ValueError("q is turned by inv_freq, which is not given")
        Hq = q.shape[1] if q.dim() == 3 else -1
        qs = _rows(q, "q", dtype, device, T, Hq, D)
        if q_out is None:
            q_out = torch.empty((T, Hq, D), dtype=dtype, device=device)
        elif q_out.data_ptr() == q.data_ptr():
            if _rows(q_out, "q_out", dtype, device, T, Hq, D) != qs:
                raise ValueError("q_out in place of q must have its strides")
        else:
            _array(q_out, "q_out", dtype, device, (T, Hq, D))
    elif q_out is not None:
        raise ValueError("q_out is given without q")
    if T == 0:
        return q_out
    with _on(device) as stream:
        _check(_api().kda_cache_append(
            _p(q), _p(k), _p(v), qs, ks, vs, _p(k_cache), _p(v_cache), kps, vps, _p(block_table), ts,
            _p(seq_lens), _p(cu_seqlens), N, T, Hq, Hk, D, k_cache.shape[0], M, k_cache.shape[2],
            code, _p(inv_freq), R, ROPE_INTERLEAVED if interleaved else 0, scale, _p(q_out), stream),
            "kda_cache_append")
    return q_out


def attn_workspace_size(num_seqs, total_tokens, num_q_heads, num_kv_heads, head_dim, dtype) -> int:
    """Workspace bytes of attn_paged for this shape."""
    code = KDA_DTYPE_BF16 if dtype == torch.bfloat16 else KDA_DTYPE_F32
    return int(_api().kda_attn_paged_workspace_size(num_seqs, total_tokens, num_q_heads,
                                                    num_kv_heads, head_dim, code))


def attn_paged(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens=None, scale=None, window=0,
               o=None, lse=None, workspace=None):
    """kda_attn_paged: causal attention of the new tokens' queries q [T, Hq, D] over the pages
    of their sequences, which hold the new tokens' k and v already (layouts as in
    cache_append). ``scale`` defaults to D^-1/2; ``window`` > 0 keeps the last ``window`` keys
    of each row. ``lse`` (fp32 [T, Hq]) receives the log of each row's sum of e^score. Returns
    o [T, Hq, D]; a row with no key is 0, its lse -inf."""
    device, dtype, code = q.device, q.dtype, _code(q, "q")
    if q.dim() != 3:
        raise ValueError("q must be [tokens, heads, dim], got shape %s" % (tuple(q.shape),))
    T, Hq, D = q.shape
    N, M, ts = _batch(block_table, seq_lens, cu_seqlens, device)
    kps, vps = _cache(k_cache, v_cache, dtype, device)
    P, Hk, ps, _ = k_cache.shape
    if k_cache.shape[3] != D:
        raise ValueError("k_cache has head dim %d, expected %d" % (k_cache.shape[3], D))
    qs = _rows(q, "q", dtype, device, T, Hq, D)
    if o is None:
        o = torch.empty((T, Hq, D), dtype=dtype, device=device)
    else:
        _array(o, "o", dtype, device, (T, Hq, D))
    if lse is not None:
        _array(lse, "lse", torch.float32, device, (T, Hq))
    if T == 0:
        return o
    lib = _api()
    need = lib.kda_attn_paged_workspace_size(N, T, Hq, Hk, D, code)
    if need == 0:
        raise KdaError(2 if D not in (64, 128, 256) else 1, "kda_attn_paged_workspace_size")
    with _on(device) as stream:
        workspace, size = _workspace(workspace, need, device, "kda_attn_paged")
        _check(lib.kda_attn_paged(
            _p(q), qs, _p(k_cache), _p(v_cache), kps, vps, _p(block_table), ts, _p(seq_lens),
            _p(cu_seqlens), N, T, Hq, Hk, D, P, M, ps, code, D ** -0.5 if scale is None else scale,
            window, _p(o), _p(lse), _p(workspace), size, stream), "kda_attn_paged")
    return o


# ------------------------------------------------------------------ pages
def _pool(t, page_dim, device):
    """A kda_page_pool of a tensor whose dimension page_dim counts the pages: what follows it is
    one page, what precedes it the planes."""
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError("a pool must be a torch.Tensor on %s" % device)
    if not 0 <= page_dim < t.dim():
        raise ValueError("page_dim %d of a pool of %d dimensions" % (page_dim, t.dim()))
    shape, strides, es = t.shape, t.stride(), t.element_size()
    width = 1
    for j in range(t.dim() - 1, page_dim, -1):
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
    if t.numel() == 0:
        raise ValueError("a pool is empty")
    return _Pool(t.data_ptr(), step * es, strides[page_dim] * es if P > 1 else 0, width * es, outer, P)


def _pools(pools, page_dim, device):
    if pools is None:
        return None, 0
    if isinstance(pools, torch.Tensor):
        pools = (pools,)
    if len(pools) > MAX_POOLS:
        raise ValueError("at most %d pools in one call, got %d" % (MAX_POOLS, len(pools)))
    return (_Pool * len(pools))(*(_pool(t, page_dim, device) for t in pools)), len(pools)


def _state(page_refs, block_table, seq_lens):
    device = page_refs.device
    if page_refs.dim() != 1:
        raise ValueError("page_refs must be a vector")
    _array(page_refs, "page_refs", torch.int32, device, (page_refs.shape[0],))
    N, M, ts = _table(block_table, device)
    if seq_lens is not None:
        _array(seq_lens, "seq_lens", torch.int32, device, (N,))
    return device, page_refs.shape[0], N, M, ts


def _plan(granted, count, workspace, N, P, device):
    if granted is None:
        granted = torch.empty(count, dtype=torch.int32, device=device)
    else:
        _array(granted, "granted", torch.int32, device, (count,))
    workspace, size = _workspace(workspace, _api().kda_pages_plan_workspace_size(count, N, P), device,
                                 "kda_pages_plan_workspace_size")
    return granted, workspace, size


def pages_alloc(page_refs, block_table, seq_lens, new_tokens, page_size, seqs=None, granted=None,
                workspace=None):
    """kda_pages_alloc: room for new_tokens[i] more tokens in sequence seqs[i] (default:
    sequence i), from the lowest free pages, in order. page_refs [P], block_table [N,
    max_pages] and seq_lens [N], all int32, change in place. Returns granted [count] int32: 1,
    or 0 where nothing was done."""
    device, P, N, M, ts = _state(page_refs, block_table, seq_lens)
    count = new_tokens.shape[0] if new_tokens.dim() == 1 else -1
    _array(new_tokens, "new_tokens", torch.int32, device, (count,))
    if seqs is not None:
        _array(seqs, "seqs", torch.int32, device, (count,))
    elif count != N:
        raise ValueError("new_tokens has %d values for %d sequences" % (count, N))
    with _on(device) as stream:
        granted, workspace, size = _plan(granted, count, workspace, N, P, device)
        _check(_api().kda_pages_alloc(_p(page_refs), _p(block_table), ts, _p(seq_lens), _p(seqs),
                                      _p(new_tokens), count, N, P, M, page_size, _p(granted),
                                      _p(workspace), size, stream), "kda_pages_alloc")
    return granted


def pages_fork(pools, page_refs, block_table, seq_lens, parents, children, page_size, page_dim=0,
               granted=None, workspace=None):
    """kda_pages_fork: sequence children[i] (empty) becomes a copy of parents[i]: full pages are
    shared, a page that is not full is copied to the lowest free one in every pool. ``pools``:
    a tensor whose dimension ``page_dim`` counts the pages, up to 8 of them, or None (the
    bookkeeping alone). Returns granted [count] int32."""
    device, P, N, M, ts = _state(page_refs, block_table, seq_lens)
    count = children.shape[0] if children.dim() == 1 else -1
    _array(children, "children", torch.int32, device, (count,))
    _array(parents, "parents", torch.int32, device, (count,))
    arr, n = _pools(pools, page_dim, device)
    with _on(device) as stream:
        granted, workspace, size = _plan(granted, count, workspace, N, P, device)
        _check(_api().kda_pages_fork(arr, n, _p(page_refs), _p(block_table), ts, _p(seq_lens),
                                     _p(parents), _p(children), count, N, P, M, page_size,
                                     _p(granted), _p(workspace), size, stream), "kda_pages_fork")
    return granted


def pages_free(page_refs, block_table, seq_lens, seqs, page_size):
    """kda_pages_free: the sequences seqs [count] int32 become empty; every page they hold loses
    one reference."""
    device, P, N, M, ts = _state(page_refs, block_table, seq_lens)
    count = seqs.shape[0] if seqs.dim() == 1 else -1
    _array(seqs, "seqs", torch.int32, device, (count,))
    with _on(device) as stream:
        _check(_api().kda_pages_free(_p(page_refs), _p(block_table), ts, _p(seq_lens), _p(seqs), count,
                                     N, P, M, page_size, stream), "kda_pages_free")


def pages_compact(pools, page_refs, block_table, page_dim=0, out_refs=None, out_table=None,
                  moved=None, workspace=None):
    """kda_pages_compact: the highest live page moves to the lowest free page until the live
    pages are the lowest ones, in every pool (as in pages_fork) and, unless out_refs /
    out_table are given, in page_refs and block_table themselves. Returns moved, int32 [1]."""
    device, P, N, M, ts = _state(page_refs, block_table, None)
    arr, n = _pools(pools, page_dim, device)
    if out_refs is None:
        out_refs = page_refs
    else:
        _array(out_refs, "out_refs", torch.int32, device, (P,))
    if out_table is None:
        out_table = block_table
    No, Mo, ots = _table(out_table, device)
    if (No, Mo) != (N, M):
        raise ValueError("out_table has shape %s, expected %s" % ((No, Mo), (N, M)))
    if moved is None:
        moved = torch.empty(1, dtype=torch.int32, device=device)
    else:
        _array(moved, "moved", torch.int32, device, (1,))
    with _on(device) as stream:
        workspace, size = _workspace(workspace, _api().kda_pages_compact_workspace_size(P), device,
                                     "kda_pages_compact_workspace_size")
        _check(_api().kda_pages_compact(arr, n, _p(page_refs), _p(block_table), ts, N, P, M,
                                        _p(out_refs), _p(out_table), ots, _p(moved), _p(workspace),
                                        size, stream), "kda_pages_compact")
    return moved


def pages_copy(pools, src, dst, page_dim=0):
    """kda_pages_copy: page src[i] to page dst[i] of every pool (any per-slot data: pages of a
    cache, or the states of KDA layers). No page may be a dst twice, or both a src and a dst."""
    device = src.device
    count = src.shape[0] if src.dim() == 1 else -1
    _array(src, "src", torch.int32, device, (count,))
    _array(dst, "dst", torch.int32, device, (count,))
    arr, n = _pools(pools, page_dim, device)
    with _on(device) as stream:
        _check(_api().kda_pages_copy(arr, n, _p(src), _p(dst), count, stream), "kda_pages_copy")
