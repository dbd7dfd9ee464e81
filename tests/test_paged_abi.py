"""include/kda_paged.h without a GPU: symbols, the header, workspace sizes and every synchronous
refusal (each returns before anything is enqueued, so no device is touched)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import gated_delta_rule_30_amd as kda
from gated_delta_rule_30_amd import _paged

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "kda_paged.h")
SUCCESS, INVALID, NOT_SUPPORTED, WS_SMALL = 0, 1, 2, 3
F32, BF16 = 0, 1
A = 1 << 20  # fake device addresses: never read, every call below is refused first
BIG = 1 << 40


def test_every_declared_symbol_is_exported():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(kda_[a-z_]+)\s*\(", src))
    assert names == {"kda_rope", "kda_cache_append", "kda_attn_paged_workspace_size", "kda_attn_paged",
                     "kda_pages_plan_workspace_size", "kda_pages_alloc", "kda_pages_fork", "kda_pages_free",
                     "kda_pages_compact_workspace_size", "kda_pages_compact", "kda_pages_copy"}
    out = subprocess.run(["nm", "-D", "--defined-only", kda.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    exported = {l.split()[-1] for l in out.splitlines() if " T " in l}
    assert names <= exported


@pytest.mark.parametrize("cc,std,ext", [("gcc", "c99", "c"), ("g++", "c++11", "cpp")])
def test_header_compiles_standalone(cc, std, ext, tmp_path):
    src = tmp_path / ("t." + ext)
    src.write_text('#include "kda_paged.h"\nint main(void){ kda_page_pool p; p.outer = KDA_MAX_POOLS; '
                   'return (int)kda_pages_compact_workspace_size(p.outer) < 0; }\n')
    subprocess.run([cc, "-std=" + std, "-Wall", "-Werror", "-fsyntax-only", "-I", os.path.dirname(HEADER),
                    str(src)], check=True)


def _rope(**kw):
    a = dict(q=A, k=2 * A, pos=3 * A, f=4 * A, T=8, Hq=4, Hk=2, D=64, R=64, qs=256, ks=128, dtype=BF16,
             flags=0, scale=1.0, qo=5 * A, ko=6 * A)
    a.update(kw)
    return _paged._api().kda_rope(a["q"], a["k"], a["pos"], a["f"], a["T"], a["Hq"], a["Hk"], a["D"], a["R"],
                                  a["qs"], a["ks"], a["dtype"], a["flags"], a["scale"], a["qo"], a["ko"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(T=-1), INVALID),
    (dict(T=1 << 31), INVALID),
    (dict(D=40), NOT_SUPPORTED),
    (dict(D=528, qs=4 * 528, ks=2 * 528), NOT_SUPPORTED),
    (dict(R=0), NOT_SUPPORTED),
    (dict(R=24), NOT_SUPPORTED),
    (dict(R=80), NOT_SUPPORTED),
    (dict(dtype=2), NOT_SUPPORTED),
    (dict(flags=4), NOT_SUPPORTED),
    (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID),
    (dict(q=None, qo=None, k=None, ko=None), INVALID),
    (dict(qo=None), INVALID),
    (dict(k=None), INVALID),
    (dict(pos=None), INVALID),
    (dict(f=4 * A + 4), INVALID),
    (dict(pos=3 * A + 2), INVALID),
    (dict(q=A + 8), INVALID),
    (dict(ko=6 * A + 8), INVALID),
    (dict(qs=255), INVALID),
    (dict(qs=252), INVALID),              # rows would overlap
    (dict(qs=260), INVALID),              # not a multiple of 16 bytes
    (dict(Hq=0), INVALID),
    (dict(Hk=-1), INVALID),
    (dict(qo=A + 64), INVALID),           # partly over q
    (dict(qo=2 * A), INVALID),            # over k
    (dict(ko=5 * A), INVALID),            # over q_out
    (dict(q=2 * A, qo=2 * A, ko=2 * A), INVALID),
])
def test_rope_refusals(kw, expect):
    assert _rope(**kw) == expect


def _append(**kw):
    a = dict(q=A, k=2 * A, v=3 * A, qs=256, ks=128, vs=128, kp=16 * A, vp=32 * A, kps=2048, vps=2048, table=4 * A,
             ts=8, lens=5 * A, cu=None, N=4, T=8, Hq=4, Hk=2, D=64, P=64, M=8, ps=16, dtype=BF16, f=6 * A, R=64,
             flags=0, scale=1.0, qo=7 * A)
    a.update(kw)
    return _paged._api().kda_cache_append(
        a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["kp"], a["vp"], a["kps"], a["vps"], a["table"],
        a["ts"], a["lens"], a["cu"], a["N"], a["T"], a["Hq"], a["Hk"], a["D"], a["P"], a["M"], a["ps"], a["dtype"],
        a["f"], a["R"], a["flags"], a["scale"], a["qo"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(N=0), INVALID),
    (dict(N=3), INVALID),                 # equal lengths need T % N == 0
    (dict(T=-8), INVALID),
    (dict(P=0), INVALID),
    (dict(M=0), INVALID),
    (dict(ts=7), INVALID),
    (dict(ps=48), NOT_SUPPORTED),
    (dict(ps=8), NOT_SUPPORTED),
    (dict(ps=512), NOT_SUPPORTED),
    (dict(D=72), NOT_SUPPORTED),
    (dict(R=8), NOT_SUPPORTED),
    (dict(dtype=9), NOT_SUPPORTED),
    (dict(flags=2), NOT_SUPPORTED),       # the append has no inverse
    (dict(table=None), INVALID),
    (dict(lens=5 * A + 1), INVALID),
    (dict(cu=9 * A + 2), INVALID),
    (dict(k=None), INVALID),
    (dict(v=3 * A + 4), INVALID),
    (dict(qo=None), INVALID),
    (dict(f=None), INVALID),              # q without frequencies
    (dict(kps=2047), INVALID),
    (dict(vps=1024), INVALID),
    (dict(kp=32 * A), INVALID),           # K and V in the same pages
    (dict(k=16 * A + 4096), INVALID),     # new keys inside the cache
    (dict(qo=32 * A), INVALID),
    (dict(qo=2 * A), INVALID),
    (dict(scale=float("inf")), INVALID),
    (dict(Hk=0), INVALID),
])
def test_append_refusals(kw, expect):
    assert _append(**kw) == expect


def _attn(**kw):
    a = dict(q=A, qs=512, kp=16 * A, vp=32 * A, kps=2048, vps=2048, table=4 * A, ts=8, lens=5 * A, cu=None, N=4,
             T=8, Hq=8, Hk=2, D=64, P=64, M=8, ps=16, dtype=BF16, scale=0.1, window=0, o=2 * A, lse=3 * A,
             ws=64 * A, wsb=BIG)
    a.update(kw)
    return _paged._api().kda_attn_paged(
        a["q"], a["qs"], a["kp"], a["vp"], a["kps"], a["vps"], a["table"], a["ts"], a["lens"], a["cu"], a["N"],
        a["T"], a["Hq"], a["Hk"], a["D"], a["P"], a["M"], a["ps"], a["dtype"], a["scale"], a["window"], a["o"],
        a["lse"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(N=0), INVALID),
    (dict(N=3), INVALID),
    (dict(T=-1), INVALID),
    (dict(Hq=7), INVALID),                # not a multiple of the K/V heads
    (dict(Hk=0), INVALID),
    (dict(D=96), NOT_SUPPORTED),
    (dict(D=32), NOT_SUPPORTED),
    (dict(ps=24), NOT_SUPPORTED),
    (dict(dtype=3), NOT_SUPPORTED),
    (dict(scale=0.0), INVALID),
    (dict(scale=-1.0), INVALID),
    (dict(scale=float("nan")), INVALID),
    (dict(window=-1), INVALID),
    (dict(q=None), INVALID),
    (dict(o=None), INVALID),
    (dict(o=A), INVALID),
    (dict(o=16 * A + 64), INVALID),
    (dict(lse=2 * A), INVALID),
    (dict(lse=3 * A + 2), INVALID),
    (dict(lse=32 * A), INVALID),
    (dict(qs=511), INVALID),
    (dict(kp=16 * A + 8), INVALID),
    (dict(vps=2040), INVALID),
    (dict(ws=None), INVALID),
    (dict(ws=64 * A + 128), INVALID),
    (dict(wsb=16), WS_SMALL),
    (dict(T=1 << 30, N=1, Hq=8), INVALID),  # more rows than are numbered
])
def test_attn_refusals(kw, expect):
    assert _attn(**kw) == expect


def _pool(**kw):
    a = dict(base=16 * A, outer_stride=4096 * 64, page_stride=4096, page_bytes=4096, outer=2, num_pages=64)
    a.update(kw)
    return _paged._Pool(a["base"], a["outer_stride"], a["page_stride"], a["page_bytes"], a["outer"], a["num_pages"])


def _arr(*pools):
    return (_paged._Pool * len(pools))(*pools)


def _fork(pools=None, n=None, **kw):
    a = dict(refs=A, table=2 * A, ts=8, lens=3 * A, par=4 * A, kids=5 * A, count=3, N=4, P=64, M=8, ps=16,
             granted=6 * A, ws=64 * A, wsb=BIG)
    a.update(kw)
    pools = [_pool()] if pools is None else pools
    return _paged._api().kda_pages_fork(_arr(*pools) if pools else None, len(pools) if n is None else n, a["refs"], a["table"],
                                        a["ts"], a["lens"], a["par"], a["kids"], a["count"], a["N"], a["P"], a["M"],
                                        a["ps"], a["granted"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(refs=None), INVALID), (dict(table=2 * A + 1), INVALID), (dict(lens=None), INVALID),
    (dict(count=-1), INVALID), (dict(N=0), INVALID), (dict(P=0), INVALID), (dict(M=0), INVALID),
    (dict(ts=7), INVALID), (dict(ps=20), NOT_SUPPORTED), (dict(par=None), INVALID), (dict(kids=5 * A + 2), INVALID),
    (dict(granted=None), INVALID), (dict(ws=None), INVALID), (dict(ws=64 * A + 4), INVALID), (dict(wsb=64), WS_SMALL),
    (dict(pools=[], n=1), INVALID), (dict(pools=[], n=-1), INVALID), (dict(pools=[_pool()] * 9), INVALID),
    (dict(pools=[_pool(num_pages=63)]), INVALID),      # not the counted pages
    (dict(pools=[_pool(base=16 * A + 8)]), INVALID), (dict(pools=[_pool(page_bytes=24)]), INVALID),
    (dict(pools=[_pool(page_stride=4080)]), INVALID), (dict(pools=[_pool(outer_stride=4096)]), INVALID),
    (dict(pools=[_pool(outer=0)]), INVALID), (dict(pools=[_pool(page_bytes=0)]), INVALID),
    (dict(count=0), SUCCESS),                          # nothing to do, nothing enqueued
])
def test_fork_refusals(kw, expect):
    assert _fork(**kw) == expect


def test_alloc_free_compact_copy_refusals():
    L = _paged._api()

    def alloc(refs=A, seqs=3 * A, new=4 * A, count=3, wsb=BIG, granted=5 * A, ps=16):
        return L.kda_pages_alloc(refs, 2 * A, 8, 6 * A, seqs, new, count, 4, 64, 8, ps, granted, 64 * A, wsb, None)

    assert alloc(refs=None) == INVALID
    assert alloc(seqs=None) == INVALID        # without a list, one request per sequence
    assert alloc(new=None) == INVALID
    assert alloc(granted=5 * A + 1) == INVALID
    assert alloc(ps=0) == NOT_SUPPORTED
    assert alloc(wsb=4) == WS_SMALL
    assert alloc(count=0) == SUCCESS

    def free(refs=A, seqs=3 * A, count=3, ts=8):
        return L.kda_pages_free(refs, 2 * A, ts, 6 * A, seqs, count, 4, 64, 8, 16, None)

    assert free(refs=A + 2) == INVALID
    assert free(seqs=None) == INVALID
    assert free(ts=4) == INVALID
    assert free(count=-2) == INVALID
    assert free(count=0) == SUCCESS

    def compact(pools=(_pool(),), refs=A, table=2 * A, out_refs=A, out_table=2 * A, ots=8, moved=3 * A, ws=64 * A,
                wsb=BIG, P=64):
        return L.kda_pages_compact(_arr(*pools), len(pools), refs, table, 8, 4, P, 8, out_refs, out_table, ots,
                                   moved, ws, wsb, None)

    assert compact(refs=None) == INVALID
    assert compact(out_refs=A + 16) == INVALID     # partly over page_refs
    assert compact(out_table=2 * A + 16) == INVALID
    assert compact(ots=9) == INVALID               # in place with other strides
    assert compact(out_refs=2 * A) == INVALID
    assert compact(moved=None) == INVALID
    assert compact(moved=A) == INVALID
    assert compact(ws=None) == INVALID
    assert compact(wsb=8) == WS_SMALL
    assert compact(P=0) == INVALID
    assert compact(pools=(_pool(num_pages=5),)) == INVALID

    def copy(pools=(_pool(),), src=A, dst=2 * A, count=3):
        return L.kda_pages_copy(_arr(*pools), len(pools), src, dst, count, None)

    assert copy(src=None) == INVALID
    assert copy(dst=2 * A + 2) == INVALID
    assert copy(count=-1) == INVALID
    assert copy(pools=(_pool(page_stride=16),)) == INVALID
    assert copy(count=0) == SUCCESS
    # planes inside pages (a pool of [page][layer]) are as good as pages inside planes
    inside = _pool(outer_stride=4096, page_stride=2 * 4096)
    assert copy(pools=(inside,), count=0) == SUCCESS


def test_workspace_sizes():
    ws = kda.attn_workspace_size
    assert ws(4, 4, 32, 8, 128, torch.bfloat16) > 0
    assert ws(0, 4, 32, 8, 128, torch.bfloat16) == 0
    assert ws(4, 4, 30, 8, 128, torch.bfloat16) == 0
    assert ws(4, 4, 32, 8, 100, torch.bfloat16) == 0
    assert ws(4, -1, 32, 8, 128, torch.float32) == 0
    L = _paged._api()
    assert L.kda_pages_plan_workspace_size(0, 1, 1) > 0
    assert L.kda_pages_plan_workspace_size(1, 0, 1) == 0
    assert L.kda_pages_compact_workspace_size(0) == 0


def test_binding_refusals_on_the_cpu():
    """Shapes, types, strides and devices are refused in Python before the library is called."""
    q, k = torch.zeros((4, 2, 64)), torch.zeros((4, 1, 64))
    pos, f = torch.zeros(4, dtype=torch.int32), kda.rope_freqs(64)[0]
    with pytest.raises(ValueError):
        kda.rope(q, k, pos, f)                               # not on a GPU
    for bad in (dict(q=q.half()), dict(k=torch.zeros((3, 1, 64))), dict(pos=pos.long()), dict(pos=pos[:3]),
                dict(f=f.float()), dict(q=q.transpose(0, 1)), dict(q=q[..., ::2], k=None), dict(q=None, k=None)):
        a = dict(q=q, k=k, pos=pos, f=f)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            kda.rope(a["q"], a["k"], a["pos"], a["f"])
    with pytest.raises(ValueError):
        kda.rope(q, None, pos, f, k_out=k)
    with pytest.raises(ValueError):
        kda.rope_freqs(64, scaling="other")
    with pytest.raises(ValueError):
        kda.rope_freqs(63)
    cache = torch.zeros((6, 1, 16, 64))
    table, lens = torch.zeros((4, 3), dtype=torch.int32), torch.ones(4, dtype=torch.int32)
    for bad in (dict(kc=cache.double()), dict(vc=cache[:5]), dict(kc=cache.transpose(1, 2)), dict(kc=cache[:, :, ::2]),
                dict(table=table.long()), dict(table=table[:, ::2]), dict(lens=lens[:3]),
                dict(cu=torch.zeros(4, dtype=torch.int32)), dict(kc=cache[..., :32])):
        a = dict(kc=cache, vc=cache.clone(), table=table, lens=lens, cu=None)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            kda.attn_paged(q, a["kc"], a["vc"], a["table"], a["lens"], cu_seqlens=a["cu"])
        with pytest.raises((ValueError, TypeError)):
            kda.cache_append(k, k, a["kc"], a["vc"], a["table"], a["lens"], cu_seqlens=a["cu"])
    with pytest.raises(ValueError):
        kda.cache_append(k, k, cache, cache.clone(), table, lens, q=q)      # q without frequencies
    refs = torch.zeros(6, dtype=torch.int32)
    one = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        kda.pages_alloc(refs, table, lens, one, 16)
    with pytest.raises(ValueError):
        kda.pages_fork(cache, refs, table, lens, one, torch.zeros(2, dtype=torch.int32), 16)
    with pytest.raises(ValueError):
        kda.pages_copy(cache.transpose(2, 3), one, one)
    with pytest.raises(ValueError):
        kda.pages_copy([cache] * 9, one, one)
    with pytest.raises(TypeError):
        kda.pages_free(refs, table, lens, one.long(), 16)


# Rows of 4 + 2 heads of 64 bf16: q takes 512 bytes, k 256.
@pytest.mark.parametrize("kw", [
    dict(q=A, k=A + 256, qs=384, ks=384, qo=A, ko=6 * A),          # k begins inside q's heads
    dict(q=A + 128, k=A, qs=384, ks=384, qo=5 * A, ko=A),          # q begins inside k's
    dict(q=A, k=A + 512, qs=384, ks=512, qo=A, ko=6 * A),          # other strides: rows cross
])
def test_rope_in_place_over_the_other_input(kw):
    assert _rope(**kw) == INVALID


@pytest.mark.parametrize("kw", [
    dict(q=A, k=A + 256, qs=512, ks=512, qo=A),                    # k begins inside q's heads
    dict(q=A, v=A + 896, qs=512, vs=512, qo=A),                    # v ends inside the next token's q
])
def test_append_in_place_over_the_other_inputs(kw):
    assert _append(**kw) == INVALID


@pytest.mark.parametrize("at", ["q", "o", "lse", "kp", "vp"])
def test_attn_workspace_apart(at):
    base = dict(q=A, o=2 * A, lse=3 * A, kp=16 * A, vp=32 * A)
    assert _attn(ws=base[at]) == INVALID


def _plan_call(name, **kw):
    a = dict(refs=A, table=2 * A, ts=8, lens=3 * A, x=4 * A, y=5 * A, count=4, N=4, P=64, M=8, ps=16, granted=6 * A,
             ws=7 * A, wsb=BIG)
    a.update(kw)
    L = _paged._api()
    rest = (a["count"], a["N"], a["P"], a["M"], a["ps"], a["granted"], a["ws"], a["wsb"], None)
    if name == "alloc":
        return L.kda_pages_alloc(a["refs"], a["table"], a["ts"], a["lens"], a["x"], a["y"], *rest)
    return L.kda_pages_fork(None, 0, a["refs"], a["table"], a["ts"], a["lens"], a["x"], a["y"], *rest)


@pytest.mark.parametrize("name", ["alloc", "fork"])
@pytest.mark.parametrize("kw", [dict(ws=A), dict(ws=2 * A), dict(ws=3 * A), dict(ws=6 * A), dict(granted=A + 4),
                                dict(granted=2 * A + 64), dict(granted=3 * A), dict(P=(1 << 30) + 1)])
def test_plan_outputs_apart(name, kw):
    assert _plan_call(name, **kw) == INVALID


def test_page_count_limit():
    L = _paged._api()
    assert L.kda_pages_plan_workspace_size(1, 1, (1 << 30) + 1) == 0
    assert L.kda_pages_compact_workspace_size((1 << 30) + 1) == 0
    assert L.kda_pages_plan_workspace_size(1, 1, 1 << 30) >= 4 << 30
    assert _attn(P=(1 << 30) + 1) == INVALID
    assert _append(P=(1 << 30) + 1) == INVALID
    assert L.kda_pages_compact(None, 0, A, 2 * A, 8, 4, 64, 8, 3 * A, 4 * A, 8, 5 * A, A, BIG, None) == INVALID
