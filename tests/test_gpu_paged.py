"""The paged KV cache and the attention over it on the GPU, against the fp64 form row by row."""
import math

import pytest
import torch

import gated_delta_rule_30_amd as kda
import paged_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def make(new, ctx, Hq, Hk, D, ps, dtype, seed=0, extra_rows=0, spare=3, width=None, garbage=math.nan):
    """A cache of sequences with ctx[n] stored tokens before their new[n] new ones; what lies in
    the pool beside them is ``garbage``."""
    gen = torch.Generator().manual_seed(seed + 1)
    lens = [c + m for c, m in zip(ctx, new)]
    need = [-(-max(0, x) // ps) for x in lens]
    P = sum(need) + spare
    order = torch.randperm(P, generator=gen).tolist()
    W = width or max(need + [1]) + 1
    table = torch.full((len(new), W), -1, dtype=torch.int32)
    kc = torch.full((P, Hk, ps, D), garbage, dtype=dtype)
    vc = torch.full((P, Hk, ps, D), garbage, dtype=dtype)
    at = 0
    for n, m in enumerate(need):
        for j in range(m):
            p = order[at]
            at += 1
            table[n, j] = p
            rows = min(ps, lens[n] - j * ps)
            kc[p, :, :rows] = torch.randn((Hk, rows, D), generator=gen).to(dtype)
            vc[p, :, :rows] = torch.randn((Hk, rows, D), generator=gen).to(dtype)
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)
    q = torch.randn((cu[-1] + extra_rows, Hq, D), generator=gen).to(dtype)
    return dict(q=q, kc=kc, vc=vc, table=table, lens=torch.tensor(lens, dtype=torch.int32), cu=cu)


def dev(s):
    d = {k: s[k].to(DEV) for k in ("q", "kc", "vc", "table", "lens")}
    d["cu"] = torch.tensor(s["cu"], dtype=torch.int32, device=DEV)
    return d


def run(d, window=0, scale=None, cu=True, **kw):
    lse = torch.full(d["q"].shape[:2], 77.0, device=DEV)
    o = torch.full(d["q"].shape, 55.0, dtype=d["q"].dtype, device=DEV)
    kda.attn_paged(d["q"], d["kc"], d["vc"], d["table"], d["lens"], cu_seqlens=d["cu"] if cu else None,
                   window=window, scale=scale, o=o, lse=lse, **kw)
    return o, lse


def check(s, o, lse, window=0, scale=None):
    D = s["q"].shape[-1]
    ro, rl, to, tl = ref.attention(s["q"], s["kc"], s["vc"], s["table"], s["lens"], s["cu"],
                                   D ** -0.5 if scale is None else scale, window)
    o, lse, T = o.double().cpu(), lse.double().cpu(), s["cu"][-1]
    assert torch.equal(o[T:], torch.full_like(o[T:], 55.0)), "rows behind the last sequence"
    assert torch.equal(lse[T:], torch.full_like(lse[T:], 77.0))
    o, lse, ro, rl, to, tl = o[:T], lse[:T], ro[:T], rl[:T], to[:T], tl[:T]
    empty = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse) & (lse < 0), empty)
    assert torch.all(o[empty] == 0)
    over = (o - ro).abs() - to
    assert not torch.isnan(o).any()
    assert over.numel() == 0 or over.max() <= 0, "o beyond its tolerance by %.3e" % over.max()
    over = ((lse - rl).abs() - tl)[~empty]
    assert over.numel() == 0 or over.max() <= 0, "lse beyond its tolerance by %.3e" % over.max()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Hq,Hk,D,ps", [(4, 4, 64, 16), (8, 2, 128, 16), (8, 1, 128, 64), (5, 1, 64, 32),
                                        (40, 2, 128, 128), (4, 2, 256, 16), (12, 4, 64, 256)])
def test_decode(Hq, Hk, D, ps, dtype):
    """One token per sequence: lengths around page and tile borders, an empty table row."""
    ctx = [0, 1, 14, 15, 16, 30, 31, 32, 63, 64, 126, 127, 128, 200, 511, 700]
    s = make([1] * len(ctx), ctx, Hq, Hk, D, ps, dtype, seed=Hq)
    d = dev(s)
    check(s, *run(d, cu=False))
    check(s, *run(d, cu=True))
    o = kda.attn_paged(d["q"], d["kc"], d["vc"], d["table"], d["lens"])
    assert torch.equal(o, run(d)[0])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Hq,Hk,D,ps,window", [(4, 2, 128, 16, 0), (8, 1, 64, 32, 40), (3, 3, 64, 16, 1),
                                               (4, 1, 256, 64, 100), (2, 2, 128, 256, 0), (7, 1, 128, 32, 17)])
def test_chunks(Hq, Hk, D, ps, window, dtype):
    """Ragged chunks beside single tokens and empty sequences, rows behind the last one."""
    new = [33, 1, 0, 130, 5, 1, 64, 17]
    ctx = [0, 300, 20, 100, 0, 0, 63, 250]
    s = make(new, ctx, Hq, Hk, D, ps, dtype, seed=D + Hq, extra_rows=3)
    check(s, *run(dev(s), window=window), window=window)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window", [0, 300])
def test_long_split(window, dtype):
    """Long contexts over few rows, which are split over many workgroups and joined."""
    s = make([1, 3, 40], [5000, 2100, 1500], 8, 2, 128, 64, dtype, seed=9)
    check(s, *run(dev(s), window=window), window=window)
    s = make([1], [6000], 2, 1, 64, 16, dtype, seed=10)
    check(s, *run(dev(s), window=window, cu=False), window=window)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_one_long_chunk(dtype):
    s = make([400], [700], 2, 1, 128, 16, dtype, seed=12)
    check(s, *run(dev(s), cu=False))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_without_keys(dtype):
    """Lengths shorter than the new tokens (negative positions), zero lengths, entries that name
    no page, lengths beyond the table."""
    s = make([4, 2, 3, 40, 1, 1], [60, 30, 40, 90, 100, 0], 4, 2, 64, 16, dtype, seed=2)
    s["lens"][0] = 2            # rows at -2, -1, 0, 1
    s["lens"][1] = 0            # rows at -2, -1
    s["table"][2, :] = -1       # no page at all
    s["table"][3, 2] = 10 ** 6  # holes
    s["table"][3, 5] = -7
    s["lens"][4] = s["table"].shape[1] * 16 + 50
    s["table"][4, :] = -1
    s["table"][4, 1] = s["table"][3, 0]
    s["lens"][5] = -5
    check(s, *run(dev(s)))
    check(s, *run(dev(s), window=7), window=7)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("window", [0, 20])
@pytest.mark.parametrize("new,ctx", [([70], [30]), ([6, 1, 3], [40, 80, 150])])
def test_unseen_values_do_not_reach_the_result(new, ctx, window, bad, dtype):
    """NaN and infinities in keys and values of later tokens (hidden from earlier rows by the
    causal mask), left of every window, and in the rest of the pool."""
    s = make(new, ctx, 4, 2, 128, 16, dtype, seed=7, garbage=bad)
    clean = dev(s)
    o0, l0 = run(clean, window=window)
    for n in range(len(new)):
        L = int(s["lens"][n])
        hit = [L - 1]  # the last token: its own row alone sees it
        if window:
            hit += list(range(0, max(0, L - new[n] - window)))
        for j in hit:
            p = int(s["table"][n, j // 16])
            s["kc"][p, :, j % 16] = bad
            s["vc"][p, :, j % 16] = bad
    o1, l1 = run(dev(s), window=window)
    last = torch.tensor(s["cu"][1:], device=DEV) - 1
    keep = torch.ones(o0.shape[0], dtype=torch.bool, device=DEV)
    keep[last] = False
    assert torch.isfinite(o0.float()).all()
    assert torch.equal(o0[keep], o1[keep]) and torch.equal(l0[keep], l1[keep])
    if bad != bad:
        assert torch.isnan(o1[last].float()).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_values_alone_unseen(dtype):
    """Only V is infinite at a later token: the rows that see it carry it, the others do not."""
    s = make([40], [11], 4, 2, 64, 16, dtype, seed=8)
    o0, _ = run(dev(s))
    j = 11 + 25
    s["vc"][int(s["table"][0, j // 16]), 1, j % 16, 5] = math.inf
    o1, _ = run(dev(s))
    assert torch.equal(o0[:25], o1[:25])
    assert torch.equal(o0[:, :2], o1[:, :2])
    assert torch.isinf(o1[25:, 2:, 5].float()).all()
    rest = [c for c in range(64) if c != 5]
    assert torch.equal(o0[:, :, rest], o1[:, :, rest])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_an_infinity_far_back(D, dtype):
    """An infinity and a NaN among the values of a long context, in different parts of it: every row
    that sees them carries them, in their channels alone."""
    s = make([150, 1], [2500, 700], 4, 2, D, 32, dtype, seed=21)
    o0, l0 = run(dev(s))
    for n, j, ch, x in ((0, 1700, 3, -math.inf), (0, 77, D - 1, math.nan), (0, 2500 + 60, 17, math.inf), (1, 300, 9, math.inf)):
        s["vc"][int(s["table"][n, j // 32]), 0, j % 32, ch] = x
    o1, l1 = run(dev(s))
    assert torch.equal(l0, l1) and torch.equal(o0[:, 2:], o1[:, 2:])
    a, b = o1[:150, :2].float(), o1[150, :2].float()
    assert (a[:, :, 3] == -math.inf).all() and torch.isnan(a[:, :, D - 1]).all()
    assert (a[60:, :, 17] == math.inf).all() and torch.equal(o0[:60, :2, 17], o1[:60, :2, 17])
    assert not torch.isfinite(b[:, 9]).any()
    rest = [c for c in range(D) if c not in (3, 9, 17, D - 1)]
    assert torch.equal(o0[:, :, rest], o1[:, :, rest])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("scale", [1e-36, 1e-3, 3.0])
def test_scales(scale, dtype):
    """From a scale that makes all weights equal to one that leaves a few: rows split over
    workgroups and not."""
    for new, ctx in (([1, 50], [1500, 100]), ([1, 1], [700, 20])):
        s = make(new, ctx, 2, 1, 64, 16, dtype, seed=22)
        check(s, *run(dev(s), scale=scale), scale=scale)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_large_scores(dtype):
    """Scores of a few hundred, growing and falling along the sequence: the running maximum moves
    often, and early weights vanish."""
    for sign in (1, -1):
        s = make([50, 1], [200, 300], 2, 1, 64, 16, dtype, seed=11)
        s["q"] *= 8
        for n in range(2):
            for j in range(int(s["lens"][n])):
                p = int(s["table"][n, j // 16])
                s["kc"][p, :, j % 16] *= 1 + 0.02 * (j if sign > 0 else 300 - j)
        check(s, *run(dev(s)))


def test_equal_keys_give_the_mean():
    """All keys alike: every weight is 1 / n exactly representable sums; all scores -inf: a row of
    zeros."""
    s = make([2], [126], 2, 2, 64, 16, F32, seed=3)
    s["kc"][:] = 0.0
    o, lse = run(dev(s))
    check(s, o, lse)
    s["kc"][:] = -math.inf
    s["q"][:] = 1.0
    o, lse = run(dev(s))
    assert torch.all(o == 0) and torch.all(torch.isinf(lse) & (lse < 0))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides(dtype):
    """q as a slice of a fused projection, pages of one pool that holds K and V of two layers, a
    table that is part of a wider one: the same bits as contiguous tensors."""
    for new, ctx in (([1, 1, 1], [40, 3, 200]), ([40, 1, 20], [17, 90, 0])):
        s = make(new, ctx, 4, 2, 64, 16, dtype, seed=4)
        d = dev(s)
        want = run(d)
        T, P = d["q"].shape[0], d["kc"].shape[0]
        qkv = torch.zeros((T, 8, 64), dtype=dtype, device=DEV)
        qkv[:, :4] = d["q"]
        pool = torch.zeros((P, 2, 2, 2, 16, 64), dtype=dtype, device=DEV)
        pool[:, 1, 0], pool[:, 1, 1] = d["kc"], d["vc"]
        wide = torch.full((len(new), d["table"].shape[1] + 9), 0, dtype=torch.int32, device=DEV)
        wide[:, 4:4 + d["table"].shape[1]] = d["table"]
        d2 = dict(d, q=qkv[:, :4], kc=pool[:, 1, 0], vc=pool[:, 1, 1],
                  table=wide[:, 4:4 + d["table"].shape[1]])
        got = run(d2)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new,ctx", [([1, 1, 1, 1], [0, 15, 16, 77]), ([40, 0, 1, 300], [5, 9, 31, 64])])
def test_append(new, ctx, dtype, inter):
    """k and v of the new tokens in their pages, k and q turned by their positions; everything
    else in the pool, and rows behind the last sequence, as they were."""
    Hq, Hk, D, ps, R = 6, 2, 64, 16, 32
    s = make(new, ctx, Hq, Hk, D, ps, dtype, seed=5, extra_rows=2, garbage=3.0)
    gen = torch.Generator().manual_seed(9)
    T, rows = s["cu"][-1], s["q"].shape[0]
    k, v = (torch.randn((rows, Hk, D), generator=gen).to(dtype) for _ in range(2))
    f, _ = kda.rope_freqs(R)
    d = dev(s)
    kc, vc = d["kc"].clone(), d["vc"].clone()
    q_out = torch.full((rows, Hq, D), 9.0, dtype=dtype, device=DEV)
    kda.cache_append(k.to(DEV), v.to(DEV), kc, vc, d["table"], d["lens"], cu_seqlens=d["cu"], q=d["q"],
                     inv_freq=f.to(DEV), interleaved=inter, scale=1.25, q_out=q_out)
    at = ref.positions(s["lens"], s["cu"])
    pos = [p for _, _, p in at]
    qw, qs = ref.rope(s["q"][:T].double().numpy(), pos, f.numpy(), inter, 1.25)
    kw, ks = ref.rope(k[:T].double().numpy(), pos, f.numpy(), inter, 1.25)
    err = abs(q_out[:T].double().cpu().numpy() - qw) - ref.rope_tol(qw, qs, 1.25, dtype)
    assert err.max() <= 0
    assert torch.all(q_out[T:] == 9.0)
    want_k, want_v = s["kc"].clone(), s["vc"].clone()
    got_k = kc.cpu().clone()
    for t, n, p in at:
        pg, r = int(s["table"][n, p // ps]), p % ps
        err = abs(got_k[pg, :, r].double().numpy() - kw[t]) - ref.rope_tol(kw[t], ks[t], 1.25, dtype)
        assert err.max() <= 0
        got_k[pg, :, r] = want_k[pg, :, r]
        want_v[pg, :, r] = v[t]
    assert torch.equal(got_k, want_k) and torch.equal(vc.cpu(), want_v)
    # without rotation, k as it is; rows of T / N each without cu_seqlens
    kc, vc = d["kc"].clone(), d["vc"].clone()
    assert kda.cache_append(k.to(DEV), v.to(DEV), kc, vc, d["table"], d["lens"], cu_seqlens=d["cu"]) is None
    for t, n, p in at:
        want_k[int(s["table"][n, p // ps]), :, p % ps] = k[t]
    assert torch.equal(kc.cpu(), want_k) and torch.equal(vc.cpu(), want_v)
    if all(m == 1 for m in new):
        kc2, vc2 = d["kc"].clone(), d["vc"].clone()
        kda.cache_append(k[:T].to(DEV), v[:T].to(DEV), kc2, vc2, d["table"], d["lens"])
        assert torch.equal(kc2, kc) and torch.equal(vc2, vc)


def test_append_in_place_and_nowhere():
    """q turned in place in a fused projection; tokens at negative positions, in rows without a
    page and past the table are stored nowhere."""
    s = make([3, 2, 2, 1], [20, 5, 20, 3], 2, 1, 64, 16, BF16, seed=6, garbage=1.0)
    s["lens"][0] = 1           # rows at -2, -1, 0
    s["table"][1, :] = 99
    s["lens"][2] = s["table"].shape[1] * 16 + 1  # its last token is past the table
    s["table"][2, -1] = s["table"][2, 0]
    d = dev(s)
    T = s["cu"][-1]
    qkv = torch.randn((T, 4, 64), device=DEV).bfloat16()
    f, _ = kda.rope_freqs(64, device=DEV)
    want = kda.cache_append(qkv[:, 2:3], qkv[:, 3:], d["kc"].clone(), d["vc"].clone(), d["table"], d["lens"],
                            cu_seqlens=d["cu"], q=qkv[:, :2], inv_freq=f)
    kc, vc, mine = d["kc"].clone(), d["vc"].clone(), qkv.clone()
    kda.cache_append(mine[:, 2:3], mine[:, 3:], kc, vc, d["table"], d["lens"], cu_seqlens=d["cu"],
                     q=mine[:, :2], inv_freq=f, q_out=mine[:, :2])
    assert torch.equal(mine[:, :2], want) and torch.equal(mine[:, 2:], qkv[:, 2:])
    expect = s["vc"].clone()
    for t, n, p in ref.positions(s["lens"], s["cu"]):
        j = p // 16
        if p >= 0 and j < s["table"].shape[1] and 0 <= int(s["table"][n, j]) < expect.shape[0]:
            expect[int(s["table"][n, j]), :, p % 16] = qkv[t, 3:].cpu()
    assert torch.equal(vc.cpu(), expect)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new,ctx", [([1, 60, 1, 3], [900, 30, 2000, 77]), ([400], [700]), ([40], [11]),
                                     ([1, 1, 1], [900, 17, 2000])])
def test_same_bits_every_run(new, ctx, D, dtype):
    s = make(new, ctx, 8, 2, D, 16, dtype, seed=13)
    d = dev(s)
    a = run(d)
    for _ in range(5):
        b = run(d)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows", [31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257])
def test_rows_at_the_borders(rows, dtype):
    """As many rows as either kernel takes at most, one less and one more, and so at the tiles' sizes."""
    s = make([rows] * 2, [100, 0], 1, 1, 64, 16, dtype, seed=rows)
    d = dev(s)
    check(s, *run(d, cu=False))
    check(s, *run(d))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_shares_of_many_steps(dtype):
    """Tiles whose workgroups walk over more steps than one reading of the page table covers (64)."""
    s = make([300], [40000], 16, 16, 64, 64, dtype, seed=21)
    o, lse = run(dev(s))
    some = slice(0, 16, 15)  # (the first and the last head: the rest would take the fp64 form a minute)
    check(dict(s, q=s["q"][:, some], kc=s["kc"][:, some], vc=s["vc"][:, some]), o[:, some], lse[:, some])


def test_two_calls_at_once():
    """Two batches on two streams, with a workspace each: neither sees the other."""
    batches = [make([200, 1, 40], [900, 2000, 77], 8, 2, 128, 16, BF16, seed=31),
               make([1, 1, 1], [3000, 20, 500], 8, 2, 128, 16, BF16, seed=32)]
    devs = [dev(s) for s in batches]
    want = [run(d) for d in devs]
    size = [kda.attn_workspace_size(3, d["q"].shape[0], 8, 2, 128, BF16) for d in devs]
    work = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in size]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(run(devs[i], workspace=work[i]))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for o, lse in g:
            assert torch.equal(o, w[0]) and torch.equal(lse, w[1])


def test_other_stream():
    s = make([1, 60, 1, 3], [900, 30, 2000, 77], 8, 2, 128, 16, BF16, seed=13)
    d = dev(s)
    want = run(d)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = run(d)
    st.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_graph_replay_follows_the_lengths():
    """Append and attention of a decode step captured once and replayed as the sequences grow: each replay
    equals an eager step. The workspace holds what an earlier call left."""
    Hq, Hk, D, ps = 8, 2, 128, 16
    s = make([1, 1, 1], [30, 500, 1200], Hq, Hk, D, ps, BF16, seed=14, width=90, spare=30)
    for n, L in enumerate([31, 501, 1201]):  # pages for what comes
        have = -(-L // ps)
        used = set(s["table"].flatten().tolist())
        free = [p for p in range(s["kc"].shape[0]) if p not in used]
        s["table"][n, have:have + 3] = torch.tensor(free[:3], dtype=torch.int32)
    d = dev(s)
    f, _ = kda.rope_freqs(D, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(3)
    qkv = torch.randn((3, Hq + 2 * Hk, D), generator=gen, device=DEV).bfloat16()
    ws = torch.empty(kda.attn_workspace_size(3, 3, Hq, Hk, D, BF16), dtype=torch.uint8, device=DEV)
    q_out = torch.empty((3, Hq, D), dtype=BF16, device=DEV)
    o = torch.empty_like(q_out)

    def step():
        kda.cache_append(qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:], d["kc"], d["vc"], d["table"], d["lens"],
                         q=qkv[:, :Hq], inv_freq=f, q_out=q_out)
        kda.attn_paged(q_out, d["kc"], d["vc"], d["table"], d["lens"], o=o, workspace=ws)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
    torch.cuda.current_stream().wait_stream(st)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for rep in range(20):  # across a page border in each sequence
        d["lens"].add_(1)
        qkv.copy_(torch.randn(qkv.shape, generator=gen, device=DEV).bfloat16())
        kc, vc = d["kc"].clone(), d["vc"].clone()
        o.fill_(math.nan)
        ws.fill_(255)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got, gk, gv = o.clone(), d["kc"].clone(), d["vc"].clone()
        d["kc"].copy_(kc)
        d["vc"].copy_(vc)
        o.fill_(math.nan)
        step()
        torch.cuda.synchronize()
        assert torch.isfinite(o.float()).all() and torch.equal(got, o), rep
        for a, b in ((gk, d["kc"]), (gv, d["vc"])):  # bits: the rest of the pool is NaN
            assert torch.equal(a.view(torch.int16), b.view(torch.int16)), rep


def test_far_offsets():
    """A page more than 2^32 elements into the pool."""
    Hk, ps, D = 1, 256, 128
    P = (1 << 32) // (Hk * ps * D) + 3
    free, _ = torch.cuda.mem_get_info()
    if free < 3 * P * Hk * ps * D * 2:
        pytest.skip("needs %d GB" % (3 * P * Hk * ps * D * 2 >> 30))
    s = make([1, 20], [300, 40], 4, Hk, D, ps, BF16, seed=15, garbage=0.0)
    n = s["kc"].shape[0]
    kc = torch.zeros((P, Hk, ps, D), dtype=BF16, device=DEV)
    vc = torch.zeros((P, Hk, ps, D), dtype=BF16, device=DEV)
    d = dev(s)
    kc[P - n:], vc[P - n:] = d["kc"], d["vc"]
    want = run(d)
    far = torch.where(d["table"] >= 0, d["table"] + (P - n), d["table"])
    got = run(dict(d, kc=kc, vc=vc, table=far.contiguous()))
    assert torch.equal(got[0], want[0])
    k = torch.randn((21, Hk, D), device=DEV).bfloat16()
    kda.cache_append(k, k, kc, vc, far.contiguous(), d["lens"], cu_seqlens=d["cu"])
    kda.cache_append(k, k, d["kc"], d["vc"], d["table"], d["lens"], cu_seqlens=d["cu"])
    assert torch.equal(kc[P - n:], d["kc"]) and torch.equal(vc[P - n:], d["vc"])
    assert not kc[:P - n].any()
