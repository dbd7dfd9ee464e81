"""What is measured of the operators of a hybrid stack's full-attention layers: rotary positions, the
append to a paged KV cache, attention over it, and the pages' bookkeeping and copies. Each case is given
in plain torch operations and as the calls a user makes of the framework."""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _kda():
    import gated_delta_rule_30_amd as kda
    return kda


# ---------------------------------------------------------------------------------------- cases
def listed():
    return [
        # rotary positions of a training step, forward and backward: packed sequences of q and k as
        # slices of a fused projection, positions far out on a scaled context
        dict(name="rope_train_16k", kind="rope", T=16384, Hq=32, Hk=8, D=128, R=128, inter=False, base=500000.0,
             factor=8.0, far=1 << 20, dtype="bf16", mix=1),
        # fp32, an odd token count, half of the head rotated in the interleaved layout
        dict(name="rope_fp32_partial", kind="rope", T=1023, Hq=16, Hk=16, D=64, R=32, inter=True, base=10000.0,
             factor=1.0, far=32768, dtype="fp32", mix=2),
        # one decode step's append for a full batch: one launch between the projection and the attention
        dict(name="append_decode_256", kind="append", N=256, new_lo=1, new_hi=1, ctx_lo=1, ctx_hi=700, Hq=32, Hk=8,
             D=128, ps=16, R=128, inter=False, dtype="bf16", mix=3),
        # chunks of prompts being stored, ragged
        dict(name="append_chunks", kind="append", N=20, new_lo=64, new_hi=2048, ctx_lo=0, ctx_hi=1500, Hq=32, Hk=4,
             D=128, ps=64, R=64, inter=False, dtype="bf16", mix=4),
        # a handful of short conversations, one token each: latency
        dict(name="attn_decode_small", kind="attn", N=4, new_lo=1, new_hi=1, ctx_lo=200, ctx_hi=1000, Hq=32, Hk=8,
             D=128, ps=16, window=0, dtype="bf16", mix=5),
        # a serving batch with long ragged contexts, one token each: bandwidth
        dict(name="attn_decode_long", kind="attn", N=64, new_lo=1, new_hi=1, ctx_lo=1024, ctx_hi=32768, Hq=32, Hk=8,
             D=128, ps=64, window=0, dtype="bf16", mix=6),
        # a mixed batch: decode tokens beside prompt chunks, sliding window
        dict(name="attn_mixed_window", kind="attn", N=24, new_lo=1, new_hi=512, ctx_lo=1, ctx_hi=8192, Hq=32, Hk=4,
             D=64, ps=32, window=1024, dtype="bf16", mix=7),
        # a long prompt's chunk over what is stored of it: matrix rate
        dict(name="attn_chunk_long", kind="attn", N=1, new_lo=4096, new_hi=4096, ctx_lo=16384, ctx_hi=16384, Hq=32, Hk=8,
             D=128, ps=64, window=0, dtype="bf16", mix=8),
        # fp32 cache and queries, one K/V head per query head
        dict(name="attn_chunk_fp32", kind="attn", N=3, new_lo=100, new_hi=300, ctx_lo=500, ctx_hi=4000, Hq=16, Hk=16,
             D=128, ps=16, window=0, dtype="fp32", mix=9),
        # one sequence branching into four drafts: the old branches are freed, new ones forked, room for the
        # draft tokens taken, the recurrent states copied along
        dict(name="branch_small", kind="branch", parents=1, fan=4, draft=5, ctx_lo=300, ctx_hi=700, layers=1, Hk=2,
             D=128, ps=16, P=512, H=4, mix=10),
        # the same for a batch
        dict(name="branch_batch", kind="branch", parents=32, fan=3, draft=8, ctx_lo=500, ctx_hi=6000, layers=2, Hk=2,
             D=128, ps=64, P=4096, H=16, mix=11),
        # a fragmented pool closed up after long sequences have left
        dict(name="compact_pool", kind="compact", P=8192, live=0.6, N=128, layers=2, Hk=2, D=128, ps=64, mix=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "append", "attn", "attn", "attn", "branch", "compact"])
    mix = rng.randrange(1 << 30)
    if kind == "rope":
        D = rng.choice([64, 128, 256])
        Hk = rng.choice([1, 2, 4, 8])
        return dict(kind=kind, T=_log(rng, 1, 16384), Hq=Hk * rng.choice([1, 2, 4]), Hk=Hk, D=D,
                    R=rng.choice([D, D // 2]), inter=rng.random() < 0.5, base=rng.choice([10000.0, 500000.0]),
                    factor=rng.choice([1.0, 4.0, 32.0]), far=_log(rng, 100, 1 << 20), dtype=rng.choice(["bf16", "fp32"]),
                    mix=mix)
    D = rng.choice([64, 128])
    Hk = rng.choice([1, 2, 4, 8])
    ps = rng.choice([16, 32, 64, 128])
    if kind == "append":
        N = _log(rng, 1, 256)
        return dict(kind=kind, N=N, new_lo=1, new_hi=_log(rng, 1, max(1, 16384 // N)), ctx_lo=0, ctx_hi=_log(rng, 1, 1500),
                    Hq=Hk * rng.choice([1, 4, 8]), Hk=Hk, D=D, ps=ps, R=rng.choice([D, D // 2]), inter=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "bf16", "fp32"]), mix=mix)
    if kind == "attn":
        shape = rng.choice(["decode", "decode", "chunk", "mixed"])
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        G = rng.choice([1, 4, 8])
        window = rng.choice([0, 0, 0, _log(rng, 16, 4096)])
        if shape == "decode":
            N = _log(rng, 1, 96)
            return dict(kind=kind, N=N, new_lo=1, new_hi=rng.choice([1, 1, 4]), ctx_lo=1,
                        ctx_hi=_log(rng, 100, min(32768, 524288 // N)), Hq=Hk * G, Hk=Hk, D=D, ps=ps, window=window,
                        dtype=dtype, mix=mix)
        if shape == "chunk":
            new = _log(rng, 64, 2048)
            return dict(kind=kind, N=rng.choice([1, 1, 2]), new_lo=max(1, new // 2), new_hi=new, ctx_lo=0,
                        ctx_hi=_log(rng, 16, 8192), Hq=Hk * G, Hk=Hk, D=D, ps=ps, window=window, dtype=dtype, mix=mix)
        return dict(kind=kind, N=_log(rng, 2, 24), new_lo=1, new_hi=_log(rng, 8, 384), ctx_lo=0, ctx_hi=_log(rng, 64, 4096),
                    Hq=Hk * G, Hk=Hk, D=D, ps=ps, window=window, dtype=dtype, mix=mix)
    if kind == "branch":
        return dict(kind=kind, parents=_log(rng, 1, 32), fan=rng.randrange(1, 5), draft=rng.randrange(1, 17), ctx_lo=1,
                    ctx_hi=_log(rng, 50, 4000), layers=rng.choice([1, 2]), Hk=rng.choice([1, 2]), D=D, ps=rng.choice([32, 64]),
                    P=4096, H=rng.choice([1, 4, 16]), mix=mix)
    return dict(kind=kind, P=_log(rng, 100, 8192), live=rng.uniform(0.1, 0.95), N=_log(rng, 1, 128),
                layers=rng.choice([1, 2]), Hk=rng.choice([1, 2]), D=D, ps=rng.choice([16, 32, 64]), mix=mix)


def _spread(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm (lo may be 0)."""
    return int(math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 1)))) - 1 if hi > lo else lo


def _lengths(c):
    """New tokens of each sequence and its length with them: a part of the case, the same for every seed."""
    rng = random.Random(c["mix"])
    new = [max(c["new_lo"], min(c["new_hi"], _spread(rng, c["new_lo"], c["new_hi"]))) for _ in range(c["N"])]
    return new, [m + max(c["ctx_lo"], _spread(rng, c["ctx_lo"], c["ctx_hi"])) for m in new]


def _cu(new):
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)
    return cu


def _inv_freq(R, base, factor):
    """Radians per position of each pair, 64 bits: base^(-2i/R), and for a context that is `factor` times
    longer than the 8192 tokens of the original one, turns that are slow on it stretched by the factor, fast
    ones kept, a ramp between (32 and 1 turns)."""
    f = base ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    if factor != 1.0:
        at = [R * math.log(8192.0 / (t * 2 * math.pi)) / (2 * math.log(base)) for t in (32.0, 1.0)]
        low, high = max(0, math.floor(at[0])), min(R - 1, math.ceil(at[1]))
        keep = 1 - ((torch.arange(R // 2, dtype=torch.float64) - low) / max(high - low, 0.001)).clamp(0, 1)
        f = f / factor * (1 - keep) + f * keep
    return f


# ---------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1000003 * seed + 17)
    host = random.Random(7919 * seed + 11)

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (std * torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)).to(dtype)

    if c["kind"] == "rope":
        t = TYPES[c["dtype"]]
        T, Hq, Hk, D = c["T"], c["Hq"], c["Hk"], c["D"]
        qkv = normal(T, Hq + 2 * Hk, D, dtype=t)
        cuts = sorted(random.Random(c["mix"]).randrange(T) for _ in range(T // 1000))
        pos, at = [], 0
        for e in cuts + [T]:
            start = host.randrange(max(1, c["far"] - (e - at) + 1))
            pos += range(start, start + e - at)
            at = e
        return dict(c=c, q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hk], dq=normal(T, Hq, D, dtype=t), dk=normal(T, Hk, D, dtype=t),
                    pos=torch.tensor(pos, dtype=torch.int32, device=DEV),
                    inv_freq=_inv_freq(c["R"], c["base"], c["factor"]).to(DEV),
                    scale=1.0 + 0.1 * math.log(c["factor"]))
    if c["kind"] in ("append", "attn"):
        t = TYPES[c["dtype"]]
        Hq, Hk, D, ps = c["Hq"], c["Hk"], c["D"], c["ps"]
        new, lens = _lengths(c)
        need = [-(-x // ps) for x in lens]
        width, P = max(need) + 1, sum(need) + 7
        pages = list(range(P))
        host.shuffle(pages)
        table = torch.full((c["N"], width), -1, dtype=torch.int32)
        at = 0
        for n, m in enumerate(need):
            table[n, :m] = torch.tensor(pages[at:at + m], dtype=torch.int32)
            at += m
        T = sum(new)
        qkv = normal(T, Hq + 2 * Hk, D, dtype=t)
        cache = torch.empty((2, P, Hk, ps, D), dtype=t, device=DEV)
        for half in cache:
            for i in range(0, P, 4096):
                half[i:i + 4096] = torch.randn(half[i:i + 4096].shape, generator=gen, device=DEV).to(t)
        out = dict(c=c, q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hk], v=qkv[:, Hq + Hk:], kc=cache[0], vc=cache[1],
                   table=table.to(DEV), lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
                   cu=torch.tensor(_cu(new), dtype=torch.int32, device=DEV), most=max(new),
                   one=all(m == 1 for m in new))
        if c["kind"] == "append":
            out["inv_freq"] = _inv_freq(c["R"], 500000.0, 4.0).to(DEV)
        return out
    if c["kind"] == "branch":
        ps, P, np_, fan = c["ps"], c["P"], c["parents"], c["fan"]
        lens = _branch_lengths(c)
        nc = np_ * fan
        N = np_ + nc
        width = -(-(max(lens) + c["draft"]) // ps) + 1
        # the parents' pages lie scattered over the lower part of the pool; the children are empty
        need = [-(-x // ps) for x in lens]
        assert sum(need) + nc * (2 + c["draft"] // ps) <= P
        pages = list(range(min(P, 2 * sum(need))))
        host.shuffle(pages)
        table = torch.full((N, width), -1, dtype=torch.int32)
        refs = torch.zeros(P, dtype=torch.int32)
        slots = list(range(N))
        host.shuffle(slots)
        lengths = torch.zeros(N, dtype=torch.int32)
        at = 0
        for i, m in enumerate(need):
            own_pages = torch.tensor(pages[at:at + m], dtype=torch.long)
            table[slots[i], :m] = own_pages.to(torch.int32)
            refs[own_pages] = 1
            lengths[slots[i]] = lens[i]
            at += m
        parents = [slots[i // fan] for i in range(nc)]
        dev = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
        return dict(c=c, pool=normal(c["layers"], 2, P, c["Hk"], ps, c["D"], dtype=torch.bfloat16),
                    states=normal(c["layers"], N, c["H"], 128, 128, std=0.1), refs=refs.to(DEV), table=table.to(DEV),
                    lens=lengths.to(DEV), parents=dev(parents), children=dev(slots[np_:]),
                    draft=torch.full((nc,), c["draft"], dtype=torch.int32, device=DEV))
    P, N = c["P"], c["N"]
    shape = random.Random(c["mix"])
    alive = shape.sample(range(P), max(1, int(c["live"] * P)))
    host.shuffle(alive)
    refs = torch.zeros(P, dtype=torch.int32)
    rows = [[] for _ in range(N)]
    for i, p in enumerate(alive):
        n = 1 + (shape.random() < 0.1)  # some pages are shared by two sequences
        refs[p] = n
        for j in range(n):
            rows[(i + j) % N].append(p)
    table = torch.full((N, max(len(r) for r in rows) + 2), -1, dtype=torch.int32)
    for n, r in enumerate(rows):
        table[n, :len(r)] = torch.tensor(r, dtype=torch.int32)
    return dict(c=c, pool=normal(c["layers"], 2, P, c["Hk"], c["ps"], c["D"], dtype=torch.bfloat16), refs=refs.to(DEV),
                table=table.to(DEV), new_refs=torch.empty(P, dtype=torch.int32, device=DEV),
                new_table=torch.empty(table.shape, dtype=torch.int32, device=DEV))


def _branch_lengths(c):
    rng = random.Random(c["mix"])
    room = (c["P"] - c["parents"] * c["fan"] * (2 + c["draft"] // c["ps"])) // (2 * c["parents"]) * c["ps"]
    return [max(1, min(room, max(c["ctx_lo"], _spread(rng, c["ctx_lo"], c["ctx_hi"])))) for _ in range(c["parents"])]


# ---------------------------------------------------------------------------------------- the passes
def run(state):
    return {"rope": _rope, "append": _append, "attn": _attn, "branch": _branch, "compact": _compact}[state["c"]["kind"]](state)


def _rotate(x, pos, inv_freq, inter, scale, sign):
    """Rotary positions of x [T, H, D] at pos [T]: angles in 64 bits, products in 32, one rounding."""
    R = 2 * inv_freq.numel()
    a = pos.double()[:, None] * inv_freq
    cos, sin = (scale * a.cos()).float()[:, None], (sign * scale * a.sin()).float()[:, None]
    y = x.float()
    x1, x2 = (y[..., 0:R:2], y[..., 1:R:2]) if inter else (y[..., :R // 2], y[..., R // 2:R])
    y1, y2 = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    rot = torch.stack((y1, y2), -1).flatten(-2) if inter else torch.cat((y1, y2), -1)
    return torch.cat((rot, y[..., R:]), -1).to(x.dtype)


def _rope(s):
    c = s["c"]
    if own:
        kda = _kda()
        q, k = kda.rope(s["q"], s["k"], s["pos"], s["inv_freq"], interleaved=c["inter"], scale=s["scale"])
        dq, dk = kda.rope_bwd(s["dq"], s["dk"], s["pos"], s["inv_freq"], interleaved=c["inter"], scale=s["scale"])
        return q, k, dq, dk
    args = (s["pos"], s["inv_freq"], c["inter"], s["scale"])
    return (_rotate(s["q"], *args, 1), _rotate(s["k"], *args, 1), _rotate(s["dq"], *args, -1), _rotate(s["dk"], *args, -1))


def _append(s):
    c = s["c"]
    if own:
        q = _kda().cache_append(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["lens"],
                                cu_seqlens=None if s["one"] else s["cu"], q=s["q"], inv_freq=s["inv_freq"],
                                interleaved=c["inter"])
        return q, s["kc"], s["vc"]
    t = torch.arange(s["k"].shape[0], device=DEV)
    n = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    pos = (s["lens"][n] - s["cu"][n + 1]) + t
    page, row = s["table"][n, pos // c["ps"]].long(), pos % c["ps"]
    s["kc"][page, :, row] = _rotate(s["k"], pos, s["inv_freq"], c["inter"], 1.0, 1)
    s["vc"][page, :, row] = s["v"]
    return _rotate(s["q"], pos, s["inv_freq"], c["inter"], 1.0, 1), s["kc"], s["vc"]


def _attn(s):
    c = s["c"]
    if own:
        return _kda().attn_paged(s["q"], s["kc"], s["vc"], s["table"], s["lens"],
                                 cu_seqlens=None if s["one"] else s["cu"], window=c["window"])
    N, Hk, D, m = c["N"], c["Hk"], c["D"], s["most"]
    G, L = c["Hq"] // Hk, s["table"].shape[1] * c["ps"]
    t = torch.arange(s["q"].shape[0], device=DEV)
    n = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    i = t - s["cu"][n]
    q = torch.zeros((N, m, c["Hq"], D), dtype=torch.float32, device=DEV)
    q[n, i] = s["q"].float() * D ** -0.5
    q = q.view(N, m, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(N, Hk, G * m, D)
    at = s["table"].clamp(min=0).long()
    k = s["kc"][at].permute(0, 2, 4, 1, 3).reshape(N, Hk, D, L).float()
    p = torch.matmul(q, k).view(N, Hk, G, m, L)
    pos = (s["lens"] - (s["cu"][1:] - s["cu"][:-1]))[:, None] + torch.arange(m, device=DEV)
    key = torch.arange(L, device=DEV)
    seen = key <= pos[..., None]
    if c["window"]:
        seen &= key > pos[..., None] - c["window"]
    p.masked_fill_(~seen[:, None, None], float("-inf"))
    p.sub_(p.amax(-1, keepdim=True)).exp_()
    p.div_(p.sum(-1, keepdim=True))
    v = s["vc"][at].permute(0, 2, 1, 3, 4).reshape(N, Hk, L, D).float()
    v.masked_fill_((key >= s["lens"][:, None])[:, None, :, None], 0.0)
    o = torch.matmul(p.view(N, Hk, G * m, L), v).view(N, Hk, G, m, D).permute(0, 3, 1, 2, 4).reshape(N, m, c["Hq"], D)
    return o[n, i].to(s["q"].dtype)


def _take(refs, need):
    """The lowest free pages for requests of `need` pages each, in order: (granted, the rank of each request's first page, free pages in order)."""
    end = need.cumsum(0)
    order = torch.sort((refs > 0).to(torch.int8), stable=True).indices
    granted = (need == 0) | (end <= (refs == 0).sum())
    return granted, end - need, order


def _branch(s):
    c, refs, table, lens = s["c"], s["refs"], s["table"], s["lens"]
    par, chi, ps = s["parents"], s["children"], c["ps"]
    if own:
        kda = _kda()
        kda.pages_free(refs, table, lens, chi, ps)
        forked = kda.pages_fork(s["pool"], refs, table, lens, par, chi, ps, page_dim=2)
        grown = kda.pages_alloc(refs, table, lens, s["draft"], ps, seqs=chi)
        kda.pages_copy(s["states"], par, chi, page_dim=1)
        return forked, grown, refs, table, lens, s["pool"], s["states"]
    par, chi = par.long(), chi.long()
    col = torch.arange(table.shape[1], device=DEV)
    # the old branches go
    held = (col < ((lens[chi] + ps - 1) // ps)[:, None]) & (table[chi] >= 0)
    refs.index_add_(0, table[chi].clamp(min=0).long().flatten(), -held.flatten().int())
    table[chi] = torch.where(held, -1, table[chi])
    lens[chi] = 0
    # new ones share the parents' full pages and get a copy of the page that is not full
    part = lens[par] % ps != 0
    granted, first, order = _take(refs, part.int())
    full = (lens[par] // ps)[:, None]
    page = order[first].int()
    got, src = part & granted, table[par].gather(1, full.long().clamp(max=table.shape[1] - 1))[:, 0].clamp(min=0).long()
    shared = (col < full) & granted[:, None]
    row = torch.where(shared, table[par], torch.where((col == full) & got[:, None], page[:, None], table[chi]))
    refs.index_add_(0, row.clamp(min=0).long().flatten(), (shared | ((col == full) & got[:, None])).flatten().int())
    table[chi] = row
    lens[chi] = torch.where(granted, lens[par], 0)
    s["pool"][:, :, page[got].long()] = s["pool"][:, :, src[got]]
    # room for the draft tokens
    have, want = (lens[chi] + ps - 1) // ps, (lens[chi] + s["draft"] + ps - 1) // ps
    grown, first, order = _take(refs, want - have)
    grown &= want <= table.shape[1]
    new = (col >= have[:, None]) & (col < want[:, None]) & grown[:, None]
    page = order[(first[:, None] + col - have[:, None]).clamp(0, c["P"] - 1).long()].int()
    table[chi] = torch.where(new, page, table[chi])
    refs.index_add_(0, page.long().flatten(), new.flatten().int())
    lens[chi] += torch.where(grown, s["draft"], 0)
    s["states"][:, chi] = s["states"][:, par]
    return granted.int(), grown.int(), refs, table, lens, s["pool"], s["states"]


def _compact(s):
    refs, table = s["refs"], s["table"]
    if own:
        moved = _kda().pages_compact(s["pool"], refs, table, page_dim=2, out_refs=s["new_refs"], out_table=s["new_table"])
        return moved, s["new_refs"], s["new_table"], s["pool"]
    P, live = refs.numel(), refs > 0
    at = torch.arange(P, device=DEV)
    n = live.sum()
    holes = (~live & (at < n)).nonzero()[:, 0]
    movers = (live & (at >= n)).nonzero()[:, 0].flip(0)
    to = at.clone()
    to[movers] = holes
    s["new_refs"].zero_()
    s["new_refs"].index_put_((to[live],), refs[live])
    s["new_table"].copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].int(), table))
    s["pool"][:, :, holes] = s["pool"][:, :, movers]
    return torch.full((1,), holes.numel(), dtype=torch.int32, device=DEV), s["new_refs"], s["new_table"], s["pool"]


# ---------------------------------------------------------------------------------------- work
def work(case):
    c = case
    if c["kind"] == "rope":
        e = 2 if c["dtype"] == "bf16" else 4
        n = c["T"] * (c["Hq"] + c["Hk"]) * c["D"]
        return {"bytes": 4 * n * e + 8 * c["T"], "flops": 12 * c["T"] * (c["Hq"] + c["Hk"]) * c["R"] // 2}
    if c["kind"] in ("append", "attn"):
        e = 2 if c["dtype"] == "bf16" else 4
        new, lens = _lengths(c)
        T, D, Hq, Hk = sum(new), c["D"], c["Hq"], c["Hk"]
        if c["kind"] == "append":
            return {"bytes": 2 * T * (Hq + 2 * Hk) * D * e, "flops": 6 * T * (Hq + Hk) * c["R"] // 2}
        w = c["window"] or 1 << 40
        keys = sum(L - max(0, L - m + 1 - w) for m, L in zip(new, lens))
        pairs = sum(min(p + 1, w) for m, L in zip(new, lens) for p in range(L - m, L))
        return {"bytes": 2 * T * Hq * D * e + 2 * keys * Hk * D * e, "flops": 4 * pairs * Hq * D}
    page = 2 * c["layers"] * c["Hk"] * c["ps"] * c["D"] * 2
    if c["kind"] == "branch":
        lens, nc = _branch_lengths(c), c["parents"] * c["fan"]
        part = sum(x % c["ps"] != 0 for x in lens) * c["fan"]
        state = c["layers"] * c["H"] * 128 * 128 * 4
        rows = sum(-(-x // c["ps"]) for x in lens) * c["fan"]
        return {"bytes": 2 * part * page + 2 * nc * state + 4 * (2 * rows + c["P"]), "flops": 0}
    alive = random.Random(c["mix"]).sample(range(c["P"]), max(1, int(c["live"] * c["P"])))
    moves = sum(p >= len(alive) for p in alive)
    return {"bytes": 2 * moves * page + 8 * c["P"] + 8 * len(alive), "flops": 0}


# ---------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The operators' definitions, sequence by sequence, in 64 bits; whole numbers by counting."""
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "attn": _exact_attn, "branch": _exact_branch,
            "compact": _exact_compact}[case["kind"]](s)


def _turned(x, pos, s, sign, scale):
    """x as complex numbers times scale e^(i sign pos f)."""
    f = s["inv_freq"]
    R = 2 * f.numel()
    y = x.double().clone()
    z = torch.view_as_complex(y[..., :R].unflatten(-1, (R // 2, 2)).contiguous()) if s["c"]["inter"] else \
        torch.complex(y[..., :R // 2], y[..., R // 2:R])
    z = z * (scale * torch.polar(torch.ones_like(f), sign * pos.double()[:, None] * f))[:, None]
    if s["c"]["inter"]:
        y[..., 0:R:2], y[..., 1:R:2] = z.real, z.imag
    else:
        y[..., :R // 2], y[..., R // 2:R] = z.real, z.imag
    return y


def _exact_rope(s):
    return tuple(_turned(s[n], s["pos"], s, sign, s["scale"]) for n, sign in (("q", 1), ("k", 1), ("dq", -1), ("dk", -1)))


def _exact_append(s):
    c = s["c"]
    new, lens = _lengths(c)
    cu, ps = _cu(new), c["ps"]
    kc, vc, table = s["kc"].double(), s["vc"].double(), s["table"].cpu().tolist()
    qs = []
    for n, (m, L) in enumerate(zip(new, lens)):
        a, e = cu[n], cu[n + 1]
        pos = torch.arange(L - m, L, device=DEV)
        qs.append(_turned(s["q"][a:e], pos, s, 1, 1.0))
        k, v = _turned(s["k"][a:e], pos, s, 1, 1.0), s["v"][a:e].double()
        for j in range((L - m) // ps, -(-L // ps)):
            lo, hi = max(L - m, j * ps), min(L, (j + 1) * ps)
            kc[table[n][j], :, lo - j * ps:hi - j * ps] = k[lo - (L - m):hi - (L - m)].transpose(0, 1)
            vc[table[n][j], :, lo - j * ps:hi - j * ps] = v[lo - (L - m):hi - (L - m)].transpose(0, 1)
    return torch.cat(qs), kc, vc


def _exact_attn(s):
    c = s["c"]
    new, lens = _lengths(c)
    cu, G, D = _cu(new), c["Hq"] // c["Hk"], c["D"]
    o = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    for n, (m, L) in enumerate(zip(new, lens)):
        pages = s["table"][n, :-(-L // c["ps"])].long()
        first = 0 if not c["window"] else max(0, L - m + 1 - c["window"])
        pos = torch.arange(L - m, L, device=DEV)[:, None]
        key = torch.arange(first, L, device=DEV)[None]
        hidden = (key > pos) | (key <= pos - (c["window"] or 1 << 40))
        for h in range(c["Hk"]):
            k = s["kc"][pages, h].double().flatten(0, 1)[first:L]
            v = s["vc"][pages, h].double().flatten(0, 1)[first:L]
            for g in range(G):
                x = s["q"][cu[n]:cu[n + 1], h * G + g].double() @ k.t().contiguous() / math.sqrt(D)
                o[cu[n]:cu[n + 1], h * G + g] = torch.softmax(x.masked_fill_(hidden, float("-inf")), -1) @ v
    return o


def _exact_branch(s):
    c = s["c"]
    ps = c["ps"]
    refs, table, lens = s["refs"].cpu().tolist(), s["table"].cpu().tolist(), s["lens"].cpu().tolist()
    pool, states = s["pool"], s["states"].double()
    pairs = list(zip(s["parents"].cpu().tolist(), s["children"].cpu().tolist()))

    def lowest():
        for p, r in enumerate(refs):
            if r == 0:
                refs[p] = 1
                return p

    for a, b in pairs:  # prepared states have empty children: nothing to free
        full = lens[a] // ps
        for j in range(full):
            table[b][j] = table[a][j]
            refs[table[a][j]] += 1
        if lens[a] % ps:
            table[b][full] = lowest()
            pool[:, :, table[b][full]] = pool[:, :, table[a][full]]
        lens[b] = lens[a]
    for _, b in pairs:
        for j in range(-(-lens[b] // ps), -(-(lens[b] + c["draft"]) // ps)):
            table[b][j] = lowest()
        lens[b] += c["draft"]
    for a, b in pairs:
        states[:, b] = states[:, a]
    one = torch.ones(len(pairs), dtype=torch.int32)
    whole = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return one, one.clone(), whole(refs), whole(table), whole(lens), pool.double(), states


def _exact_compact(s):
    refs, table = s["refs"].cpu().tolist(), s["table"].cpu().tolist()
    pool, to, moved = s["pool"].double(), {}, 0
    low, high = 0, len(refs) - 1
    while True:
        while low < len(refs) and refs[low] > 0:
            low += 1
        while high >= 0 and refs[high] == 0:
            high -= 1
        if low > high:
            break
        refs[low], refs[high] = refs[high], 0
        to[high] = low
        moved += 1
    if to:
        pool[:, :, list(to.values())] = pool[:, :, list(to.keys())]
    whole = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return whole([moved]), whole(refs), whole([[to.get(p, p) for p in row] for row in table]), pool
