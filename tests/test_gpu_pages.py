"""Page bookkeeping and copies on the GPU against plain lists, and a run of the serving operators
together: prompts, decoding, a fork, its branches, freeing and compaction."""
import random

import pytest
import torch

import gated_delta_rule_30_amd as kda
import paged_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Both:
    """The state on the GPU and its plain form, compared after every call."""

    def __init__(self, P, N, width, ps, page=(2, 16), planes=(), dtype=torch.float32, seed=0):
        gen = torch.Generator().manual_seed(seed)
        pool = torch.randn(tuple(planes) + (P,) + tuple(page), generator=gen).to(dtype)
        self.dim = len(planes)
        self.host = ref.Pages([0] * P, [[-1] * width for _ in range(N)], [0] * N, ps, [pool], self.dim)
        self.pool = pool.to(DEV)
        self.refs, self.table, self.lens = ints([0] * P), ints([[-1] * width] * N), ints([0] * N)
        self.ps = ps

    def same(self):
        assert self.refs.tolist() == self.host.refs
        assert self.table.tolist() == self.host.table
        assert self.lens.tolist() == self.host.lens
        assert torch.equal(self.pool.cpu(), self.host.pools[0])

    def alloc(self, seqs, new):
        if seqs is None:
            got = kda.pages_alloc(self.refs, self.table, self.lens, ints(new), self.ps)
            seqs = range(len(new))
        else:
            got = kda.pages_alloc(self.refs, self.table, self.lens, ints(new), self.ps, seqs=ints(seqs))
        assert got.tolist() == self.host.alloc(list(seqs), new)
        self.same()

    def fork(self, parents, children):
        got = kda.pages_fork(self.pool, self.refs, self.table, self.lens, ints(parents), ints(children), self.ps,
                             page_dim=self.dim)
        assert got.tolist() == self.host.fork(parents, children)
        self.same()

    def free(self, seqs):
        kda.pages_free(self.refs, self.table, self.lens, ints(seqs), self.ps)
        self.host.free(seqs)
        self.same()

    def compact(self):
        moved = kda.pages_compact(self.pool, self.refs, self.table, page_dim=self.dim)
        assert moved.item() == self.host.compact()
        self.same()


def test_alloc_in_order():
    b = Both(20, 5, 8, 16)
    b.alloc(None, [1, 16, 17, 0, 33])
    b.alloc([4, 0, 2], [15, 15, 16])
    b.alloc([1, 3], [100, 128])      # 3 is too long for what is left after 1
    b.alloc([3, 0], [200, 0])        # a row that is too short; no page needed
    b.alloc([0, 0, 7, -1, 2], [1, 1, 5, 5, -1])  # twice, no such sequences, a negative count


def test_refusals_take_nothing():
    """A request that does not fit keeps its place in the order: none after it that needs a page is
    served, one that needs none is."""
    b = Both(4, 4, 8, 16)
    b.alloc([0], [20])
    b.alloc([1, 2, 0, 3], [48, 1, 5, 1])
    b.alloc([2, 3], [16, 16])
    b.alloc([1], [1])
    b.free([0, 2])
    b.alloc([1, 0], [2 ** 31 - 1, 30])


@pytest.mark.parametrize("planes,page", [((), (16,)), ((3,), (2, 4)), ((2, 2), (5000,))])
def test_fork_shares_and_copies(planes, page):
    b = Both(40, 10, 6, 16, page=page, planes=planes)
    b.alloc([0, 1, 2], [40, 32, 5])
    b.fork([0, 0, 1, 2], [3, 4, 5, 6])
    b.fork([3], [7])                       # a fork of a fork
    b.alloc([0, 3, 4], [1, 20, 30])        # each goes on in its own page
    b.free([0])
    b.free([3, 3, 4, -2, 99])              # twice, none
    b.fork([5, 6, 8, 0], [0, 0, 3, 8])     # a child twice; an empty parent; a parent that is a child here
    b.fork([5, 99, 5], [1, 4, -1])         # a child that is not empty; no such sequences
    b.compact()


def test_fork_without_room():
    b = Both(6, 6, 4, 16)
    b.alloc([0, 1], [40, 32])              # 5 pages
    b.fork([0, 0, 1, 0], [2, 3, 4, 5])     # one copy fits; sharing alone always does
    b.free([0, 1, 2, 3, 4, 5])
    assert not any(b.host.refs)


def test_fork_bookkeeping_alone():
    b = Both(8, 3, 4, 16)
    b.alloc([0], [20])
    want = ref.Pages(b.host.refs, b.host.table, b.host.lens, 16)
    want.fork([0], [2])
    kda.pages_fork(None, b.refs, b.table, b.lens, ints([0]), ints([2]), 16)
    assert b.refs.tolist() == want.refs and b.table.tolist() == want.table and b.lens.tolist() == want.lens
    assert torch.equal(b.pool.cpu(), b.host.pools[0])


@pytest.mark.parametrize("P", [1, 63, 4096, 4097, 20000])
def test_random_life(P):
    """Many rounds of every call, over one and several blocks of pages."""
    rng = random.Random(P)
    N, width, ps = 24, 12 if P < 4096 else 400, 16
    b = Both(P, N, width, ps, page=(4,), seed=P)
    for _ in range(12):
        seqs = rng.sample(range(N), rng.randrange(1, N))
        b.alloc(seqs, [rng.randrange(0, width * ps // 3) for _ in seqs])
        empty = [n for n in range(N) if b.host.lens[n] == 0]
        if empty:
            kids = rng.sample(empty, rng.randrange(1, len(empty) + 1))
            b.fork([rng.randrange(N) for _ in kids], kids)
        b.free(rng.sample(range(N), rng.randrange(0, N // 2)) or [0])
        if rng.random() < 0.5:
            b.compact()


def test_many_requests():
    """More requests than the planning workgroup has threads."""
    N = 2500
    b = Both(6000, N, 4, 16, page=(4,))
    rng = random.Random(3)
    b.alloc(None, [rng.randrange(0, 40) for _ in range(N)])
    b.free(list(range(0, N, 3)))
    b.fork([rng.randrange(N) for _ in range(0, N, 3)], list(range(0, N, 3)))
    b.compact()


def test_needs_past_32_bits():
    """1024 requests of 2^21 pages each pass 32 bits together; none fits, and neither does what follows them."""
    N, width, ps, P = 1026, 1 << 21, 16, 64
    table = torch.empty((N, width), dtype=torch.int32, device=DEV)
    refs, lens = ints([0] * P), ints([0] * N)
    new = [width * ps] * 1024 + [1, 0]
    got = kda.pages_alloc(refs, table, lens, ints(new), ps)
    assert got.tolist() == [0] * 1025 + [1]
    assert refs.tolist() == [0] * P and lens.tolist() == [0] * N


def test_entries_outside_the_pool():
    """Entries that name no page are passed over by fork, free and compact."""
    b = Both(12, 4, 4, 16)
    b.alloc([0, 1], [50, 20])
    for j, p in ((1, -5), (3, 4000)):
        b.table[0, j] = p
        b.host.table[0][j] = p
    b.fork([0], [2])
    b.free([0])
    b.compact()


def test_compact_out_of_place():
    b = Both(50, 6, 8, 16)
    b.alloc(None, [40, 100, 7, 64, 30, 90])
    b.free([0, 3, 4])
    refs, table, keep = b.refs.clone(), b.table.clone(), torch.empty_like(b.refs)
    wide = torch.full((6, 11), 5, dtype=torch.int32, device=DEV)
    out = wide[:, 2:10]
    moved = kda.pages_compact(b.pool, b.refs, b.table, out_refs=keep, out_table=out)
    assert torch.equal(b.refs, refs) and torch.equal(b.table, table)
    assert moved.item() == b.host.compact()
    assert keep.tolist() == b.host.refs and out.tolist() == b.host.table
    assert torch.all(wide[:, :2] == 5) and torch.all(wide[:, 10:] == 5)
    assert torch.equal(b.pool.cpu(), b.host.pools[0])


@pytest.mark.parametrize("full", [False, True])
def test_compact_nothing_to_do(full):
    b = Both(4, 1, 4, 16)
    if full:
        b.alloc([0], [64])
    b.compact()


def test_copy():
    """Copies in pools of different types, planes and strides; pairs without a page or onto themselves are passed
    over."""
    gen = torch.Generator().manual_seed(1)
    a = torch.randn((3, 10, 2, 128, 128), generator=gen)
    b = torch.randn((10, 3, 8), generator=gen).bfloat16()[:, 1]
    c = torch.randint(0, 100, (10, 4), generator=gen, dtype=torch.int32)
    da, db, dc = a.to(DEV), torch.zeros((10, 3, 8), dtype=torch.bfloat16, device=DEV), c.to(DEV)
    db[:, 1] = b.to(DEV)
    src, dst = [0, 3, 5, 9, 11, -1, 2], [1, 4, 5, 8, 2, 6, 7]
    kda.pages_copy(da, ints(src), ints(dst), page_dim=1)
    kda.pages_copy([db[:, 1], dc], ints(src), ints(dst))
    for s, t in zip(src, dst):
        if 0 <= s < 10 and 0 <= t < 10:
            a[:, t], b[t], c[t] = a[:, s].clone(), b[s].clone(), c[s].clone()
    assert torch.equal(da.cpu(), a) and torch.equal(db[:, 1].cpu(), b) and torch.equal(dc.cpu(), c)
    assert not db[:, 0].any() and not db[:, 2].any()
    kda.pages_copy(da, ints([]), ints([]), page_dim=1)


def test_graph_replay():
    """Free, fork and alloc of a branching step, captured and replayed."""
    b = Both(64, 8, 8, 16, planes=(2,))
    b.alloc([0, 1], [40, 70])
    par, kids, more = ints([0, 0, 1]), ints([2, 3, 4]), ints([5, 30, 1])
    granted = ints([0, 0, 0])
    ws = torch.empty(int(kda.lib().kda_pages_plan_workspace_size(3, 8, 64)), dtype=torch.uint8, device=DEV)
    grown = torch.zeros_like(granted)

    def step():
        kda.pages_free(b.refs, b.table, b.lens, kids, 16)
        kda.pages_fork(b.pool, b.refs, b.table, b.lens, par, kids, 16, page_dim=1, granted=granted, workspace=ws)
        kda.pages_alloc(b.refs, b.table, b.lens, more, 16, seqs=kids, granted=grown, workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()

    def host():
        b.host.free([2, 3, 4])
        assert b.host.fork(par.tolist(), [2, 3, 4]) == granted.tolist()
        assert b.host.alloc([2, 3, 4], more.tolist()) == grown.tolist()
        b.same()

    host()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for rep in range(3):
        par.copy_(ints([[1, 0, 1], [2, 0, 0], [1, 1, 1]][rep]))
        more.copy_(ints([rep, 40, 17]))
        ws.fill_(255)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        host()


def test_serving_run():
    """Two prompts in chunks, decode steps, a fork with diverging branches, a sequence freed,
    the pool compacted, more decode steps: after each attention call the result equals attention over
    every sequence's own tokens, kept on the host, and each sequence's KDA state goes along."""
    dtype, Hq, Hk, D, ps, P, N, W = torch.bfloat16, 8, 2, 64, 16, 60, 6, 20
    H, K = 2, 32
    pool = torch.zeros((2, P, Hk, ps, D), dtype=dtype, device=DEV)
    states = torch.zeros((N, H, K, K), device=DEV)
    refs, table, lens = ints([0] * P), ints([[-1] * W] * N), ints([0] * N)
    f, _ = kda.rope_freqs(D, device=DEV)
    host_k, host_v = [[] for _ in range(N)], [[] for _ in range(N)]
    host_s = [torch.zeros((H, K, K), dtype=torch.float64) for _ in range(N)]
    gen = torch.Generator(device=DEV).manual_seed(2)

    def tokens(new):
        """A model step: new[n] tokens of every sequence through both kinds of layers."""
        cu = [0]
        for m in new:
            cu.append(cu[-1] + m)
        T = cu[-1]
        assert kda.pages_alloc(refs, table, lens, ints(new), ps).tolist() == [1] * N
        qkv = torch.randn((T, Hq + 2 * Hk, D), generator=gen, device=DEV).to(dtype)
        q = kda.cache_append(qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:], pool[0], pool[1], table, lens,
                             cu_seqlens=ints(cu), q=qkv[:, :Hq], inv_freq=f)
        o = kda.attn_paged(q, pool[0], pool[1], table, lens, cu_seqlens=ints(cu))
        pos = torch.cat([torch.arange(int(lens[n]) - new[n], int(lens[n])) for n in range(N)]).to(DEV).int()
        k, _ = kda.rope(qkv[:, Hq:Hq + Hk], None, pos, f)
        for n in range(N):
            host_k[n] += list(k[cu[n]:cu[n + 1]].cpu())
            host_v[n] += list(qkv[cu[n]:cu[n + 1], Hq + Hk:].cpu())
        # the same tokens stored densely, one sequence after the other
        seqs = [n for n in range(N) if new[n]]
        need = [-(-len(host_k[n]) // ps) for n in seqs]
        kc, vc = (torch.zeros((sum(need), Hk, ps, D), dtype=dtype) for _ in range(2))
        tab, at = torch.full((len(seqs), max(need)), -1, dtype=torch.int32), 0
        for i, n in enumerate(seqs):
            for j in range(need[i]):
                tab[i, j] = at
                for r in range(j * ps, min((j + 1) * ps, len(host_k[n]))):
                    kc[at, :, r - j * ps], vc[at, :, r - j * ps] = host_k[n][r], host_v[n][r]
                at += 1
        L = torch.tensor([len(host_k[n]) for n in seqs])
        assert L.tolist() == [int(lens[n]) for n in seqs]
        want, _, tol, _ = ref.attention(q.cpu(), kc, vc, tab, L, [0] + [cu[n + 1] for n in seqs], D ** -0.5, 0)
        assert torch.all((o.double().cpu() - want).abs() <= tol)
        # the KDA side, one token per sequence of this step
        x = torch.randn((4, N, H, K), generator=gen, device=DEV)
        beta = torch.rand((N, H), generator=gen, device=DEV)
        la = -torch.rand((N, H, K), generator=gen, device=DEV) * 0.1
        kk = x[1] / x[1].norm(dim=-1, keepdim=True)
        kda.decode_step(x[0], kk, x[2], la, beta, state=states)
        for n in range(N):
            s, key = host_s[n], kk[n].double().cpu()
            s = s * la[n].double().cpu().exp()[:, :, None]
            u = torch.einsum("hkv,hk->hv", s, key)
            host_s[n] = s + torch.einsum("hk,hv->hkv", key * beta[n].double().cpu()[:, None],
                                         x[2, n].double().cpu() - u)
        assert torch.allclose(states.double().cpu(), torch.stack(host_s), atol=1e-4)

    def fork(par, kids):
        assert kda.pages_fork(pool, refs, table, lens, ints(par), ints(kids), ps, page_dim=1).tolist() == [1] * len(kids)
        kda.pages_copy(states, ints(par), ints(kids))
        for a, b in zip(par, kids):
            host_k[b], host_v[b], host_s[b] = list(host_k[a]), list(host_v[a]), host_s[a].clone()

    tokens([37, 0, 100, 0, 0, 0])
    tokens([1, 0, 20, 0, 0, 0])
    fork([0, 0, 2], [1, 3, 4])
    tokens([1, 1, 1, 5, 1, 0])
    kda.pages_free(refs, table, lens, ints([0]), ps)
    host_k[0], host_v[0] = [], []
    kda.pages_compact(pool, refs, table, page_dim=1)
    live = int((refs > 0).sum())
    assert torch.all(refs[:live] > 0) and torch.all(refs[live:] == 0)
    tokens([0, 1, 1, 1, 1, 17])
    fork([3], [0])
    tokens([2, 1, 1, 1, 3, 1])
