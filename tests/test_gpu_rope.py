"""Rotary positions on the GPU against the fp64 form: layouts, part of the head, scaling, far and
negative positions, strided and in-place rows, gradients."""
import math

import numpy as np
import pytest
import torch

import gated_delta_rule_30_amd as kda
import paged_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _f64(t):
    return t.detach().double().cpu().numpy()


def _check(got, x, pos, inv_freq, inter, scale, inverse=False):
    y, size = ref.rope(_f64(x), pos.cpu().numpy(), inv_freq.cpu().numpy(), inter, scale, inverse)
    err = np.abs(_f64(got) - y) - ref.rope_tol(y, size, scale, x.dtype)
    assert err.size == 0 or err.max() <= 0, "beyond the tolerance by %.3e" % err.max()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,R", [(1, 1, 1, 16, 16), (5, 3, 1, 64, 32), (33, 8, 2, 128, 128),
                                         (7, 2, 2, 256, 64), (4100, 2, 1, 48, 32), (2, 1, 5, 512, 512)])
def test_rope(T, Hq, Hk, D, R, inter, dtype):
    gen = torch.Generator(device=DEV).manual_seed(T + D)
    q = torch.randn((T, Hq, D), generator=gen, device=DEV).to(dtype)
    k = torch.randn((T, Hk, D), generator=gen, device=DEV).to(dtype)
    pos = torch.randint(-50, 1 << 20, (T,), generator=gen, device=DEV, dtype=torch.int32)
    for scaling, factor in ((None, 1.0), ("yarn", 8.0)):
        f, scale = kda.rope_freqs(R, 500000.0, scaling, factor, device=DEV)
        qo, ko = kda.rope(q, k, pos, f, interleaved=inter, scale=scale)
        _check(qo, q, pos, f, inter, scale)
        _check(ko, k, pos, f, inter, scale)
        dq, dk = kda.rope_bwd(q, k, pos, f, interleaved=inter, scale=scale)
        _check(dq, q, pos, f, inter, scale, inverse=True)
        _check(dk, k, pos, f, inter, scale, inverse=True)


def test_extreme_positions():
    """The ends of int32, where one double for the angle would no longer do."""
    pos = torch.tensor([0, 1, -1, 2**31 - 1, -2**31, 2**31 - 12345, 10**9], dtype=torch.int32, device=DEV)
    x = torch.randn((7, 2, 64), device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    f, _ = kda.rope_freqs(64, device=DEV)
    y, none = kda.rope(x, None, pos, f)
    assert none is None
    _check(y, x, pos, f, False, 1.0)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_strided_and_in_place(inter):
    T, Hq, Hk, D = 37, 4, 2, 128
    gen = torch.Generator(device=DEV).manual_seed(3)
    qkv = torch.randn((T, Hq + 2 * Hk, D), generator=gen, device=DEV).bfloat16()
    pos = torch.arange(T, dtype=torch.int32, device=DEV) * 97
    f, _ = kda.rope_freqs(64, device=DEV)
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    want = kda.rope(q.contiguous(), k.contiguous(), pos, f, interleaved=inter)
    got = kda.rope(q, k, pos, f, interleaved=inter)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    v = qkv[:, Hq + Hk:].clone()
    kda.rope(q, k, pos, f, interleaved=inter, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(qkv[:, Hq + Hk:], v)
    only, _ = kda.rope(want[0], None, pos, f, interleaved=inter)
    none, ko = kda.rope(None, want[1], pos, f, interleaved=inter)
    both = kda.rope(want[0], want[1], pos, f, interleaved=inter)
    assert none is None and torch.equal(only, both[0]) and torch.equal(ko, both[1])


def test_empty():
    f, _ = kda.rope_freqs(16, device=DEV)
    q = torch.empty((0, 2, 16), device=DEV)
    a, b = kda.rope(q, None, torch.empty(0, dtype=torch.int32, device=DEV), f)
    assert a.shape == q.shape and b is None


def test_gradient_by_differences():
    """sum(w * rope(x)) changes along a direction as the gradient says; rope is linear, so a
    difference of any step is exact but for the fp32 of the two outputs."""
    gen = torch.Generator(device=DEV).manual_seed(5)
    x, w, d = (torch.randn((9, 3, 64), generator=gen, device=DEV) for _ in range(3))
    pos = torch.randint(0, 5000, (9,), generator=gen, device=DEV, dtype=torch.int32)
    f, scale = kda.rope_freqs(32, scaling="yarn", factor=4.0, device=DEV)
    for inter in (False, True):
        go, _ = kda.rope_bwd(w, None, pos, f, interleaved=inter, scale=scale)
        hi, _ = kda.rope(x + d, None, pos, f, interleaved=inter, scale=scale)
        lo, _ = kda.rope(x - d, None, pos, f, interleaved=inter, scale=scale)
        num = ((hi.double() - lo.double()) * w.double()).sum().item() / 2
        ana = (go.double() * d.double()).sum().item()
        # per element: 2^-21 of the sizes of x, d and their turned pair, on 1728 elements
        size = (w.double().abs() * (x.double().abs() + d.double().abs())).sum().item() * 2 * scale
        assert abs(num - ana) <= 2.0 ** -20 * size


def test_rope_into_the_delta_rule_and_back():
    """A training step: rope on q and k, chunk_fwd, chunk_bwd, rope_bwd; the gradients of the raw
    q and k against the oracle's, turned back in fp64."""
    import oracle
    import workloads
    T, H, K = 130, 2, 64
    inp = workloads.gen_forward(T, H, K, K, dtype=torch.float32, device=DEV, seed=4)
    pos = torch.arange(T, dtype=torch.int32, device=DEV) + 7
    f, _ = kda.rope_freqs(K, device=DEV)
    q, k = kda.rope(inp["q"], inp["k"], pos, f)
    kda.chunk_fwd(q, k, inp["v"], inp["log_alpha"], inp["beta"])
    d_o = torch.randn((T, H, K), device=DEV, generator=torch.Generator(device=DEV).manual_seed(6))
    g = kda.chunk_bwd(q, k, inp["v"], inp["log_alpha"], inp["beta"], d_o)
    dq, dk = kda.rope_bwd(g[0], g[1], pos, f)
    turned = [ref.rope(_f64(inp[n]), pos.cpu().numpy(), f.cpu().numpy(), False, 1.0)[0] for n in "qk"]
    want = oracle.kda_bwd(*turned, _f64(inp["v"]), _f64(inp["log_alpha"]), _f64(inp["beta"]), _f64(d_o))
    for got, w in ((dq, want[0]), (dk, want[1])):
        w = ref.rope(np.asarray(w), pos.cpu().numpy(), f.cpu().numpy(), False, 1.0, inverse=True)[0]
        assert np.abs(_f64(got) - w).max() <= 1e-4 * np.abs(w).max()  # the backward's own fp32 tolerance


def test_freqs():
    for R in (16, 128):
        i = np.arange(R // 2)
        base = 10000.0 ** (-2 * i / R)
        assert np.allclose(kda.rope_freqs(R)[0], base, rtol=1e-14)
        assert np.allclose(kda.rope_freqs(R, scaling="linear", factor=4.0)[0], base / 4, rtol=1e-14)
        ntk = kda.rope_freqs(R, scaling="ntk", factor=4.0)[0].numpy()
        assert abs(ntk[0] - 1) < 1e-14 and abs(ntk[-1] * 4 / base[-1] - 1) < 1e-12
        yarn, scale = kda.rope_freqs(R, scaling="yarn", factor=4.0, original_length=4096)
        turns = 4096 * base / (2 * math.pi)
        assert scale == 0.1 * math.log(4.0) + 1
        assert np.allclose(yarn.numpy()[turns > 64], base[turns > 64], rtol=1e-14)
        assert np.allclose(yarn.numpy()[turns < 0.5], base[turns < 0.5] / 4, rtol=1e-14)
        assert np.all(np.diff(yarn.numpy()) < 0)


def test_graph_replay():
    T = 64
    x = torch.randn((T, 4, 128), device=DEV).bfloat16()
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    f, _ = kda.rope_freqs(128, device=DEV)
    out = torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        kda.rope(x, None, pos, f, q_out=out)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.rope(x, None, pos, f, q_out=out)
    for rep in range(3):
        pos.add_(rep + 1)
        x.mul_(-1)
        want, _ = kda.rope(x, None, pos, f)
        out.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), rep


def test_more_tokens_than_one_grid_dimension():
    """2^24 tokens and a few: 2^32 threads and more. Equal bit for bit to calls on parts."""
    T, D = (1 << 24) + 5, 16
    f, _ = kda.rope_freqs(D, device=DEV)
    k = torch.randn((T, 1, D), device=DEV).bfloat16()
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    got = kda.rope(None, k, pos, f)[1]
    for a, b in ((0, 9), ((1 << 22) - 3, (1 << 22) + 3), (T - 9, T)):
        assert torch.equal(got[a:b], kda.rope(None, k[a:b], pos[a:b].contiguous(), f)[1])
    ps = 256
    P = -(-T // ps)
    cache = torch.zeros((2, P, 1, ps, D), dtype=torch.bfloat16, device=DEV)
    table = torch.arange(P, dtype=torch.int32, device=DEV).view(1, P)
    kda.cache_append(k, k, cache[0], cache[1], table, torch.tensor([T], dtype=torch.int32, device=DEV), inv_freq=f)
    assert torch.equal(cache[0].view(-1, 1, D)[:T], got)
    assert torch.equal(cache[1].view(-1, 1, D)[:T], k)
    assert not cache.view(2, -1)[:, T * D:].any()
