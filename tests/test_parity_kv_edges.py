"""GPU parity of the paged 8-bit cache at its edges: infinities and NaN in
places a mask hides, scales far from 1, every split of the context, other
streams, graphs and the cache's life as a server runs it."""
import pytest
import torch

import mamba_selective_scan_04_amd as m
from kv_util import attend, check, inputs
from test_parity_kv import E4M3, I8, cache_of, definition, run

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,Lq", [(64, 40), (128, 7), (128, 40)])
def test_masked_active_tokens_may_hold_anything(dev, d, Lq, dtype):
    """Causal: a token's infinities and NaN reach the queries that see it, and no other."""
    c = inputs(2, [50, 0], 40, Lq, 4, 2, d, 16, E4M3, dtype, seed=11, device=dev)
    want = attend(c, True)
    at = 37
    c["nk"][:, at + 1] = float("nan")
    c["nv"][:, at] = float("nan")
    c["nv"][:, at + 1] = float("inf")
    c["nv"][:, at + 2, :, ::2] = -float("inf")
    o = run(c, causal=True)
    first = 40 - Lq                          # the token of query 0
    seen = slice(0, at - first)
    check(o[:, seen], [x[:, seen] for x in want])
    assert not torch.isfinite(o[:, at - first:]).any()


@pytest.mark.parametrize("splits", [1, 2, 3, 7, 40])
@pytest.mark.parametrize("code", [E4M3, I8])
def test_every_split_agrees(dev, monkeypatch, splits, code):
    """Ranges that are empty, that end inside a page, more of them than steps."""
    monkeypatch.setenv("BDSSM_KV_SPLITS", str(splits))
    c = inputs(3, [0, 33, 517], 9, 5, 6, 2, 64, 32, code, torch.bfloat16, seed=12, device=dev, lens=[9, 4, 0])
    for causal in (False, True):
        check(run(c, causal=causal), attend(c, causal))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("code", [E4M3, I8])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 16), (64, 64), (64, 128), (128, 128)])
@pytest.mark.parametrize("power", [-125, -88, -60, 0, 90, 118])
def test_commit_at_every_magnitude(dev, d, page, code, dtype, power):
    """Codes are the documented ones where scale or quotients leave the usual range."""
    gen = torch.Generator().manual_seed(13)
    x = (torch.randn(1, page, 2, d, generator=gen).clamp(-3, 3) * 2.0 ** power).to(dtype)
    y = (torch.rand(1, page, 2, d, generator=gen) * 2.0 ** power).to(dtype)
    cache = m.kv_cache(1, 2, d, page, code, device=dev)
    z = torch.zeros(1, 1, dtype=torch.int32, device=dev)
    m.kv_commit(cache, x.to(dev), y.to(dev), z, z[0])
    for h in range(2):
        for t, codes, scales in ((x[0, :, h], cache.k[0, h], cache.k_scale), (y[0, :, h], cache.v[0, h].T, cache.v_scale)):
            ref, scale = definition(t, code)
            assert float(scales[0, h]) == float(scale)
            assert torch.equal(codes.cpu().float(), ref.float())


@pytest.mark.parametrize("code", [E4M3, I8])
@pytest.mark.parametrize("d,page", [(128, 16), (128, 128)])
def test_commit_special_values_of_one_head(dev, d, page, code):
    """Infinities and NaN in one unit leave its neighbours (other waves and workgroups) as they are."""
    gen = torch.Generator().manual_seed(14)
    x = torch.randn(1, 2 * page, 4, d, generator=gen)
    x[0, page - 1, 1, -1] = float("nan")
    x[0, 3, 1, 5] = -float("inf")
    x[0, page:, 2] = float("inf")
    cache = m.kv_cache(2, 4, d, page, code, device=dev)
    table = torch.tensor([[1, 0]], dtype=torch.int32, device=dev)
    m.kv_commit(cache, x.to(dev), x.to(dev), table, torch.zeros(1, dtype=torch.int32, device=dev))
    top = 448.0 if code == E4M3 else 127.0
    for b in range(2):
        for h in range(4):
            t = x[0, b * page:(b + 1) * page, h]
            ref, scale = definition(t, code)
            ref = ref.float()
            ref[torch.isnan(t)] = float("nan") if code == E4M3 else 0.0
            ref[torch.isinf(t)] = top * torch.sign(t[torch.isinf(t)])
            for got, s in ((cache.k[1 - b, h], cache.k_scale), (cache.v[1 - b, h].T, cache.v_scale)):
                assert float(s[1 - b, h]) == float(scale)
                assert torch.equal(torch.nan_to_num(got.cpu().float(), nan=1e9), torch.nan_to_num(ref, nan=1e9))


def test_commit_behind_the_table(dev):
    """Blocks that a row's table has no entry for are not written; negative lengths count as 0."""
    x = torch.randn(3, 48, 1, 64, generator=torch.Generator().manual_seed(15)).to(dev)
    cache = m.kv_cache(6, 1, 64, 16, I8, device=dev)
    table = torch.arange(6, dtype=torch.int32, device=dev).reshape(3, 2)
    ctx = torch.tensor([16, -4, 1 << 30], dtype=torch.int32, device=dev)
    m.kv_commit(cache, x, x, table, ctx, lens=torch.tensor([48, 16, 48], dtype=torch.int32, device=dev))
    written = cache.k_scale[:, 0] != 0
    assert written.tolist() == [False, True, True, False, False, False]
    m.kv_commit(cache, x, x, table, ctx, lens=torch.tensor([-1, 15, 0], dtype=torch.int32, device=dev))
    assert torch.equal(cache.k_scale[:, 0] != 0, written)


@pytest.mark.parametrize("code", [E4M3, I8])
def test_graph_of_a_block_step(dev, code):
    """Attention (two ranges and more) and commit captured together; each replay, with eager work
    between, equals the eager calls on a second cache, bit for bit."""
    c = inputs(2, [700, 2000], 16, 16, 4, 2, 64, 16, code, torch.bfloat16, seed=16, device=dev)
    cache, other = cache_of(c), m.KvCache(*(t.clone() for t in cache_of(c)))
    ctx, q, nk, nv = (c[n].clone() for n in ("ctx", "q", "nk", "nv"))
    ctx -= ctx % 16

    def step(cache, ctx):
        o = m.kv_attn_step(cache, q, nk, nv, c["table"], ctx)
        m.kv_commit(cache, nk, nv, c["table"], ctx)
        return o

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(m.KvCache(*(t.clone() for t in cache)), ctx)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(cache, ctx)
    gen = torch.Generator().manual_seed(17)
    for i in range(3):
        q.copy_(torch.randn(q.shape, generator=gen).to(q))
        nk.copy_(torch.randn(q.shape, generator=gen)[:, :, :2].to(q))
        nv.copy_(torch.randn(q.shape, generator=gen)[:, :, :2].to(q))
        ctx -= 16
        want = step(other, ctx)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        for a, b in zip(cache, other):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_two_streams_at_once(dev):
    """Calls on two streams, each with its own workspace, while the other runs."""
    cs = [inputs(2, [3000, 4100], 16, 16, 8, 2, 64, 16, E4M3, torch.bfloat16, seed=s, device=dev) for s in (18, 19)]
    want = [run(c) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(cs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])
