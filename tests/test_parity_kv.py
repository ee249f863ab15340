"""GPU parity of the paged 8-bit cache and the attention over it."""
import pytest
import torch

import mamba_selective_scan_04_amd as m
from kv_util import attend, check, inputs

pytestmark = pytest.mark.gpu
E4M3, I8 = torch.float8_e4m3fn, torch.int8
DTYPES = [torch.float32, torch.bfloat16]


def cache_of(c):
    return m.KvCache(c["k"], c["ks"], c["v"], c["vs"])


def run(c, **kw):
    return m.kv_attn_step(cache_of(c), c["q"], c["nk"], c["nv"], c["table"], c["ctx"], lens=c["lens"], **kw)


# batch, ctx, L, Lq, heads_q, heads_kv, d, page
ATTN = [(1, [1], 1, 1, 1, 1, 64, 16), (2, [0, 63], 1, 1, 4, 1, 128, 16), (3, [64, 65, 130], 16, 16, 4, 2, 64, 16),
        (2, [300, 17], 5, 5, 6, 2, 128, 32), (2, [1000, 700], 16, 16, 16, 4, 128, 64), (1, [513], 70, 3, 3, 3, 64, 128),
        (4, [0, 1, 127, 128], 33, 33, 8, 4, 64, 128)]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("code", [E4M3, I8])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size", ATTN)
def test_attention(dev, size, dtype, code, causal):
    c = inputs(*size, code, dtype, device=dev)
    check(run(c, causal=causal), attend(c, causal))


@pytest.mark.parametrize("dtype", DTYPES)
def test_ragged_rows(dev, dtype):
    """Rows without context, without active tokens, with neither; fewer active tokens than queries."""
    c = inputs(5, [0, 100, 0, 37, -5], 16, 16, 4, 2, 64, 16, I8, dtype, seed=1, device=dev, lens=[16, 0, 0, 3, 40])
    for b, n in enumerate([16, 0, 0, 3, 16]):
        c["nk"][b, n:] = float("nan")
        c["nv"][b, n:] = float("nan")
    for causal in (False, True):
        o = run(c, causal=causal)
        assert (o[1] == 0).all() and (o[2] == 0).all() and (o[3, 3:] == 0).all()
        check(o, attend(c, causal))


@pytest.mark.parametrize("code", [E4M3, I8])
def test_what_lies_behind_the_context(dev, code):
    """NaN codes and scales in unused pages, codes behind the context in its last page, table entries that name no page."""
    c = inputs(2, [70, 200], 4, 4, 4, 2, 128, 32, code, torch.bfloat16, seed=2, device=dev)
    c["table"][1, 2] = -1
    c["table"][1, 3] = 1 << 20
    want = attend(c)
    bad = 0x7F
    c["k"].view(torch.uint8)[c["table"][0, 2].long(), :, 6:] = bad
    c["v"].view(torch.uint8)[c["table"][0, 2].long(), :, :, 6:] = bad
    used = {int(x) for x in c["table"][0, :3]} | {int(x) for x in c["table"][1, [0, 1, 4, 5, 6]]}
    for p in set(range(c["k"].shape[0])) - used:
        c["ks"][p] = c["vs"][p] = float("nan")
        c["k"].view(torch.uint8)[p] = c["v"].view(torch.uint8)[p] = bad
    check(run(c), want)


def test_large_scores(dev):
    """One key that takes everything, scores far apart: the running maximum moves."""
    c = inputs(1, [400], 4, 4, 2, 1, 64, 16, I8, torch.float32, seed=3, device=dev)
    c["q"] *= 30
    check(run(c), attend(c))
    check(run(c, scale=1e-6), attend(c, scale=1e-6))


def test_long_context_splits(dev):
    """Ranges of keys joined through the workspace, a shared page among rows."""
    c = inputs(2, [5000, 4100], 16, 16, 8, 2, 64, 16, E4M3, torch.bfloat16, seed=4, device=dev)
    c["table"][1, :100] = c["table"][0, :100]
    s = m.KvShape(2, 8, 2, 64, 16, c["k"].shape[0], c["table"].shape[1], 1, 0)
    import ctypes
    assert m.load().bdssm_kv_workspace_bytes(ctypes.byref(s), 16) > 0
    a, b = run(c), run(c)
    assert torch.equal(a, b)
    check(a, attend(c))


def definition(x, code):
    """Codes and scale of one block and head, by the documented 32-bit definition."""
    top = 448.0 if code == E4M3 else 127.0
    x = x.float()
    fin = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x))
    scale = torch.maximum(fin.max() * (torch.tensor(1.0) / top), torch.tensor(2.0 ** -126))
    y = (x / scale).clamp(-top, top)
    return (y.round() if code == I8 else y).to(code), scale


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("code", [E4M3, I8])
@pytest.mark.parametrize("d,page,T", [(64, 16, 16), (128, 16, 50), (64, 32, 64), (128, 64, 130), (64, 128, 300), (128, 128, 128)])
def test_commit(dev, d, page, T, code, dtype):
    gen = torch.Generator().manual_seed(7)
    batch, heads, per = 3, 2, T // page + 2
    n = batch * per + 2
    k, v = (torch.randn(batch, T, heads, d, generator=gen).to(dtype) for _ in range(2))
    k[0, 0, 0] *= 100
    v[1, :, 1] = 0
    table = torch.randperm(n, generator=gen)[: batch * per].reshape(batch, per).to(torch.int32)
    ctx = torch.tensor([0, page, page + 3], dtype=torch.int32)
    lens = torch.tensor([T, page, T + 7], dtype=torch.int32)
    table[0, 0] = n + 5 if T // page > 1 else table[0, 0]   # names no page
    cache = m.kv_cache(n, heads, d, page, code, device=dev)
    for t in (cache.k, cache.v):
        t.view(torch.uint8).fill_(0x55)
    before = [t.clone() for t in cache]
    m.kv_commit(cache, k.to(dev), v.to(dev), table.to(dev), ctx.to(dev), lens=lens.to(dev))
    want = [t.cpu().clone() for t in before]
    for b in range(batch):
        for j in range(min(T, int(lens[b])) // page):
            at = int(table[b, int(ctx[b]) // page + j])
            if at >= n:
                continue
            for h in range(heads):
                for x, ci, si in ((k, 0, 1), (v, 2, 3)):
                    codes, scale = definition(x[b, j * page:(j + 1) * page, h], code)
                    want[ci].view(torch.uint8)[at, h] = (codes if ci == 0 else codes.T.contiguous()).view(torch.uint8)
                    want[si][at, h] = scale
    for got, ref in zip(cache, want):
        # -0 and 0 are one value
        assert torch.equal(got.cpu().float(), ref.float())


@pytest.mark.parametrize("code", [E4M3, I8])
def test_commit_of_special_values(dev, code):
    x = torch.randn(1, 16, 1, 64, generator=torch.Generator().manual_seed(8))
    x[0, 0, 0, :5] = torch.tensor([float("inf"), -float("inf"), float("nan"), 1e-38, -0.0])
    tiny = torch.full((1, 16, 1, 64), 1e-39)
    cache = m.kv_cache(1, 1, 64, 16, code, device=dev)
    m.kv_commit(cache, x.to(dev), tiny.to(dev), torch.zeros(1, 1, dtype=torch.int32, device=dev),
                torch.zeros(1, dtype=torch.int32, device=dev))
    codes, scale = definition(x[0, :, 0], code)
    got = cache.k[0, 0].cpu().float()
    top = 448.0 if code == E4M3 else 127.0
    assert float(cache.k_scale[0, 0]) == float(scale)
    assert got[0, 0] == top and got[0, 1] == -top and got[0, 3] == 0
    assert torch.isnan(got[0, 2]) if code == E4M3 else got[0, 2] == 0
    assert torch.equal(got[1:], codes.float()[1:])
    assert float(cache.v_scale[0, 0]) == 2.0 ** -126


def test_commit_then_attend(dev):
    """As used: a prompt's blocks committed, the rest active; then block by block."""
    gen = torch.Generator().manual_seed(9)
    T, page, hq, hkv, d = 100, 16, 4, 2, 64
    k, v = (torch.randn(1, T, hkv, d, generator=gen).to(dev) for _ in range(2))
    q = torch.randn(1, T, hq, d, generator=gen).to(dev)
    cache = m.kv_cache(8, hkv, d, page, I8, device=dev)
    table = torch.arange(7, -1, -1, dtype=torch.int32, device=dev)[None].contiguous()
    zero = torch.zeros(1, dtype=torch.int32, device=dev)
    m.kv_commit(cache, k[:, :70].clone(), v[:, :70].clone(), table, zero)   # four whole blocks of 70 tokens
    o = m.kv_attn_step(cache, q[:, 64:70].clone(), k[:, 64:70].clone(), v[:, 64:70].clone(), table, zero + 64)
    c = dict(k=cache.k, v=cache.v, ks=cache.k_scale, vs=cache.v_scale, q=q[:, 64:70], nk=k[:, 64:70], nv=v[:, 64:70],
             table=table, ctx=zero + 64, lens=None)
    check(o, attend(c))
    m.kv_commit(cache, k[:, 64:80].clone(), v[:, 64:80].clone(), table, zero + 64)
    o = m.kv_attn_step(cache, q[:, 80:96].clone(), k[:, 80:96].clone(), v[:, 80:96].clone(), table, zero + 80)
    c.update(q=q[:, 80:96], nk=k[:, 80:96], nv=v[:, 80:96], ctx=zero + 80)
    check(o, attend(c))
