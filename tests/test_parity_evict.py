"""The attention's log-sum-exp, the pages' weights and the eviction against their
definitions.  Tolerances of weights: kv_util's, for the same scores."""
import math

import pytest
import torch

import mamba_selective_scan_04_amd as m
from kv_util import attend, check, inputs

CODES = [torch.float8_e4m3fn, torch.int8]
DTYPES = [torch.float32, torch.bfloat16]
# batch, contexts, L, Lq, heads_q, heads_kv, d, page
SIZES = [
    (1, [0], 1, 1, 1, 1, 64, 16),
    (2, [1, 15], 3, 2, 2, 1, 64, 16),
    (2, [16, 33], 5, 5, 4, 2, 128, 32),
    (3, [127, 128, 129], 16, 16, 6, 3, 64, 64),
    (2, [300, 7], 4, 1, 12, 4, 64, 128),
    (1, [517], 17, 17, 8, 1, 128, 16),
    (4, [200, 0, 64, 131], 9, 7, 5, 5, 64, 32),
]


def reference(c, scale=None):
    """lse [batch, Lq, heads_q] (non-causal) and weights by page [batch, max_pages], fp64."""
    x = {n: t.detach().cpu() if t is not None else None for n, t in c.items()}
    batch, Lq, hq, d = x["q"].shape
    L, hkv = x["nk"].shape[1:3]
    page, pages = x["k"].shape[2], x["table"].shape[1]
    scale = d ** -0.5 if scale is None else scale
    lse = torch.full((batch, Lq, hq), -math.inf, dtype=torch.float64)
    mass = torch.zeros(batch, pages, dtype=torch.float64)
    for b in range(batch):
        ctx = min(max(0, int(x["ctx"][b])), pages * page)
        n = L if x["lens"] is None else min(max(0, int(x["lens"][b])), L)
        at = [t for t in range(ctx) if 0 <= int(x["table"][b, t // page]) < x["k"].shape[0]]
        ids = torch.tensor([int(x["table"][b, t // page]) for t in at], dtype=torch.long)
        off = torch.tensor([t % page for t in at], dtype=torch.long)
        where = torch.tensor([t // page for t in at], dtype=torch.long)
        for h in range(hq):
            hk = h // (hq // hkv)
            K = x["k"].float().double()[ids, hk, off] * x["ks"].double()[ids, hk][:, None]
            K = torch.cat([K, x["nk"][b, :n, hk].double()])
            for i in range(min(n, Lq)):
                w = scale * (K @ x["q"][b, i, h].double())
                if len(w):
                    lse[b, i, h] = torch.logsumexp(w, 0)
                    mass[b].index_add_(0, where, (w[:len(at)] - lse[b, i, h]).exp())
    return lse, mass


def cache(c):
    return m.KvCache(c["k"], c["ks"], c["v"], c["vs"])


def run(c, **kw):
    o, lse = m.kv_attn_step(cache(c), c["q"], c["nk"], c["nv"], c["table"], c["ctx"], lens=c["lens"], want_lse=True)
    return o, lse, m.kv_attn_weights(cache(c), c["q"], lse, c["table"], c["ctx"], lens=c["lens"], **kw)


def check_weights(got, want):
    g = got.cpu().double()
    assert torch.isfinite(g).all()
    assert (g - want).norm() <= 2e-5 * max(float(want.norm()), 1e-30), float((g - want).norm() / want.norm())


@pytest.mark.gpu
@pytest.mark.parametrize("splits", [None, 3])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("size", SIZES)
def test_lse_and_weights(dev, monkeypatch, code, dtype, size, splits):
    if splits:
        monkeypatch.setenv("BDSSM_KV_SPLITS", str(splits))
    lens = [max(0, size[2] - 2 * b) for b in range(size[0])]
    c = inputs(*size, code, dtype, seed=sum(size[1]) + size[2], device=dev, lens=lens)
    lse, mass = reference(c)
    o, got, weights = run(c)
    check(o, attend(c), "o")
    none = lse == -math.inf
    assert torch.equal(got.cpu() == -math.inf, none)
    off = (got.cpu().double() - lse)[~none].abs()
    assert (off <= 1.3e-4 + 4 * 2.0 ** -24 * lse[~none].abs()).all() and (not off.numel() or off.norm() <= 2e-5 * lse[~none].norm() + 1e-6 * off.numel())
    check_weights(weights, mass)
    plain = m.kv_attn_step(cache(c), c["q"], c["nk"], c["nv"], c["table"], c["ctx"], lens=c["lens"])
    assert torch.equal(plain, o)
    # what was there before, to another place and in place; behind the context nothing moves
    had = torch.rand(mass.shape, generator=torch.Generator().manual_seed(1)).to(dev)
    both = run(c, mass=had)[2]
    assert torch.equal(both, had + weights)
    mine = had.clone()
    assert run(c, mass=mine, out=mine)[2] is mine and torch.equal(mine, both)
    # of a query and head, the weights of the cache and of the active tokens are 1: the total is at most that
    assert float(weights.sum()) <= sum(min(n, size[3]) for n in lens) * size[4] * (1 + 1e-4)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_causal_lse(dev, dtype):
    c = inputs(2, [70, 0], 20, 20, 4, 2, 64, 16, torch.int8, dtype, seed=5, device=dev, lens=[20, 9])
    _, lse = m.kv_attn_step(cache(c), c["q"], c["nk"], c["nv"], c["table"], c["ctx"], lens=c["lens"], causal=True, want_lse=True)
    for i in range(20):              # query i alone, with the tokens it sees
        for b, n in ((0, 20), (1, 9)):
            if i >= n:
                assert (lse[b, i] == -math.inf).all()
                continue
            one = {k: x[b:b + 1].contiguous() if k in ("table", "ctx") else x for k, x in c.items()}
            one.update(q=c["q"][b:b + 1, i:i + 1].contiguous(), nk=c["nk"][b:b + 1, :i + 1].contiguous(), nv=c["nv"][b:b + 1, :i + 1].contiguous(),
                       lens=None)
            want, _ = reference(one)
            assert ((lse[b, i].cpu().double() - want[0, 0]).abs() <= 1.3e-4).all()


@pytest.mark.gpu
@pytest.mark.parametrize("code", CODES)
def test_what_is_not_seen(dev, code):
    """Codes and scales behind the context, pages that are not there, padding's queries and NaN of other heads stay out."""
    c = inputs(3, [130, 40, 77], 6, 6, 4, 2, 128, 32, code, torch.bfloat16, seed=6, device=dev, lens=[6, 2, 0])
    c["table"][0, 2] = -1
    c["table"][0, 3] = c["k"].shape[0]
    _, mass = reference(c)
    _, lse, weights = run(c)
    check_weights(weights, mass)
    assert (weights[0, 2:4] == 0).all() and (weights[2] == 0).all() and (weights[1, 2:] == 0).all()
    used = {int(c["table"][b, t // 32]) for b, n in ((0, 130), (1, 40), (2, 77)) for t in range(n) if 0 <= int(c["table"][b, t // 32]) < c["k"].shape[0]}
    for p in range(c["k"].shape[0]):
        if p not in used:
            c["ks"][p] = float("nan")
    if code == torch.float8_e4m3fn:
        bad = c["k"].view(torch.uint8)
        bad[int(c["table"][0, 4]), :, 2:] = 0x7f          # behind 130
        bad[int(c["table"][1, 1]), :, 8:] = 0x7f          # behind 40
    c["q"][1, 2:] = float("nan")
    c["q"][2] = float("inf")
    lse[1, 2:] = float("nan")
    lse[2] = 3.0
    got = m.kv_attn_weights(cache(c), c["q"], lse, c["table"], c["ctx"], lens=c["lens"])
    assert torch.equal(got, weights)


@pytest.mark.gpu
def test_wide_tables_and_no_pages(dev):
    c = inputs(2, [50, 20], 4, 4, 2, 2, 64, 16, torch.int8, torch.bfloat16, seed=7, device=dev)
    _, lse, w = run(c)
    wide = torch.full((2, 1000), -1, dtype=torch.int32, device=dev)
    wide[:, :c["table"].shape[1]] = c["table"]
    had = torch.rand(2, 1000, device=dev)
    got = m.kv_attn_weights(cache(c), c["q"], lse, wide, c["ctx"], mass=had)
    assert torch.equal(got[:, :4], had[:, :4] + w) and torch.equal(got[:, 4:], had[:, 4:])
    empty = m.kv_cache(0, 2, 64, 16, torch.int8, device=dev)
    assert torch.equal(m.kv_attn_weights(empty, c["q"], lse, wide, c["ctx"], mass=had), had)
    z = c["q"][:, :0].contiguous()
    assert torch.equal(m.kv_attn_weights(cache(c), z, lse[:, :0].contiguous(), wide, c["ctx"], mass=had), had)
    assert m.kv_attn_weights(cache(c), c["q"], lse, wide[:, :0].contiguous(), c["ctx"]).shape == (2, 0)


def evicted(table, ctx, mass, page, budget, sink, recent):
    """Row by row on the host."""
    T, C, M = [], [], []
    for b in range(len(ctx)):
        n = min(max(0, int(ctx[b])), table.shape[1] * page)
        whole, used = n // page, -(-n // page)
        row = list(zip(table[b].tolist(), mass[b].tolist()))
        order = sorted(range(sink, whole - recent), key=lambda i: (math.isnan(row[i][1]), 0 if math.isnan(row[i][1]) else row[i][1], i))
        gone = set(order[:max(0, whole - budget)])
        new = [row[i] for i in range(used) if i not in gone] + [(row[i][0], 0.0) for i in sorted(gone)] + row[used:]
        T.append([x[0] for x in new])
        M.append([x[1] for x in new])
        C.append(n - len(gone) * page)
    return torch.tensor(T, dtype=torch.int32).reshape(table.shape), torch.tensor(C, dtype=torch.int32), torch.tensor(M).reshape(mass.shape)


def check_evict(dev, table, ctx, mass, page, budget, sink, recent):
    got = m.kv_evict(table.to(dev), ctx.to(dev), mass.to(dev), page, budget, sink=sink, recent=recent)
    want = evicted(table, ctx, mass, page, budget, sink, recent)
    assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1])
    g, w = got[2].cpu(), want[2].float()
    assert torch.equal(g.isnan(), w.isnan()) and torch.equal(g.nan_to_num(-1.0), w.nan_to_num(-1.0))


@pytest.mark.gpu
@pytest.mark.parametrize("pages", [1, 2, 63, 64, 65, 256, 1000, 1024, 1025, 4096, 4097, 16384, 16385, 40000])
@pytest.mark.parametrize("kind", ["spread", "ties", "equal"])
def test_evict(dev, pages, kind):
    gen = torch.Generator().manual_seed(pages)
    batch, page = 4, 32
    table = torch.stack([torch.randperm(pages, generator=gen) for _ in range(batch)]).to(torch.int32)
    mass = (torch.randn(batch, pages, generator=gen) * 3).exp()
    if kind == "ties":
        mass = (mass * 2).floor().clamp(max=3)
    if kind == "equal":
        mass = torch.full_like(mass, 0.5)
    ctx = torch.tensor([pages * page, pages * page // 2 + 5, 0, max(0, pages * page - 1)], dtype=torch.int32)
    for budget, sink, recent in ((pages // 2, 0, 0), (pages // 3, min(2, pages // 3), 0), (pages // 2, min(1, pages // 4), pages // 4), (0, 0, 0),
                                 (pages, pages, 0), (pages // 2, 0, pages // 2)):
        check_evict(dev, table, ctx, mass, page, budget, sink, recent)


@pytest.mark.gpu
def test_evict_special_weights(dev):
    gen = torch.Generator().manual_seed(3)
    pages = 300
    mass = torch.randn(3, pages, generator=gen)
    mass[0, ::7], mass[0, 1::7], mass[0, 2::7], mass[0, 3::7] = float("nan"), float("inf"), float("-inf"), -0.0
    mass[0, 4::7] = 0.0
    mass[1] = torch.where(torch.rand(pages, generator=gen) < 0.5, 1e-42, -1e-42)      # below the normal numbers
    mass[2, ::2] = -torch.tensor(float("nan"))
    table = torch.arange(3 * pages, dtype=torch.int32).reshape(3, pages)
    ctx = torch.full((3,), pages * 16, dtype=torch.int32)
    for budget in (0, 40, 90, 150, 200, 299, 300, 10 ** 12):
        check_evict(dev, table, ctx, mass, 16, budget, 0, 0)
    check_evict(dev, table, ctx, mass, 16, 100, 3, 50)


@pytest.mark.gpu
def test_evict_leaves_strange_rows_alone(dev):
    """Lengths below 0 and beyond the table; a table of no entries; the caller's own outputs."""
    table = torch.arange(20, dtype=torch.int32).reshape(2, 10)
    mass = torch.rand(2, 10, generator=torch.Generator().manual_seed(4))
    check_evict(dev, table, torch.tensor([-7, 10 ** 9], dtype=torch.int32), mass, 128, 4, 1, 1)
    z = torch.zeros(2, 0, device=dev)
    t, c, _ = m.kv_evict(z.to(torch.int32), torch.tensor([0, 5], dtype=torch.int32, device=dev), z, 16, 3)
    assert t.shape == (2, 0) and (c == 0).all()
    outs = dict(table_out=torch.empty(2, 10, dtype=torch.int32, device=dev), ctx_out=torch.empty(2, dtype=torch.int32, device=dev),
                mass_out=torch.empty(2, 10, device=dev))
    a = table.to(dev), torch.tensor([160, 33], dtype=torch.int32, device=dev), mass.to(dev), 16, 3
    got = m.kv_evict(*a, **outs)
    assert all(x is y for x, y in zip(got, outs.values())) and all(torch.equal(x, y) for x, y in zip(got, m.kv_evict(*a)))


@pytest.mark.gpu
@pytest.mark.parametrize("pages", [320, 321, 8192, 8193, 20480, 20481])
@pytest.mark.parametrize("kind", ["spread", "narrow", "special", "negative"])
def test_evict_layouts(dev, pages, kind):
    """Each layout of a row over threads at its ends; weights of one exponent (more than one wave takes), of both
    infinities and NaN, all below 0."""
    gen = torch.Generator().manual_seed(pages + 1)
    table = torch.stack([torch.randperm(pages, generator=gen) for _ in range(3)]).to(torch.int32)
    mass = (torch.randn(3, pages, generator=gen) * 4).exp()
    if kind == "narrow":
        mass = 1 + torch.rand(3, pages, generator=gen).clamp(max=0.999)
    if kind == "special":
        r = torch.rand(3, pages, generator=gen)
        mass[r < 0.2], mass[(r >= 0.2) & (r < 0.4)], mass[(r >= 0.4) & (r < 0.5)] = float("inf"), float("nan"), float("-inf")
    if kind == "negative":
        mass = -mass
    ctx = torch.tensor([pages * 16, pages * 16 - 7, pages * 8], dtype=torch.int32)
    for budget in (0, 1, pages // 10, pages // 2, pages * 3 // 5, pages * 9 // 10, pages - 1, pages):
        check_evict(dev, table, ctx, mass, 16, budget, 0, 0)
    check_evict(dev, table, ctx, mass, 16, pages // 2, 5, 64)
