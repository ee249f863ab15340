"""The hybrid's operators as they are used: a prompt and its blocks through
both kinds of layer, captured and replayed, on streams of their own, at offsets
beyond 32 bits."""
import pytest
import torch

import mamba_selective_scan_04_amd as m
from delta_util import check, inputs, reference
from kv_util import attend, check as check_attn

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16]


def args(c):
    return c["q"], c["k"], c["v"], c["g"], c["beta"]


def piece(c, a, z):
    return [x[:, a:z].clone(memory_format=torch.contiguous_format) for x in args(c)]


@pytest.mark.parametrize("code", [torch.float8_e4m3fn, torch.int8])
def test_prompt_then_blocks(dev, code):
    """A padded batch of prompts, then blocks of 16: three denoising steps each (caches read only),
    then the block's commit into both caches.  Each row against its own sequence in 64 bits."""
    block, steps, blocks, Tp, hq, hkv, d = 16, 3, 3, 83, 4, 2, 64
    prompt = [80, 32]                                     # whole blocks
    total = Tp + blocks * block
    dt = torch.bfloat16
    c = inputs(2, total, 2, 4, 128, 64, dt, seed=30, device=dev)
    gen = torch.Generator().manual_seed(31)
    rn = lambda *s: torch.randn(*s, generator=gen).to(dt).to(dev)  # noqa: E731
    q, k, v = rn(2, total, hq, d), rn(2, total, hkv, d), rn(2, total, hkv, d)
    # row b's tokens: its prompt, then its blocks (each row's sequence without padding)
    lens = torch.tensor(prompt, dtype=torch.int32, device=dev)
    cache = m.kv_cache(40, hkv, d, block, code, device=dev)
    table = torch.randperm(40, generator=gen)[:18].reshape(2, 9).to(torch.int32).to(dev)
    ctx = torch.zeros(2, dtype=torch.int32, device=dev)
    _, state, _ = m.delta_scan(None, *piece(c, 0, Tp)[1:], lens=lens, want_o=False)
    m.kv_commit(cache, k[:, :Tp].clone(), v[:, :Tp].clone(), table, ctx, lens=lens)
    ctx += lens
    rows = lambda x, at: torch.stack([x[b, at[b]:at[b] + block] for b in range(2)])  # noqa: E731
    at = list(prompt)
    for i in range(blocks):
        active = [rows(x, at) for x in args(c)]
        qkv = [rows(x, at) for x in (q, k, v)]
        before = [state.clone(), *(t.clone() for t in cache)]
        for s in range(steps):                           # the block's tokens are denoised: other inputs each time
            noisy = [active[0], *(x if s == steps - 1 else x.flip(1).contiguous() for x in active[1:])]
            o = m.delta_step(state, *noisy)
            keys = [x if s == steps - 1 else x.flip(1).contiguous() for x in qkv[1:]]
            oa = m.kv_attn_step(cache, qkv[0], *keys, table, ctx)
        assert torch.equal(before[0], state)
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(before[1:], cache))
        m.delta_step(state, None, *active[1:], h_out=state, want_o=False)
        for b in range(2):
            alone = {n: (x[b:b + 1, :at[b] + block] if isinstance(x, torch.Tensor) else x) for n, x in c.items()}
            r = reference(alone)
            check(o[b:b + 1], r["o"][:, at[b]:], "o")
            check(state[b:b + 1], r["h"], "state")
        check_attn(oa, attend(dict(k=cache.k, v=cache.v, ks=cache.k_scale, vs=cache.v_scale, q=qkv[0], nk=qkv[1], nv=qkv[2],
                                   table=table, ctx=ctx, lens=None)))
        m.kv_commit(cache, *qkv[1:], table, ctx)
        ctx += block
        at = [x + block for x in at]
    # what the cache holds is the sequence, to half a step of the codes at the page's largest value
    for b in range(2):
        for p in range(at[b] // block):
            got = cache.k[table[b, p].long()].float() * cache.k_scale[table[b, p].long()][:, None, None]
            want = k[b, p * block:(p + 1) * block].float().transpose(0, 1)
            step = want.abs().amax((1, 2), keepdim=True) * (1 / 254 if code == torch.int8 else 1 / 28)
            assert ((got - want).abs() <= step * 1.001).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("decay", [-20.0, 3.0, 60.0])
def test_step_decays(dev, dtype, decay):
    """The recurrence over decays that leave the exponent's range, with the state cleared on the way."""
    c = inputs(1, 40, 1, 2, 64, 64, dtype, seed=32, device=dev, decay=decay, resets=[7, 8, 31])
    r = reference(c, h=c["h"])
    o = m.delta_step(c["h"], *args(c), h_out=(h := torch.empty_like(c["h"])))
    check(o, r["o"], "o")
    check(h, r["h"], "h")


@pytest.mark.parametrize("dtype", DTYPES)
def test_beta_at_its_ends(dev, dtype):
    """beta 0 (a token that writes nothing), 1 and 2 (a reflection); keys of zero."""
    c = inputs(1, 150, 1, 2, 64, 64, dtype, seed=33, device=dev)
    c["beta"][:, ::5] = 0
    c["beta"][:, 1::5] = 1
    c["beta"][:, 2::5] = 2
    c["k"][:, 40:44] = 0
    if dtype == torch.bfloat16:                          # rounded keys longer than 1 would expand under beta 2
        c["k"] = (c["k"].float() * (1 - 2.0 ** -7)).to(dtype)
    r = reference(c, h=c["h"], want_grads=True)
    o, h, chunks = m.delta_scan(*args(c), h_init=c["h"], want_chunks=True)
    check(o, r["o"], "o", 2.0)          # two tokens' decays no longer shrink errors between them
    check(h, r["h"], "h", 2.0)
    got = m.delta_scan_bwd(*args(c), chunks, c["do"], dh_final=c["dh"], want_dh_init=True)
    for n in ("dq", "dk", "dv", "dg", "dbeta", "dh_init"):
        check(got[n], r[n], n, 4.0)     # the product chain and its transpose, as above
    assert (got["dv"][:, ::5] == 0).all()
    check(m.delta_step(c["h"], *args(c)), r["o"], "step", 2.0)


def capture(f):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = f()
    return g, out


def refill(c, seed):
    new = inputs(*c["v"].shape[:2], c["k"].shape[2], c["v"].shape[2], c["k"].shape[3], c["v"].shape[3], c["v"].dtype, seed=seed)
    for n, x in new.items():
        if x is not None:
            c[n].copy_(x)


@pytest.mark.parametrize("size", [(2, 200, 2, 4, 64, 128), (1, 2100, 1, 1, 128, 64)])
def test_graph_of_forward_and_backward(dev, size):
    """Captured together; replays with other inputs and eager work between equal the eager calls bit for bit."""
    c = inputs(*size, torch.bfloat16, seed=34, device=dev)

    def both():
        o, h, chunks = m.delta_scan(*args(c), h_init=c["h"], want_chunks=True)
        return [o, h, *m.delta_scan_bwd(*args(c), chunks, c["do"], dh_final=c["dh"], want_dh_init=True).values()]

    g, got = capture(both)
    for i in range(3):
        refill(c, 35 + i)
        want = both()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        want = both()                                    # and after a replay
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_graph_advances_the_state(dev):
    c = inputs(3, 16, 1, 2, 128, 128, torch.bfloat16, seed=38, device=dev)
    state = c["h"].clone()
    g, o = capture(lambda: m.delta_step(state, *args(c), h_out=state))
    state.copy_(c["h"])
    h = c["h"].clone()
    for i in range(3):
        refill(c, 39 + i)
        c["h"].zero_()
        want = m.delta_step(h, *args(c), h_out=h)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(state, h)


def test_two_streams_at_once(dev):
    cs = [inputs(2, 700, 2, 2, 128, 128, torch.bfloat16, seed=s, device=dev) for s in (42, 43)]

    def both(c):
        o, h, chunks = m.delta_scan(*args(c), want_chunks=True)
        return [o, h, *(x for x in m.delta_scan_bwd(*args(c), chunks, c["do"]).values() if x is not None)]

    want = [both(c) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(both(cs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(g, want[i]))


def test_values_beyond_32_bit_offsets(dev):
    """5 rows of 65,536 tokens and 128 heads of 64: 2.7e9 values, states and matrices further still.
    The last row against a call of its own."""
    batch, T, hv = 5, 65536, 128
    if torch.cuda.mem_get_info()[0] < 160 << 30:
        pytest.skip("needs 160 GiB of device memory")
    gen = torch.Generator(device=dev).manual_seed(44)
    rn = lambda *s: torch.randn(*s, generator=gen, device=dev, dtype=torch.bfloat16)  # noqa: E731
    unit = lambda x: (x.float() / x.float().norm(dim=-1, keepdim=True)).to(x.dtype)  # noqa: E731
    q, k = unit(rn(batch, T, 1, 64)), unit(rn(batch, T, 1, 64))
    v, do = rn(batch, T, hv, 64), rn(batch, T, hv, 64)
    g = -torch.rand(batch, T, hv, generator=gen, device=dev) * 0.1
    beta = torch.rand(batch, T, hv, generator=gen, device=dev)
    last = [x[4:].clone() for x in (q, k, v, g, beta)]
    o, h, chunks = m.delta_scan(q, k, v, g, beta, want_chunks=True)
    o1, h1, chunks1 = m.delta_scan(*last, want_chunks=True)
    same = lambda a, b: (a.double() - b.double()).norm() <= 2.0 ** -8 * b.double().norm()  # noqa: E731
    assert same(o[4:], o1) and same(h[4:], h1) and same(chunks[4, -4:], chunks1[0, -4:])
    del o, o1
    got = m.delta_scan_bwd(q, k, v, g, beta, chunks, do)
    alone = m.delta_scan_bwd(*last, chunks1, do[4:].clone())
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert same(got[n][4:, -300:], alone[n][:, -300:]) and same(got[n][4:, :300], alone[n][:, :300]), n
    hb = h.clone()
    ob = m.delta_step(hb, *[x[:, -16:].contiguous() for x in (q, k, v, g, beta)])
    assert same(ob[4:], m.delta_step(hb[4:].clone(), *[x[:, -16:].contiguous() for x in last]))


@pytest.mark.parametrize("code", [torch.float8_e4m3fn, torch.int8])
def test_pages_beyond_32_bit_offsets(dev, code):
    n, hkv, d, page = 1_100_000, 2, 128, 16             # 4.5e9 codes of keys, as many of values
    cache = m.kv_cache(n, hkv, d, page, code, device=dev)
    gen = torch.Generator().manual_seed(45)
    k, v = (torch.randn(1, 64, hkv, d, generator=gen).to(torch.bfloat16).to(dev) for _ in range(2))
    table = torch.tensor([[n - 1, 1_048_576, n - 2, 5]], dtype=torch.int32, device=dev)
    zero = torch.zeros(1, dtype=torch.int32, device=dev)
    m.kv_commit(cache, k, v, table, zero)
    small = m.kv_cache(4, hkv, d, page, code, device=dev)
    m.kv_commit(small, k, v, torch.arange(4, dtype=torch.int32, device=dev)[None], zero)
    for a, b in zip(cache, small):
        assert torch.equal(a[table[0].long()].float(), b.float())
        assert float(a[:5].float().abs().sum()) == 0
    q = torch.randn(1, 1, 4, d, generator=gen).to(torch.bfloat16).to(dev)
    nk, nv = k[:, :1].clone(), v[:, :1].clone()
    o = m.kv_attn_step(cache, q, nk, nv, table, zero + 64)
    ref = m.kv_attn_step(small, q, nk, nv, torch.arange(4, dtype=torch.int32, device=dev)[None], zero + 64)
    assert torch.equal(o, ref)
