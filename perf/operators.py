"""Cases and plain forms of the hybrid layer's operators.

The block-diffusion hybrid keeps two caches per layer: a recurrent boundary
state and the attention's keys and values.  The operators here are

* scan, train, step: the gated delta rule over whole sequences, its gradients,
  and its recurrent form on the active tokens.  With a = exp(g),
      S_t = a_t S_{t-1} + k_t u_t^T,  u_t = beta_t (v_t - (a_t S_{t-1})^T k_t),
      o_t = scale S_t^T q_t;
  heads_k query/key heads, each shared by heads_v / heads_k value heads;
  tokens at and behind lens[b] are padding: no state, no gradient, o = 0;
* commit: finished blocks of keys and values into a paged 8-bit cache with one
  scale for each page and head;
* attn: the active block's queries over that cache and the block's own keys
  and values.

run() computes them by elementary torch operations in 32 bits (64 for sums of
log decays), or, with `own` set, through this repository's package.
"""
import math

import torch

own = False

DEV = "cuda"
CHUNK = 64
STREAM = {"bf16": torch.bfloat16, "f32": torch.float32}
CODE = {"e4m3": torch.float8_e4m3fn, "i8": torch.int8}
QMAX = {"e4m3": 448.0, "i8": 127.0}
TINY = 2.0 ** -126


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the smallest layer, fp32 streams, one short sequence: launch latency counts
        dict(name="scan tiny f32", op="scan", batch=1, T=256, heads_k=1, heads_v=1, dk=64, dv=64, dtype="f32",
             ragged=False, resets=False, init=True),
        # prefill of one 65,536-token context, d_inner 1536: twelve chains only, a long axis
        dict(name="scan prefill 65k b1", op="scan", batch=1, T=65536, heads_k=12, heads_v=12, dk=128, dv=128,
             dtype="bf16", ragged=False, resets=False, init=False),
        # a padded batch of prompts of every length, d_inner 2048 with shared query/key heads
        dict(name="scan prompts b8", op="scan", batch=8, T=1000, heads_k=8, heads_v=16, dk=128, dv=128, dtype="bf16",
             ragged=True, resets=False, init=True),
        # a training step's layer of the 87M shape, forward and backward
        dict(name="train 87m", op="train", batch=8, T=4096, heads_k=12, heads_v=12, dk=128, dv=128, dtype="bf16",
             ragged=False, resets=False, init=False),
        # packed documents (the state restarts at each), odd length, 64-wide heads, shared keys
        dict(name="train packed", op="train", batch=2, T=2041, heads_k=4, heads_v=8, dk=64, dv=64, dtype="bf16",
             ragged=True, resets=True, init=True),
        # one sequence, one token: a single decoding step
        dict(name="step b1 token", op="step", batch=1, T=1, heads_k=8, heads_v=16, dk=128, dv=128, dtype="bf16",
             ragged=False, resets=False, init=True),
        # sixty-four sequences finish a 16-token block
        dict(name="step b64 block", op="step", batch=64, T=16, heads_k=8, heads_v=16, dk=128, dv=128, dtype="bf16",
             ragged=True, resets=False, init=True),
        # the prompt's keys and values into the cache after a 65,536-token prefill
        dict(name="commit prompt 65k", op="commit", batch=1, T=65536, heads_kv=4, d=128, page=16, code="e4m3",
             dtype="bf16", ragged=False),
        # sixteen sequences commit one finished block each
        dict(name="commit block b16", op="commit", batch=16, T=16, heads_kv=4, d=64, page=16, code="i8", dtype="bf16",
             ragged=False),
        # one denoising step of one sequence behind 65,536 cached tokens
        dict(name="attn 65k b1", op="attn", batch=1, ctx=65536, L=16, Lq=16, heads_q=16, heads_kv=4, d=128, page=16,
             code="e4m3", dtype="bf16", ragged=False, causal=False),
        # one denoising step of four sequences of up to 262,144 cached tokens
        dict(name="attn 262k b4", op="attn", batch=4, ctx=262144, L=16, Lq=16, heads_q=16, heads_kv=4, d=128, page=16,
             code="i8", dtype="bf16", ragged=True, causal=False),
        # token-by-token decoding of many sequences, the last page still open
        dict(name="attn decode b64", op="attn", batch=64, ctx=8192, L=32, Lq=1, heads_q=12, heads_kv=4, d=64, page=32,
             code="i8", dtype="bf16", ragged=True, causal=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("scan", "scan", "train", "train", "step", "commit", "attn", "attn"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    if op in ("scan", "train", "step"):
        heads_k = rng.choice((1, 2, 3, 4, 6, 8, 12))
        heads_v = heads_k * rng.choice((1, 1, 2, 3)) if heads_k < 8 else heads_k
        batch = _log(rng, 1, 64 if op == "step" else 8)
        T = _log(rng, 1, {"scan": 20000, "train": 5000, "step": 64}[op])
        most = {"scan": 600000, "train": 300000, "step": 16384}[op] // (2 if dtype == "f32" else 1)
        T = max(1, min(T, most // (batch * heads_v)))
        return dict(op=op, batch=batch, T=T, heads_k=heads_k, heads_v=heads_v, dk=rng.choice((64, 128)),
                    dv=rng.choice((64, 128)), dtype=dtype, ragged=rng.random() < 0.5, resets=rng.random() < 0.3,
                    init=rng.random() < 0.5)
    heads_kv = rng.choice((1, 2, 3, 4, 8))
    d, page, code = rng.choice((64, 128)), rng.choice((16, 32, 64, 128)), rng.choice(("e4m3", "i8"))
    batch = _log(rng, 1, 64)
    if op == "commit":
        T = min(_log(rng, 16, 65536), max(16, 262144 // (batch * heads_kv)))
        return dict(op=op, batch=batch, T=T, heads_kv=heads_kv, d=d, page=page, code=code, dtype=dtype,
                    ragged=rng.random() < 0.5)
    L = _log(rng, 1, 64)
    ctx = min(_log(rng, 1, 262144), 2000000 // (batch * heads_kv))
    return dict(op=op, batch=batch, ctx=ctx, L=L, Lq=L if rng.random() < 0.6 else rng.randint(1, L),
                heads_q=heads_kv * rng.choice((1, 2, 3, 4, 6, 8)), heads_kv=heads_kv, d=d, page=page, code=code,
                dtype=dtype, ragged=rng.random() < 0.7, causal=rng.random() < 0.4)


# ----------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _lens(gen, batch, top, low=0):
    """Lengths of a padded batch: the first row is full, the last has `low`."""
    n = low + (torch.rand(batch, generator=gen, device=DEV) * (top - low + 1)).to(torch.int32)
    n = n.clamp(max=top)
    n[-1] = low
    n[0] = top
    return n.to(torch.int32)


def prepare(case, seed):
    gen = _gen(seed)
    c, s = case, {"case": dict(case)}
    dt = STREAM[c["dtype"]]
    if c["op"] in ("scan", "train", "step"):
        b, T, hk, hv, dk, dv = (c[n] for n in ("batch", "T", "heads_k", "heads_v", "dk", "dv"))
        # unit queries and keys (a layer normalises them), keys with a common part
        unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
        s["q"] = unit(_randn(gen, b, T, hk, dk)).to(dt)
        s["k"] = unit(_randn(gen, b, T, hk, dk) + 0.3 * _randn(gen, 1, 1, hk, dk)).to(dt)
        s["v"] = _randn(gen, b, T, hv, dv).to(dt)
        # decays from "forgets within a few tokens" to "keeps for thousands"
        g = -torch.nn.functional.softplus(_randn(gen, b, T, hv) * 1.5 - 4.0)
        if c["resets"]:  # a document starts about every 200 tokens
            start = torch.rand(b, T, 1, generator=gen, device=DEV) < 1 / 200
            g = g.masked_fill(start, -math.inf)
        s["g"] = g.contiguous()
        s["beta"] = torch.sigmoid(_randn(gen, b, T, hv))
        s["scale"] = dk ** -0.5
        s["h"] = _randn(gen, b, hv, dk, dv) * 0.1 if c["init"] else None
        s["lens"] = _lens(gen, b, T) if c["ragged"] else None
        if c["op"] == "train":
            s["do"] = _randn(gen, b, T, hv, dv).to(dt)
            s["dh"] = _randn(gen, b, hv, dk, dv) * 0.1
        if c["op"] == "step":
            s["h_out"] = torch.zeros(b, hv, dk, dv, device=DEV)
        return s
    b, hkv, d, page, code = (c[n] for n in ("batch", "heads_kv", "d", "page", "code"))
    tokens = c["T"] if c["op"] == "commit" else c["ctx"]
    per_row = max(1, -(-tokens // page)) + (1 if c["op"] == "commit" else 0)
    n_pages = b * per_row + 1
    order = torch.randperm(n_pages, generator=gen, device=DEV)[: b * per_row]
    s["table"] = order.reshape(b, per_row).to(torch.int32).contiguous()
    if c["op"] == "commit":
        # a few rows already hold one page
        s["ctx"] = (torch.rand(b, generator=gen, device=DEV) < 0.5).to(torch.int32) * page
        s["lens"] = _lens(gen, b, tokens) if c["ragged"] else None
        s["k"] = (_randn(gen, b, tokens, hkv, d) * (0.2 + torch.rand(1, 1, hkv, d, generator=gen, device=DEV) * 3)).to(dt)
        s["v"] = _randn(gen, b, tokens, hkv, d).to(dt)
        s["kc"] = torch.zeros(n_pages, hkv, page, d, device=DEV).to(CODE[code])
        s["vc"] = torch.zeros(n_pages, hkv, d, page, device=DEV).to(CODE[code])
        s["ks"] = torch.zeros(n_pages, hkv, device=DEV)
        s["vs"] = torch.zeros(n_pages, hkv, device=DEV)
        return s

    def codes(*shape):
        n = math.prod(shape)
        if code == "i8":
            return torch.randint(-127, 128, (n,), generator=gen, device=DEV, dtype=torch.int8).reshape(shape)
        return (_randn(gen, n) * 120).clamp_(-448, 448).to(CODE[code]).reshape(shape)

    s["kc"], s["vc"] = codes(n_pages, hkv, page, d), codes(n_pages, hkv, d, page)
    unit = 1 / (120 if code == "e4m3" else 73)  # the codes' spread
    s["ks"] = unit * (0.5 + torch.rand(n_pages, hkv, generator=gen, device=DEV))
    s["vs"] = unit * (0.5 + torch.rand(n_pages, hkv, generator=gen, device=DEV))
    s["q"] = _randn(gen, b, c["Lq"], c["heads_q"], d).to(dt)
    s["k"] = _randn(gen, b, c["L"], hkv, d).to(dt)
    s["v"] = _randn(gen, b, c["L"], hkv, d).to(dt)
    # ragged contexts: a quarter to all of the longest; in large batches one row has none yet
    s["ctx"] = _lens(gen, b, tokens, tokens // 4) if c["ragged"] else torch.full((b,), tokens, dtype=torch.int32,
                                                                                device=DEV)
    if c["ragged"] and b >= 8:
        s["ctx"][-1] = 0
    s["lens"] = _lens(gen, b, c["L"], 1) if c["ragged"] else None
    s["scale"] = d ** -0.5
    return s


# ------------------------------------------------------------ plain forms

def _chunked(x, n):
    """[b, T, h, ...] -> [b, h, n, CHUNK, ...], zeros behind T."""
    pad = n * CHUNK - x.shape[1]
    if pad:
        x = torch.cat([x, x.new_zeros(x.shape[0], pad, *x.shape[2:])], 1)
    return x.reshape(x.shape[0], n, CHUNK, *x.shape[2:]).movedim(3, 1)


def _delta(q, k, v, g, beta, scale, h, lens):
    """The gated delta rule in chunks -> (o, last state), 32 bits (log decays in 64)."""
    b, T, hk, dk = k.shape
    hv, dv = v.shape[2:]
    if lens is not None:
        keep = torch.arange(T, device=k.device)[None, :, None] < lens[:, None, None]
        beta, g = beta * keep, torch.where(keep, g, torch.zeros_like(g))
        # padding may hold anything
        q, k, v = (torch.where(keep[..., None], x, torch.zeros_like(x)) for x in (q, k, v))
    n = -(-T // CHUNK)
    rep = hv // hk
    q, k = (_chunked(x.float(), n).repeat_interleave(rep, 1) for x in (q, k))
    v, beta = _chunked(v.float(), n), _chunked(beta, n)[..., None]
    G = _chunked(g.double().clamp(min=-1e4), n).cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=k.device).tril()
    D = (G[..., :, None] - G[..., None, :]).masked_fill(~low, -math.inf).exp().float()
    P = scale * (q @ k.transpose(-1, -2)) * D
    N = -(beta * (k @ k.transpose(-1, -2)) * D).tril(-1)
    eye = torch.eye(CHUNK, device=k.device)
    inv = eye + N
    for _ in range(5):  # (I - N)^-1 = (I + N)(I + N^2)(I + N^4)... : N is strictly lower
        N = N @ N
        inv = inv + inv @ N
    e = G.exp().float()[..., None]
    rest = (G[..., -1:] - G).exp().float()[..., None]
    last = e[..., -1:, :]
    kw = (k * rest).transpose(-1, -2)
    kr, qr = k * e, scale * q * e
    S = k.new_zeros(b, hv, dk, dv) if h is None else h
    o = []
    for c in range(n):
        U = inv[:, :, c] @ (beta[:, :, c] * (v[:, :, c] - kr[:, :, c] @ S))
        o.append(qr[:, :, c] @ S + P[:, :, c] @ U)
        S = last[:, :, c] * S + kw[:, :, c] @ U
    o = torch.stack(o, 2).movedim(1, 3).reshape(b, n * CHUNK, hv, dv)[:, :T]
    return o, S


def _plain_train(s):
    ins = [x.detach().float().requires_grad_() for x in (s["q"], s["k"], s["v"], s["g"], s["beta"])]
    b, _, hv, dv = s["v"].shape
    h = (s["h"] if s["h"] is not None else ins[0].new_zeros(b, hv, s["k"].shape[3], dv)).detach().requires_grad_()
    with torch.enable_grad():
        o, S = _delta(*ins, s["scale"], h, s["lens"])
        grads = torch.autograd.grad([o, S], ins + [h], [s["do"].float(), s["dh"]])
    out = dict(zip(("dq", "dk", "dv", "dg", "dbeta", "dh_init"), grads))
    for n in ("dq", "dk", "dv"):
        out[n] = out[n].to(s["q"].dtype)
    out["o"] = o.detach().to(s["q"].dtype)
    return out


def _page_slots(table, ctx, lens, T, page):
    """(row, block of the row, page) of every whole block that a commit writes."""
    b = table.shape[0]
    blocks = T // page
    n = torch.full((b,), T, device=table.device) if lens is None else lens.clamp(0, T).long()
    j = torch.arange(blocks, device=table.device)
    row, blk = torch.nonzero(j[None] < (n // page)[:, None], as_tuple=True)
    return row, blk, table.long()[row, ctx.long()[row] // page + blk]


def _quantised(x, qmax, code):
    """[n, page, heads, d] -> codes, scales [n, heads]."""
    x = x.float()
    scale = (x.abs().amax((1, 3)) / qmax).clamp(min=TINY)
    y = (x / scale[:, None, :, None]).clamp(-qmax, qmax)
    return (y.round().to(torch.int8) if code == "i8" else y.to(CODE[code])), scale


def _plain_commit(s):
    c = s["case"]
    row, blk, at = _page_slots(s["table"], s["ctx"], s["lens"], c["T"], c["page"])
    whole = c["T"] // c["page"]
    for x, cache, scale, order in ((s["k"], s["kc"], s["ks"], (0, 2, 1, 3)), (s["v"], s["vc"], s["vs"], (0, 2, 3, 1))):
        blocks = x[:, : whole * c["page"]].reshape(c["batch"], whole, c["page"], c["heads_kv"], c["d"])[row, blk]
        codes, sc = _quantised(blocks, QMAX[c["code"]], c["code"])
        # fp8 tensors have no indexed store: their bytes do
        cache.view(torch.uint8)[at] = codes.permute(*order).contiguous().view(torch.uint8)
        scale[at] = sc
    return dict(k=s["kc"], k_scale=s["ks"], v=s["vc"], v_scale=s["vs"])


def _gathered(s, b0, b1, to):
    """Cached keys and values of rows b0..b1 as [rows, heads, tokens, d] in type `to`."""
    c = s["case"]
    t = s["table"][b0:b1].long()
    rows = t.shape[0]
    k = s["kc"].view(torch.uint8)[t].view(s["kc"].dtype).to(to) * s["ks"][t].to(to)[..., None, None]
    v = s["vc"].view(torch.uint8)[t].view(s["vc"].dtype).to(to) * s["vs"][t].to(to)[..., None, None]
    k = k.permute(0, 2, 1, 3, 4).reshape(rows, c["heads_kv"], -1, c["d"])
    v = v.permute(0, 2, 1, 4, 3).reshape(rows, c["heads_kv"], -1, c["d"])
    return k, v


def _plain_attn(s):
    c = s["case"]
    b, L, Lq, hq, hkv, d = (c[n] for n in ("batch", "L", "Lq", "heads_q", "heads_kv", "d"))
    k, v = _gathered(s, 0, b, torch.float32)
    cached = k.shape[2]
    k = torch.cat([k, s["k"].float().movedim(2, 1)], 2)
    v = torch.cat([v, s["v"].float().movedim(2, 1)], 2)
    ctx = s["ctx"].long()[:, None]
    n = (s["lens"].long() if s["lens"] is not None else torch.full((b,), L, device=k.device))[:, None]
    at = torch.arange(cached + L, device=k.device)[None]
    seen = torch.where(at < cached, at < ctx, at - cached < n)[:, None, :].expand(b, Lq, -1)
    i = torch.arange(Lq, device=k.device)[None]
    nq = n.clamp(max=Lq)
    pos = n - nq + i                       # the active token that query i is
    if c["causal"]:
        seen = seen & ((at < cached)[:, None, :] | (at[:, None, :] - cached <= pos[:, :, None]))
    seen = seen & (i < nq)[:, :, None]
    v = torch.where((seen.any(1))[:, None, :, None], v, torch.zeros_like(v))
    q = s["q"].float().reshape(b, Lq, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)
    w = s["scale"] * (q @ k.transpose(-1, -2).contiguous())
    w = w.reshape(b, hkv, hq // hkv, Lq, -1).masked_fill(~seen[:, None, None], -math.inf)
    top = w.amax(-1, keepdim=True).clamp(min=-1e30)
    w = (w - top).exp()
    total = w.sum(-1, keepdim=True)
    o = (w.reshape(b, hkv, -1, cached + L) @ v).reshape(b, hkv, hq // hkv, Lq, d)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    return o.permute(0, 3, 1, 2, 4).reshape(b, Lq, hq, d).to(s["q"].dtype)


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        import mamba_selective_scan_04_amd as m
        if op == "scan":
            o, h, _ = m.delta_scan(s["q"], s["k"], s["v"], s["g"], s["beta"], scale=s["scale"], h_init=s["h"],
                                   lens=s["lens"])
            return dict(o=o, h=h)
        if op == "train":
            o, _, chunks = m.delta_scan(s["q"], s["k"], s["v"], s["g"], s["beta"], scale=s["scale"], h_init=s["h"],
                                        lens=s["lens"], want_chunks=True)
            out = m.delta_scan_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], chunks, s["do"], scale=s["scale"],
                                   lens=s["lens"], dh_final=s["dh"], want_dh_init=True)
            return dict(out, o=o)
        if op == "step":
            o = m.delta_step(s["h"], s["q"], s["k"], s["v"], s["g"], s["beta"], scale=s["scale"], lens=s["lens"],
                             h_out=s["h_out"])
            return dict(o=o, h=s["h_out"])
        cache = m.KvCache(s["kc"], s["ks"], s["vc"], s["vs"])
        if op == "commit":
            m.kv_commit(cache, s["k"], s["v"], s["table"], s["ctx"], lens=s["lens"])
            return dict(k=s["kc"], k_scale=s["ks"], v=s["vc"], v_scale=s["vs"])
        return m.kv_attn_step(cache, s["q"], s["k"], s["v"], s["table"], s["ctx"], lens=s["lens"],
                              causal=s["case"]["causal"], scale=s["scale"])
    if op in ("scan", "step"):
        o, h = _delta(s["q"], s["k"], s["v"], s["g"], s["beta"], s["scale"], s["h"], s["lens"])
        return dict(o=o.to(s["q"].dtype), h=h)
    if op == "train":
        return _plain_train(s)
    return _plain_commit(s) if op == "commit" else _plain_attn(s)


# ------------------------------------------------------------------- work

def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] in ("scan", "train", "step"):
        tok = c["batch"] * c["T"]
        qk, vo = tok * c["heads_k"] * c["dk"] * e, tok * c["heads_v"] * c["dv"] * e
        gate = tok * c["heads_v"] * 4
        state = c["batch"] * c["heads_v"] * c["dk"] * c["dv"] * 4
        # read the state, correct it, read it again: three products with dk x dv
        flops = 6 * tok * c["heads_v"] * c["dk"] * c["dv"]
        first = state if c["init"] else 0
        if c["op"] == "train":   # inputs, do and dh in; o, five gradients and dh_init out
            return dict(bytes=4 * qk + 4 * vo + 4 * gate + first + 2 * state, flops=3 * flops)
        return dict(bytes=2 * qk + 2 * vo + 2 * gate + first + state, flops=flops)
    if c["op"] == "commit":
        n = c["batch"] * (c["T"] // c["page"]) * c["page"] * c["heads_kv"] * c["d"] // (2 if c["ragged"] else 1)
        return dict(bytes=max(1, 2 * n * (e + 1)), flops=4 * n)
    ctx = c["batch"] * c["ctx"] * (5 / 8 if c["ragged"] else 1)
    new = c["batch"] * (2 * c["Lq"] * c["heads_q"] + 2 * c["L"] * c["heads_kv"]) * c["d"] * e
    keys = ctx + c["batch"] * c["L"]
    return dict(bytes=2 * ctx * c["heads_kv"] * c["d"] + new, flops=4 * keys * c["Lq"] * c["heads_q"] * c["d"])


# ------------------------------------------------------------------ exact

def _exact_delta(s, train):
    """Token by token in 64 bits, straight from the recurrence."""
    q, k, v, g, beta = (s[n].double() for n in ("q", "k", "v", "g", "beta"))
    b, T, hk, dk = k.shape
    hv, dv = v.shape[2:]
    rep = hv // hk
    n = s["lens"].clamp(0, T).tolist() if s["lens"] is not None else [T] * b
    for r in range(b):
        for x in (q, k, v, g, beta):
            x[r, n[r]:] = 0
    S = torch.zeros(b, hv, dk, dv, dtype=torch.float64, device=k.device) if s["h"] is None else s["h"].double()
    a = g.exp()
    at = lambda x, t: x[:, t].repeat_interleave(rep, 1)  # noqa: E731
    kept = torch.empty(T + 1, b, hv, dk, dv, dtype=torch.float64, device=k.device) if train else None
    o = torch.zeros(b, T, hv, dv, dtype=torch.float64, device=k.device)
    err = torch.zeros_like(o)
    for t in range(T):
        if train:
            kept[t] = S
        kt = at(k, t)
        S = a[:, t, :, None, None] * S
        y = v[:, t] - (kt[..., None] * S).sum(-2)
        err[:, t] = y
        S = S + kt[..., None] * (beta[:, t, :, None] * y)[..., None, :]
        o[:, t] = s["scale"] * (at(q, t)[..., None] * S).sum(-2)
    if not train:
        return dict(o=o, h=S)
    kept[T] = S
    do = s["do"].double()
    for r in range(b):
        do[r, n[r]:] = 0
    dS = s["dh"].double()
    dq = torch.zeros(b, T, hv, dk, dtype=torch.float64, device=k.device)
    dk_ = torch.zeros_like(dq)
    dv_, dg, db = torch.zeros_like(v), torch.zeros_like(g), torch.zeros_like(beta)
    for t in reversed(range(T)):
        qt, kt, dot, y, bt = at(q, t), at(k, t), do[:, t], err[:, t], beta[:, t, :, None]
        dq[:, t] = s["scale"] * (kept[t + 1] * dot[..., None, :]).sum(-1)
        dS = dS + s["scale"] * qt[..., None] * dot[..., None, :]
        du = (kt[..., None] * dS).sum(-2)
        db[:, t] = (du * y).sum(-1)
        dy = bt * du
        dv_[:, t] = dy
        decayed = a[:, t, :, None, None] * kept[t]
        dk_[:, t] = (dS * (bt * y)[..., None, :]).sum(-1) - (decayed * dy[..., None, :]).sum(-1)
        dS = dS - kt[..., None] * dy[..., None, :]
        dg[:, t] = (dS * decayed).sum((-1, -2))
        dS = a[:, t, :, None, None] * dS
    shared = lambda x: x.reshape(b, T, hk, rep, dk).sum(3)  # noqa: E731
    out = dict(o=o, dq=shared(dq), dk=shared(dk_), dv=dv_, dg=dg, dbeta=db, dh_init=dS)
    for r in range(b):
        for name in ("dq", "dk", "dv", "dg", "dbeta"):
            out[name][r, n[r]:] = 0
    return out


def _exact_commit(s):
    c = s["case"]
    out = {}
    for name, x, cache, scales in (("k", s["k"], s["kc"], s["ks"]), ("v", s["v"], s["vc"], s["vs"])):
        codes, sc = cache.double(), scales.double()
        lens = s["lens"].tolist() if s["lens"] is not None else [c["T"]] * c["batch"]
        for r in range(c["batch"]):
            blocks = lens[r] // c["page"]
            if not blocks:
                continue
            first = int(s["ctx"][r]) // c["page"]
            at = s["table"][r, first:first + blocks].long()
            y = x[r, : blocks * c["page"]].double().reshape(blocks, c["page"], c["heads_kv"], c["d"]).transpose(1, 2)
            step = (y.abs().flatten(2).max(-1).values / QMAX[c["code"]]).clamp(min=TINY)
            sc[at] = step
            z = y / step[..., None, None]
            z = z.round() if c["code"] == "i8" else z.float().to(CODE["e4m3"]).double()
            codes[at] = z if name == "k" else z.transpose(-1, -2)
        out[name], out[name + "_scale"] = (codes if c["code"] == "e4m3" else None), sc
    return out


def _exact_attn(s):
    c = s["case"]
    b, L, Lq, hq, hkv, d = (c[n] for n in ("batch", "L", "Lq", "heads_q", "heads_kv", "d"))
    o = torch.zeros(b, Lq, hq, d, dtype=torch.float64, device=DEV)
    for r in range(b):
        ctx = int(s["ctx"][r])
        n = L if s["lens"] is None else int(s["lens"][r])
        k, v = _gathered(s, r, r + 1, torch.float64)
        keys = torch.cat([k[0, :, :ctx], s["k"][r, :n].double().transpose(0, 1)], 1)
        vals = torch.cat([v[0, :, :ctx], s["v"][r, :n].double().transpose(0, 1)], 1)
        nq = min(n, Lq)
        for h in range(hq):
            K, V = keys[h // (hq // hkv)], vals[h // (hq // hkv)]
            w = s["scale"] * (s["q"][r, :nq, h].double() @ K.T)
            if c["causal"]:
                for i in range(nq):
                    w[i, ctx + n - nq + i + 1:] = -math.inf
            if w.numel():
                o[r, :nq, h] = torch.softmax(w, -1) @ V
    return o


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("scan", "step"):
        return _exact_delta(s, False)
    if case["op"] == "train":
        return _exact_delta(s, True)
    return _exact_commit(s) if case["op"] == "commit" else _exact_attn(s)
