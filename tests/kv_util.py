"""The paged 8-bit cache and the attention over it in 64 bits, from their
definitions, on the CPU; seeded inputs and the tolerances of its tests.

Tolerances.  Codes and scales are exact: the definition is in 32 bits (a
product and a division, rounded to nearest), and so is the comparison.  Outputs:
* fp32: probabilities and values enter their product in three bf16 parts (all
  24 bits), scores are sums of head_dim products: with u = 2^-24 a score of
  magnitude s is off by up to (head_dim + 4) u sum|q k|, which moves its
  probability by that much relatively; sum|q k| scale is below 16 for the
  inputs here (N(0,1), d <= 128: mean 0.64 sqrt(d) = 7.2).  The exponential adds
  2 u s.  132 * 16 u + (keys' sum) 64 u = 1.3e-4 is the worst arrangement;
  independent roundings give its square root in the count, sqrt(132) * 16 u =
  1.1e-5.  2e-5 of the tensor's norm is held.
* bf16: the result's rounding is off by at most half a step, 2^-8 |o| (times
  1 + 2^-7 for what is of second order).  Each probability (with its page's scale)
  enters its product in two bf16 parts, off by at most 2^-16 of itself, and its
  score's 32-bit sum moves it by the 1.3e-4 < 2^-12.9 above: o = sum p v moves by
  at most 2^-12 sum p |v|.  Both by element, with sum p |v| in 64 bits.
"""
import torch


def inputs(batch, ctx, L, Lq, hq, hkv, d, page, code, dtype, seed=0, device="cpu", lens=None, extra=3):
    gen = torch.Generator().manual_seed(2000 + seed)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    per = max(1, -(-max(ctx) // page))
    n = batch * per + extra
    table = torch.randperm(n, generator=gen)[: batch * per].reshape(batch, per).to(torch.int32)

    def codes(*shape):
        if code == torch.int8:
            return torch.randint(-127, 128, shape, generator=gen, dtype=torch.int8)
        return (rn(*shape) * 120).clamp(-448, 448).to(code)

    unit = 1 / (73 if code == torch.int8 else 120)
    c = dict(k=codes(n, hkv, page, d), v=codes(n, hkv, d, page),
             ks=unit * (0.25 + torch.rand(n, hkv, generator=gen)), vs=unit * (0.25 + torch.rand(n, hkv, generator=gen)),
             q=rn(batch, Lq, hq, d).to(dtype), nk=rn(batch, L, hkv, d).to(dtype), nv=rn(batch, L, hkv, d).to(dtype),
             table=table, ctx=torch.tensor(ctx, dtype=torch.int32),
             lens=None if lens is None else torch.tensor(lens, dtype=torch.int32))
    return {n_: x if x is None else x.to(device).contiguous() for n_, x in c.items()}


def attend(c, causal=False, scale=None):
    """-> o and sum p |v|, [batch, Lq, heads_q, d] fp64."""
    x = {n: t.detach().cpu() if t is not None else None for n, t in c.items()}
    batch, Lq, hq, d = x["q"].shape
    L, hkv = x["nk"].shape[1:3]
    n_pages, page = x["k"].shape[0], x["k"].shape[2]
    scale = d ** -0.5 if scale is None else scale
    o = torch.zeros(batch, Lq, hq, d, dtype=torch.float64)
    size = torch.zeros_like(o)
    for b in range(batch):
        ctx = min(max(0, int(x["ctx"][b])), x["table"].shape[1] * page)
        n = L if x["lens"] is None else min(max(0, int(x["lens"][b])), L)
        nq = min(n, Lq)
        at = [t for t in range(ctx) if 0 <= int(x["table"][b, t // page]) < n_pages]
        ids = torch.tensor([int(x["table"][b, t // page]) for t in at], dtype=torch.long)
        off = torch.tensor([t % page for t in at], dtype=torch.long)
        for h in range(hq):
            hk = h // (hq // hkv)
            K = x["k"].float().double()[ids, hk, off] * x["ks"].double()[ids, hk][:, None]
            V = x["v"].float().double()[ids, hk, :, off] * x["vs"].double()[ids, hk][:, None]
            K = torch.cat([K, x["nk"][b, :n, hk].double()])
            V = torch.cat([V, x["nv"][b, :n, hk].double()])
            for i in range(nq):
                seen = len(at) + (n - nq + i + 1 if causal else n)
                if seen:
                    w = torch.softmax(scale * (K[:seen] @ x["q"][b, i, h].double()), 0)
                    o[b, i, h] = w @ V[:seen]
                    size[b, i, h] = w @ V[:seen].abs()
    return o, size


def check(got, want, what=""):
    ref, size = want
    g = got.detach().cpu().double()
    assert torch.isfinite(g).all(), what
    off = (g - ref).abs()
    if got.dtype == torch.bfloat16:
        assert (off <= (1 + 2.0 ** -7) * 2.0 ** -8 * ref.abs() + 2.0 ** -12 * size).all(), (what, float(off.max()))
    else:
        assert off.norm() <= 2e-5 * ref.norm(), (what, float(off.norm() / ref.norm()))
