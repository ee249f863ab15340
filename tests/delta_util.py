"""The gated delta rule in 64 bits, token by token from its definition, with
its gradients, on the CPU; seeded inputs and the tolerances of its tests.

Tolerances, derived from the arithmetic:
* fp32 results (states, fp32 outputs, dg, dbeta): a value is a sum of at most
  d_k + 2 * 64 products (a row of the state's product and of the chunk's two
  triangular ones) whose fp32 roundings are 2^-24 of the running sum each, on
  operands split with at most 2^-23 left out: (128 + 128 + 16) 2^-24 = 1.6e-5 of
  the tensor's norm.  Later chunks add no factor: the state's transition
  (decay, then I - beta k k^T with |k| = 1, beta < 1) does not expand errors.
  Gradients run through the forward's products and their transposes: twice.
* bf16 results: half a step of the result (2^-8 of it) and operands in two
  parts, 2^-15 of each of a sum's terms.  The terms' root mean square is at
  most the tensor's rms times sqrt(n) when they cancel to it, and their
  absolute sum sqrt(n) more: 2^-15 n <= 2^-7.4 in the worst arrangement, 2^-10
  for terms of independent sign (n = 256, sqrt(n) = 16): 2^-10 rms is used
  with the test's independent inputs.
"""
import math

import torch

TOL32 = (128 + 128 + 16) * 2.0 ** -24
HALF_BF16 = 2.0 ** -8


def inputs(batch, T, hk, hv, dk, dv, dtype, seed=0, device="cpu", decay=-4.0, resets=(), lens=None):
    gen = torch.Generator().manual_seed(1000 + seed)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    q, k = unit(rn(batch, T, hk, dk)), unit(rn(batch, T, hk, dk) + 0.3 * rn(1, 1, hk, dk))
    g = -torch.nn.functional.softplus(rn(batch, T, hv) * 1.5 + decay)
    for t in resets:
        g[:, t] = -math.inf
    c = dict(q=q.to(dtype), k=k.to(dtype), v=rn(batch, T, hv, dv).to(dtype), g=g,
             beta=torch.sigmoid(rn(batch, T, hv)), h=0.1 * rn(batch, hv, dk, dv), do=rn(batch, T, hv, dv).to(dtype),
             dh=0.1 * rn(batch, hv, dk, dv),
             lens=None if lens is None else torch.tensor(lens, dtype=torch.int32))
    return {n: x if x is None else x.to(device).contiguous() for n, x in c.items()}


def reference(c, scale=None, h=None, want_grads=False):
    """-> dict(o, h, chunks [batch, n, hv, dv, dk]) and, if asked, the gradients
    given c['do'], c['dh'] (their padding ignored), all fp64 on the CPU."""
    q, k, v, g, beta, do = (c[n].detach().cpu().double() for n in ("q", "k", "v", "g", "beta", "do"))
    batch, T, hk, dk = k.shape
    hv, dv = v.shape[2:]
    scale = dk ** -0.5 if scale is None else scale
    rep = hv // hk
    n = [T] * batch if c["lens"] is None else c["lens"].cpu().clamp(0, T).tolist()
    out = dict(o=torch.zeros(batch, T, hv, dv, dtype=torch.float64), h=torch.zeros(batch, hv, dk, dv, dtype=torch.float64),
               chunks=torch.zeros(batch, -(-T // 64), hv, dv, dk, dtype=torch.float64))
    for name, like in (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dbeta", beta)):
        out[name] = torch.zeros_like(like)
    out["dh_init"] = torch.zeros_like(out["h"])
    for b in range(batch):
        S = torch.zeros(hv, dk, dv, dtype=torch.float64) if h is None else h[b].detach().cpu().double()
        Q, K = q[b].repeat_interleave(rep, 1), k[b].repeat_interleave(rep, 1)
        before, err = [], []
        for t in range(-(-T // 64) * 64):
            if t % 64 == 0:
                out["chunks"][b, t // 64] = S.transpose(-1, -2)
            if t >= n[b]:
                continue
            before.append(S)
            S = torch.exp(g[b, t])[:, None, None] * S
            y = v[b, t] - torch.einsum("hkv,hk->hv", S, K[t])
            err.append(y)
            S = S + torch.einsum("hk,hv->hkv", K[t], beta[b, t][:, None] * y)
            out["o"][b, t] = scale * torch.einsum("hkv,hk->hv", S, Q[t])
        out["h"][b] = S
        if not want_grads:
            continue
        dS = c["dh"][b].detach().cpu().double() if c["dh"] is not None else torch.zeros_like(S)
        before.append(S)
        for t in reversed(range(n[b])):
            dot = do[b, t]
            dq = scale * torch.einsum("hkv,hv->hk", before[t + 1], dot)
            dS = dS + scale * torch.einsum("hk,hv->hkv", Q[t], dot)
            du = torch.einsum("hkv,hk->hv", dS, K[t])
            a = torch.exp(g[b, t])[:, None, None]
            decayed = a * before[t]
            out["dbeta"][b, t] = (du * err[t]).sum(-1)
            dy = beta[b, t][:, None] * du
            out["dv"][b, t] = dy
            dk_ = torch.einsum("hkv,hv->hk", dS, beta[b, t][:, None] * err[t]) - torch.einsum("hkv,hv->hk", decayed, dy)
            dS = dS - torch.einsum("hk,hv->hkv", K[t], dy)
            out["dg"][b, t] = (dS * decayed).sum((-1, -2))
            dS = a * dS
            out["dq"][b, t] = dq.reshape(hk, rep, dk).sum(1)
            out["dk"][b, t] = dk_.reshape(hk, rep, dk).sum(1)
        out["dh_init"][b] = dS
    return out


def check(got, ref, what="", factor=1.0):
    """fp32 or bf16 result against 64 bits, by the tolerances above."""
    g, r = got.detach().cpu().double(), ref.double()
    assert g.shape == r.shape, (what, g.shape, r.shape)
    if not r.numel():
        return
    assert torch.isfinite(g).all(), what
    norm, rms = r.norm(), r.norm() / math.sqrt(r.numel())
    off = (g - r).norm() / norm if norm > 0 else (g - r).norm()
    if got.dtype == torch.bfloat16:
        worst = ((g - r).abs() - HALF_BF16 * r.abs()).max()
        assert worst <= factor * 2.0 ** -10 * rms, (what, float(worst / rms), float(off))
    else:
        assert off <= factor * TOL32, (what, float(off))
        assert (g - r).abs().max() <= 16 * factor * TOL32 * torch.maximum(r.abs(), rms).max(), (what, float(off))
