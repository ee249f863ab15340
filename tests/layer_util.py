"""The short convolution and the residual norm in 64 bits, from their formulas, on
the CPU; seeded inputs and the tolerances of their tests.

Tolerances, with u = 2^-24 and each output's own rounding (half a step of its
type: bf16 2^-8, fp32 2^-24 of the value):
* p is a chain of W products and a bias, each step rounded: (W + 1) u S with
  S = |bias| + sum |w u|.  silu moves by at most 1.1 of p's error; its own
  operations leave (|p| + 6) u |y| (the exponent's argument |p| u, a reciprocal,
  a product and an exponential of one last bit or two each).
* silu's slope s (1 + p (1 - s)): 0.5 of p's error, and (6 |p| + 10) u of its own
  (1 - s keeps an absolute error of 4 u, which p multiplies).  dp = dy slope.
* du sums W products w dp: (W + 1) u sum |w dp| and w times each dp's error.
* dw and dbias sum dp times an input over all tokens.  A lane adds its chunks'
  tokens one after another, a workgroup its lanes' sums, and a last pass the
  workgroups': never more than 700 additions behind each other at the sizes here
  (64 tokens, 256 chunks of a workgroup, 16 + 16 parts, and the rows a part goes
  round), each rounding at most u of the terms' magnitudes.
* The norm's y and codes are exact: its definition is in 32 bits (r rounded from
  64) and so is the comparison, with r from a 64-bit sum.
* Its gradients: mean(g n) adds ch / 64 terms in a lane and joins 6 + 16 sums,
  (ch / 64 + 30) u mean |g n|; dh = r (g - n mean) + dh_out takes six roundings.
"""
import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DEPTH = 700


def conv_inputs(batch, T, ch, width, dtype, seed=0, device="cpu", lens=None, starts=None, extra=0, at=0, bias=True, init=True):
    gen = torch.Generator().manual_seed(3000 + seed)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    wide = rn(batch, T, ch + extra).to(dtype).to(device)
    c = dict(w=rn(ch, width), bias=rn(ch) * 0.3 if bias else None, c_init=rn(batch, width - 1, ch).to(dtype) if init else None,
             dy=rn(batch, T, ch).to(dtype), dc=rn(batch, width - 1, ch).to(dtype),
             lens=None if lens is None else torch.tensor(lens, dtype=torch.int32), starts=None)
    if starts is not None:
        c["starts"] = torch.zeros(batch, T, dtype=torch.bool)
        for b, t in starts:
            c["starts"][b, t] = True
    c = {n: x if x is None else x.to(device) for n, x in c.items()}
    return dict(c, u=wide[..., at:at + ch], wide=wide)


def conv_reference(c, silu=True):
    """-> {output: (value, bound on the error before its own rounding)} in 64 bits, row by row and token by token."""
    x = {n: t.detach().cpu() if t is not None else None for n, t in c.items()}
    batch, T, ch = x["u"].shape
    W = x["w"].shape[1]
    w = x["w"].double()
    bias = x["bias"].double() if x["bias"] is not None else torch.zeros(ch, dtype=torch.float64)
    z = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
    y, ey, du, edu = (z(batch, T, ch) for _ in range(4))
    dw, edw, db, edb = z(ch, W), z(ch, W), z(ch), z(ch)
    last, dci, edci = z(batch, W - 1, ch), z(batch, W - 1, ch), z(batch, W - 1, ch)
    for b in range(batch):
        n = T if x["lens"] is None else min(max(0, int(x["lens"][b])), T)
        first = x["c_init"][b].double() if x["c_init"] is not None else z(W - 1, ch)
        seq = torch.cat([first, x["u"][b, :n].double()])          # token t at t + W - 1
        grad, egrad = torch.zeros_like(seq), torch.zeros_like(seq)
        start = -10 ** 9                                          # of the document that token t is in
        for t in range(n):
            if x["starts"] is not None and x["starts"][b, t]:
                start = t
            p, S = bias.clone(), bias.abs()
            seen = [j for j in range(W) if t - (W - 1) + j >= start]
            for j in seen:
                p = p + w[:, j] * seq[t + j]
                S = S + (w[:, j] * seq[t + j]).abs()
            ep = (W + 1) * U * S
            sg = torch.sigmoid(p)
            y[b, t] = p * sg if silu else p
            ey[b, t] = 1.1 * ep + (p.abs() + 6) * U * y[b, t].abs() if silu else ep
            dy = x["dy"][b, t].double()
            dp = dy * sg * (1 + p * (1 - sg)) if silu else dy
            edp = dy.abs() * (0.5 * ep + (6 * p.abs() + 10) * U) if silu else 0 * dy
            for j in seen:
                grad[t + j] += w[:, j] * dp
                egrad[t + j] += w[:, j].abs() * (edp + (W + 1) * U * dp.abs())
                dw[:, j] += dp * seq[t + j]
                edw[:, j] += (edp + DEPTH * U * dp.abs()) * seq[t + j].abs()
            db += dp
            edb += edp + DEPTH * U * dp.abs()
        for j in range(W - 1):
            t = n - (W - 1) + j
            if t >= start:
                last[b, j] = seq[t + W - 1]
                grad[t + W - 1] += x["dc"][b, j].double()
                egrad[t + W - 1] += (W + 1) * U * x["dc"][b, j].double().abs()
        du[b, :n], edu[b, :n] = grad[W - 1:], egrad[W - 1:]
        dci[b], edci[b] = grad[:W - 1], egrad[:W - 1]
    return dict(y=(y, ey), c=(last, 0 * last), du=(du, edu), dw=(dw, edw), dbias=(db, edb), dc_init=(dci, edci))


def near(got, want, what=""):
    ref, err = want
    g = got.detach().cpu().double()
    assert g.shape == ref.shape, what
    assert torch.isfinite(g).all(), what
    bound = (1 + 2.0 ** -6) * (err + HALF[got.dtype] * (ref.abs() + err)) + 2.0 ** -126
    off = (g - ref).abs()
    assert (off <= bound).all(), (what, float((off / bound).max()))


def norm_inputs(rows, ch, dtype, res, seed=0, device="cpu"):
    gen = torch.Generator().manual_seed(4000 + seed)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    shape = (*rows, ch) if isinstance(rows, tuple) else (rows, ch)
    c = dict(x=(rn(*shape) * (0.1 + 3 * torch.rand(*shape[:-1], 1, generator=gen))).to(dtype),
             res=None if res is None else rn(*shape).to(res), w=1 + 0.3 * rn(ch), dy=rn(*shape).to(dtype),
             dh=rn(*shape).to(res or dtype))
    return {n: x if x is None else x.to(device) for n, x in c.items()}


def norm_definition(c, eps):
    """h, r and y (fp32, before its rounding to the stream's type) by the definition in 32 bits."""
    x = {n: t.detach().cpu() if t is not None else None for n, t in c.items()}
    h = x["x"] if x["res"] is None else (x["x"].float() + x["res"].float()).to(x["res"].dtype)
    r = ((h.double().square().mean(-1, keepdim=True) + eps) ** -0.5).float()
    return h, r[..., 0], (h.float() * r) * x["w"]


def norm_codes_definition(y, code, group):
    q = 448.0 if code == torch.float8_e4m3fn else 127.0
    g = y.reshape(*y.shape[:-1], -1, group or y.shape[-1])
    finite = torch.where(g.abs() < float("inf"), g.abs(), torch.zeros_like(g))
    scale = (finite.amax(-1) / q).clamp(min=2.0 ** -126)
    z = (g / scale[..., None]).reshape(y.shape)
    z = torch.where(z.isnan() & torch.tensor(code == torch.int8), torch.zeros_like(z), z).clamp(-q, q)
    codes = z.round().to(torch.int8) if code == torch.int8 else z.to(code)
    return codes, scale if group else scale[..., 0]


def norm_grads(c, h, r, with_dh):
    """-> {output: (value, bound)} in 64 bits."""
    x = {n: t.detach().cpu() if t is not None else None for n, t in c.items()}
    ch = h.shape[-1]
    h, r = h.detach().cpu().double(), r.detach().cpu().double()[..., None]
    dy, w = x["dy"].double(), x["w"].double()
    n, g = h * r, dy * w
    mean = (g * n).mean(-1, keepdim=True)
    emean = (ch / 64 + 30) * U * (g * n).abs().mean(-1, keepdim=True)
    d = r * (g - n * mean)
    ed = r * (n.abs() * emean + 6 * U * (g.abs() + (n * mean).abs()))
    if with_dh:
        d = d + x["dh"].double()
        ed = ed + 2 * U * (d.abs() + x["dh"].double().abs())
    dims = tuple(range(dy.dim() - 1))
    return dict(dx=(d, ed), dres=(d, ed), dw=((dy * n).sum(dims), (DEPTH + 2) * U * (dy * n).abs().sum(dims)))
