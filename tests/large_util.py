"""The convolution and the norm in 64 bits from their formulas, all tokens or rows at once and where the inputs are:
for sizes whose reference token by token would take too long.  Tolerances as in layer_util."""
import torch

from layer_util import DEPTH, HALF, U


def near(got, want, what=""):
    ref, err = want
    g = got.detach().double()
    assert g.shape == ref.shape, what
    assert torch.isfinite(g).all(), what
    bound = (1 + 2.0 ** -6) * (err + HALF[got.dtype] * (ref.abs() + err)) + 2.0 ** -126
    off = (g - ref).abs()
    assert (off <= bound).all(), (what, float((off / bound).max()))


def conv_reference(c, silu):
    """-> {output: (value, bound on the error before its own rounding)}, as layer_util's."""
    u, w, dy, dc = (c[n].double() for n in ("u", "w", "dy", "dc"))
    batch, T, ch = u.shape
    W, dev = w.shape[1], u.device
    bias = c["bias"].double() if c["bias"] is not None else u.new_zeros(ch)
    first = c["c_init"].double() if c["c_init"] is not None else u.new_zeros(batch, W - 1, ch)
    n = torch.full((batch,), T, device=dev) if c["lens"] is None else c["lens"].long().clamp(0, T)
    there = (torch.arange(T, device=dev) < n[:, None])[..., None]
    zero = u.new_zeros(())
    seq = torch.cat([first, torch.where(there, u, zero)], 1)                   # token t at t + W - 1
    dy = torch.where(there, dy, zero)
    doc = torch.zeros(batch, T + W - 1, dtype=torch.long, device=dev)          # which document of the row
    if c["starts"] is not None:
        doc[:, W - 1:] = (c["starts"] & there[..., 0]).long().cumsum(1)
    seen = [(doc[:, j:j + T] == doc[:, W - 1:])[..., None] for j in range(W)]
    p, S = bias.expand(batch, T, ch).clone(), bias.abs().expand(batch, T, ch).clone()
    for j in range(W):
        term = torch.where(seen[j], w[:, j] * seq[:, j:j + T], zero)
        p += term
        S += term.abs()
    ep = (W + 1) * U * S
    sg = torch.sigmoid(p)
    y = p * sg if silu else p
    ey = 1.1 * ep + (p.abs() + 6) * U * y.abs() if silu else ep
    dp = dy * sg * (1 + p * (1 - sg)) if silu else dy
    edp = dy.abs() * (0.5 * ep + (6 * p.abs() + 10) * U) if silu else torch.zeros_like(dy)
    grad, egrad = torch.zeros_like(seq), torch.zeros_like(seq)
    dw, edw = torch.zeros_like(w), torch.zeros_like(w)
    per = edp + DEPTH * U * dp.abs()
    for j in range(W):
        mine = torch.where(seen[j], dp, zero)
        grad[:, j:j + T] += w[:, j] * mine
        egrad[:, j:j + T] += w[:, j].abs() * torch.where(seen[j], edp + (W + 1) * U * dp.abs(), zero)
        dw[:, j] = (mine * seq[:, j:j + T]).sum((0, 1))
        edw[:, j] = (torch.where(seen[j], per, zero) * seq[:, j:j + T].abs()).sum((0, 1))
    at = n[:, None] + torch.arange(W - 1, device=dev)                          # the last W - 1 inputs
    same = (doc.gather(1, at) == doc.gather(1, (n + W - 2)[:, None]))[..., None]
    idx = at[..., None].expand(-1, -1, ch)
    last = torch.where(same, seq.gather(1, idx), zero)
    grad.scatter_add_(1, idx, torch.where(same, dc, zero))
    egrad.scatter_add_(1, idx, torch.where(same, (W + 1) * U * dc.abs(), zero))
    inside = lambda x: torch.where(there, x[:, W - 1:], zero)  # noqa: E731
    return dict(y=(torch.where(there, y, zero), torch.where(there, ey, zero)), c=(last, torch.zeros_like(last)),
                du=(inside(grad), inside(egrad)), dw=(dw, edw), dbias=(dp.sum((0, 1)), per.sum((0, 1))),
                dc_init=(grad[:, :W - 1], egrad[:, :W - 1]))


def norm_definition(c, eps):
    """h, and r in 64 bits."""
    h = c["x"] if c["res"] is None else (c["x"].float() + c["res"].float()).to(c["res"].dtype)
    return h, (h.double().square().mean(-1) + eps) ** -0.5


def rounds_to(got, exact):
    """got is exact rounded to fp32, where 2^-48 of exact to either side (64-bit sums in another order) may decide a tie."""
    return (got == (exact * (1 - 2.0 ** -48)).float()) | (got == (exact * (1 + 2.0 ** -48)).float())


def norm_codes_definition(y, code, group):
    """Codes and scales of y.  Quotients of fp32 values formed in 64 bits round to fp32 as fp32 divisions do."""
    q = 448.0 if code == torch.float8_e4m3fn else 127.0
    g = y.reshape(*y.shape[:-1], -1, group or y.shape[-1])
    scale = (g.abs().amax(-1).double() / q).float().clamp(min=2.0 ** -126)
    z = (g.double() / scale.double()[..., None]).float().reshape(y.shape).clamp(-q, q)
    codes = z.round().to(torch.int8) if code == torch.int8 else z.to(code)
    return codes, scale if group else scale[..., 0]


def norm_grads(c, h, r):
    """-> {output: (value, bound)}."""
    ch = h.shape[-1]
    h, r, dy, w, dh = h.double(), r.double()[..., None], c["dy"].double(), c["w"].double(), c["dh"].double()
    n, g = h * r, dy * w
    mean = (g * n).mean(-1, keepdim=True)
    emean = (ch / 64 + 30) * U * (g * n).abs().mean(-1, keepdim=True)
    d = r * (g - n * mean) + dh
    ed = r * (n.abs() * emean + 6 * U * (g.abs() + (n * mean).abs())) + 2 * U * (d.abs() + dh.abs())
    return dict(dx=(d, ed), dres=(d, ed), dw=((dy * n).sum(0), (DEPTH + 2) * U * (dy * n).abs().sum(0)))
