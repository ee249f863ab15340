"""Gradients of the gated delta rule where decays are strong, against the
recurrence's in 64 bits.

dg_t is what crosses token t: <dS_t, a_t S_{t-1}> with S_{t-1} the state before
it and dS_t the adjoint of the decayed state.  As a product of two 32-bit sums
(TOL32 of each one's norm) it may be off by 2 TOL32 a_t |dS_t| |S_{t-1}|,
however small that is beside the other tokens' gradients; where a token clears
the state, a_t = 0 and dg_t is exactly 0.  The decay itself is off by at most
(|g| + |g| log2(e)) 2^-24 < 2.5 |g| 2^-24 of itself (the argument's rounding to
32 bits and that of its product with log2(e)): 150 2^-24 at |g| = 60, within the
272 2^-24 of TOL32.
"""
import math

import pytest
import torch

import mamba_selective_scan_04_amd as m
from delta_util import TOL32, check, inputs, reference

NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dh_init")
DTYPES = [torch.float32, torch.bfloat16]


def crossing(c):
    """-> dg and a_t |dS_t| |S_{t-1}|, [batch, T, heads_v] fp64, from c['h'] on."""
    q, k, v, g, beta, do = (c[n].detach().cpu().double() for n in ("q", "k", "v", "g", "beta", "do"))
    batch, T, hk, dk = k.shape
    rep = v.shape[2] // hk
    q, k = q.repeat_interleave(rep, 2), k.repeat_interleave(rep, 2)
    a = torch.exp(g)[..., None, None]
    dg, size = torch.zeros_like(g), torch.zeros_like(g)
    for b in range(batch):
        S, states = c["h"][b].detach().cpu().double(), []
        for t in range(T):
            states.append(S)
            S = a[b, t] * S
            y = v[b, t] - torch.einsum("hkv,hk->hv", S, k[b, t])
            S = S + torch.einsum("hk,hv->hkv", k[b, t], beta[b, t][:, None] * y)
        dS = c["dh"][b].detach().cpu().double()
        for t in reversed(range(T)):
            dS = dS + dk ** -0.5 * torch.einsum("hk,hv->hkv", q[b, t], do[b, t])
            dy = beta[b, t][:, None] * torch.einsum("hkv,hk->hv", dS, k[b, t])
            dS = dS - torch.einsum("hk,hv->hkv", k[b, t], dy)
            decayed = a[b, t] * states[t]
            dg[b, t] = (dS * decayed).sum((-1, -2))
            size[b, t] = dS.flatten(1).norm(dim=1) * decayed.flatten(1).norm(dim=1)
            dS = a[b, t] * dS
    return dg, size


def gradients(c):
    args = c["q"], c["k"], c["v"], c["g"], c["beta"]
    _, _, chunks = m.delta_scan(*args, h_init=c["h"], want_chunks=True)
    return m.delta_scan_bwd(*args, chunks, c["do"], dh_final=c["dh"], want_dh_init=True)


def check_each(c):
    got, ref = gradients(c), reference(c, h=c["h"], want_grads=True)
    for n in NAMES:
        check(got[n], ref[n], n, 2.0)
    dg, size = crossing(c)
    worst = ((got["dg"].cpu().double() - dg).abs() / (2 * TOL32 * size + 1e-37)).max()   # 1e-37: below 32 bits' range
    assert worst <= 1, float(worst)
    cleared = c["g"] == -math.inf
    assert (got["dg"][cleared] == 0).all()


def test_crossing_is_the_gradient():
    c = inputs(2, 70, 1, 2, 64, 64, torch.float32, seed=50, resets=[7])
    dg, size = crossing(c)
    ref = reference(c, h=c["h"], want_grads=True)["dg"]
    assert (dg - ref).abs().max() <= 1e-12 * ref.abs().max() and (dg.abs() <= size * (1 + 1e-12)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("decay", [-20.0, 3.0, 8.0, 16.0, 60.0])
@pytest.mark.parametrize("size", [(1, 150, 1, 2, 64, 64), (1, 130, 2, 2, 128, 128), (2, 70, 1, 3, 64, 128), (1, 129, 2, 2, 128, 64)])
def test_every_decay(dev, size, decay, dtype):
    check_each(inputs(*size, dtype, seed=51, device=dev, decay=decay))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads", [(1, 2, 128, 128), (2, 2, 64, 64)])
def test_strong_tokens_among_slow_ones(dev, heads, dtype):
    """Single tokens that nearly clear the state, others that do, and a fast head beside a slow one."""
    c = inputs(1, 200, *heads, dtype, seed=52, device=dev, resets=[0, 63, 100])
    for t, g in ((20, -16.0), (21, -16.0), (64, -30.0), (127, -50.0), (150, -8.0)):
        c["g"][:, t] = g
    c["g"][:, :, 1] *= 100
    check_each(c)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_segments(dev, dtype, monkeypatch):
    monkeypatch.setenv("BDSSM_DELTA_SEGMENTS", "3")
    c = inputs(1, 330, 1, 2, 64, 128, dtype, seed=53, device=dev, decay=3.0, resets=[100])
    c["g"][:, ::7] *= 4
    check_each(c)
