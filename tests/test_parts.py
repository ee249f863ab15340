"""fp32 operands on bf16 matrix instructions: what the parts leave out.

Three parts, each rounded to nearest, hold an fp32 value; a second part is at
most 2^-8 and a third at most 2^-17 of it.  The six products of parts i, j with
i + j <= 2 leave out a1 b2 + a2 b1 + a2 b2 <= 2^-24 + 2^-34 of a b, and the sum's
rounding adds at most a step, 2^-23 (half of one if it is to nearest).  Two parts
leave out at most 2^-17 of the value; a bf16 result adds half of its step."""
import pytest
import torch

import mamba_selective_scan_04_amd as m

pytestmark = pytest.mark.gpu


def test_product_of_two_fp32_values(dev):
    """o = q.k v with one channel of q and k, from no state: the one product as it is."""
    gen = torch.Generator().manual_seed(70)
    n, hv = 512, 16
    x, y = (0.5 + 0.5 * torch.rand(n, 1, hv, generator=gen) for _ in range(2))
    x[:, :, 0] = y[:, :, 0] = (1 + 2.0 ** -7 - 2.0 ** -23) / 2
    q, k = (torch.zeros(n, 1, hv, 64) for _ in range(2))
    q[..., 5], k[..., 5] = x, y
    v, one = torch.ones(n, 1, hv, 64), torch.ones(n, 1, hv)
    o, _, _ = m.delta_scan(q.to(dev), k.to(dev), v.to(dev), (one * 0).to(dev), one.to(dev), scale=1.0)
    want = (x.double() * y.double())[..., None]
    off = (o.cpu().double() / want - 1).abs().max()
    assert off <= 2.0 ** -23 + 2.0 ** -24 + 2.0 ** -34, float(off)


@pytest.mark.parametrize("T", [1, 16])
def test_state_into_bf16_outputs(dev, T):
    """o = S q with one row of the state, near the middle between two bf16 values: the nearer
    one, but for values within 2^-17 of the middle."""
    gen = torch.Generator().manual_seed(71)
    hv, dv = 16, 128
    S = torch.zeros(1, hv, 64, dv)
    mid = 1 + (2 * torch.randint(0, 128, (hv, dv), generator=gen) + 1) * 2.0 ** -8
    S[0, :, 9] = mid + (torch.rand(hv, dv, generator=gen) - 0.5) * 2.0 ** -14
    q = torch.zeros(1, T, 1, 64)
    q[..., 9] = 1
    z = torch.zeros(1, T, hv)
    args = [x.to(dev) for x in (q.bfloat16(), torch.zeros_like(q).bfloat16(), torch.zeros(1, T, hv, dv).bfloat16(), z, z)]
    o = m.delta_step(S.to(dev), *args, scale=1.0) if T > 1 else m.delta_scan(*args, scale=1.0, h_init=S.to(dev))[0]
    want = S[:, :, 9].double()[:, None]
    off = (o.cpu().double() - want).abs() - 2.0 ** -8
    assert (off <= 2.0 ** -17 * want).all(), float((off / want).max())
