"""Attention beside the type's largest and lowest values, as buffers are filled
with: where a query does not see them nothing of them reaches it, and where it
does its output is p v, in fp32 too, whose largest value bf16 rounds to infinity."""
import pytest
import torch

from kv_util import attend, check, inputs
from test_parity_kv import E4M3, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d,Lq", [(64, 40), (128, 7), (128, 40)])
@pytest.mark.parametrize("sign", [1, -1])
def test_hidden_tokens(dev, d, Lq, dtype, sign):
    c = inputs(2, [50, 0], 40, Lq, 4, 2, d, 16, E4M3, dtype, seed=90, device=dev)
    want, at = attend(c, True), 37
    c["nk"][:, at:] = c["nv"][:, at:] = sign * torch.finfo(dtype).max
    seen = slice(0, at - (40 - Lq))
    check(run(c, causal=True)[:, seen], [x[:, seen] for x in want])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("causal", [False, True])
def test_visible_tokens(dev, dtype, causal):
    """One token's value in one step of keys: p <= 1, and p v is in range.  Its weight is as any other's
    (score and exponential off by 2^-12.9, as the other tests have it), its rounding the type's."""
    c = inputs(1, [0], 16, 16, 2, 1, 64, 16, E4M3, dtype, seed=91, device=dev)
    c["nv"][0, 0, 0, 3], c["nv"][0, 0, 0, 9] = torch.finfo(dtype).max, -torch.finfo(dtype).max
    want, _ = attend(c, causal)
    o = run(c, causal=causal).cpu().double()
    for ch in (3, 9):
        off = (o[..., ch] / want[..., ch] - 1).abs().max()
        assert off <= 2.0 ** -12 + 2.0 ** -8 * (dtype == torch.bfloat16), float(off)
    keep = [x for x in range(64) if x not in (3, 9)]
    check(o[..., keep].to(dtype), [x[..., keep] for x in attend(c, causal)])
