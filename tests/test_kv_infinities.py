"""Attention over active values that hold infinities and NaN: a channel of a
query's output is the sum of p v over what it sees, so one sign of infinity
there is that infinity, both or a NaN are a NaN, and other channels and queries
are as without them."""
import pytest
import torch

from kv_util import attend, check, inputs
from test_parity_kv import E4M3, I8, run

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d,L,Lq,lens,code", [(64, 1, 1, None, I8), (128, 40, 40, None, E4M3), (64, 70, 7, [70, 37], I8),
                                              (128, 33, 33, [5, 33], I8), (128, 16, 16, None, E4M3)])
def test_visible_values(dev, d, L, Lq, lens, code, dtype, causal):
    c = inputs(2, [50, 0], L, Lq, 4, 2, d, 16, code, dtype, seed=60, device=dev, lens=lens)
    want, size = attend(c, causal)
    n = [L, L] if lens is None else lens
    # (row, token from the row's last, channel of key head 1, value)
    special = [(b, back, ch, x) for b in range(2) for back, ch, x in
               ((0, 3, INF), (1, 3, INF), (0, 9, -INF), (2, 17, INF), (2, 18, -INF), (1, 40, INF), (3, 40, -INF), (2, 41, NAN))
               if back < n[b]]
    for b, back, ch, x in special:
        c["nv"][b, n[b] - 1 - back, 1, ch] = x
    o = run(c, causal=causal).cpu()
    free = torch.ones(2, d, dtype=torch.bool)
    for b in range(2):
        nq = min(Lq, n[b])
        for ch in {s[2] for s in special if s[0] == b}:
            free[b, ch] = False
            at = [(n[b] - 1 - back, x) for r, back, y, x in special if r == b and y == ch]
            for i in range(nq):
                seen = [x for t, x in at if not causal or t <= n[b] - nq + i]
                for h in (2, 3):                     # the query heads of key head 1
                    got = o[b, i, h, ch].double()
                    if not seen:
                        near = 2.0 ** -7 * want[b, i, h, ch].abs() + 2.0 ** -12 * size[b, i, h, ch] + 1e-6
                        assert (got - want[b, i, h, ch]).abs() <= near, (b, i, h, ch)
                    elif len(set(map(str, seen))) == 1 and seen[0] == seen[0]:
                        assert got == seen[0], (b, i, h, ch, float(got))
                    else:
                        assert got != got, (b, i, h, ch, float(got))
        others = [x[b:b + 1, :, 2:][..., free[b]] for x in (want, size)]
        check(o[b:b + 1, :, 2:][..., free[b]], others)
        check(o[b:b + 1, :, :2], [x[b:b + 1, :, :2] for x in (want, size)])


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("causal", [False, True])
def test_behind_a_context_in_ranges(dev, monkeypatch, splits, causal):
    monkeypatch.setenv("BDSSM_KV_SPLITS", str(splits))
    c = inputs(1, [900], 8, 8, 4, 2, 64, 32, I8, torch.bfloat16, seed=61, device=dev)
    want, size = attend(c, causal)
    c["nv"][0, 0, :, 5] = -INF
    o = run(c, causal=causal).cpu()
    assert (o[..., 5] == -INF).all()
    keep = [x for x in range(64) if x != 5]
    check(o[..., keep], (want[..., keep], size[..., keep]))
