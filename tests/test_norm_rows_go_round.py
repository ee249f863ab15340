"""The norm where each workgroup takes several rows, in every layout of a row: outputs, both kinds of codes and the
gradients of all rows against their definitions.

r is held to its 64-bit value's rounding (where sums in another order decide a tie, to either one), y and the codes to
equality, given r.  Additions behind each other in dw (layer_util's 700): the rows of a workgroup, at most 5 here, four
waves, 64 parts of a wave and 16 waves."""
import pytest
import torch

import mamba_selective_scan_04_amd as m
from large_util import near, norm_codes_definition, norm_definition, norm_grads, rounds_to

F32, BF16 = torch.float32, torch.bfloat16
TYPES = [(BF16, None), (BF16, BF16), (BF16, F32), (F32, None), (F32, F32)]
EPS = 1e-5


def rows_of(ch):
    """More than two rows for each of the at most 2,048 workgroups, which take four at a time up to 1,024 channels."""
    return 2 * 2048 * 4 + 37 if ch <= 1024 else 2 * 2048 + 37


def inputs(dev, ch, dtype, res, seed):
    gen = torch.Generator(device=dev).manual_seed(8000 + seed)
    rows = rows_of(ch)
    rn = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    return dict(x=(rn(rows, ch) * (0.1 + 3 * torch.rand(rows, 1, generator=gen, device=dev))).to(dtype),
                res=None if res is None else rn(rows, ch).to(res), w=1 + 0.3 * rn(ch), dy=rn(rows, ch).to(dtype), dh=rn(rows, ch).to(res or dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,res", TYPES)
@pytest.mark.parametrize("ch", [40, 300, 700, 1000, 1500, 4000, 5003, 8192, 9000])
def test_norm_and_gradients(dev, ch, dtype, res):
    c = inputs(dev, ch, dtype, res, ch)
    h, r = norm_definition(c, EPS)
    gy, gh, gr = m.rms_norm(c["x"], c["w"], res=c["res"], eps=EPS, want_rstd=True)
    assert torch.equal(gh, h) and rounds_to(gr, r).all()
    assert torch.equal(gy, ((h.float() * gr[:, None]) * c["w"]).to(dtype))
    g = m.rms_norm_bwd(gh, c["w"], gr, c["dy"], dh=c["dh"])
    for n, want in norm_grads(c, h, gr).items():
        near(g[n], want, n)
    if res is not None:        # in place: a row's residual is read ahead, while the row before is worked on
        mine = c["res"].clone()
        y2, h2, _ = m.rms_norm(c["x"], c["w"], res=mine, eps=EPS, h=mine)
        assert h2 is mine and torch.equal(mine, h) and torch.equal(y2, gy)


@pytest.mark.gpu
@pytest.mark.parametrize("code", [torch.float8_e4m3fn, torch.int8])
@pytest.mark.parametrize("dtype,res", [(BF16, None), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("ch,group", [(40, 0), (256, 128), (300, 0), (640, 128), (700, 0), (1000, 0), (1024, 128), (1500, 0), (1536, 128), (4000, 0),
                                      (4096, 128), (5003, 0), (8064, 128), (8192, 0), (9000, 0), (8960, 128)])
def test_codes(dev, ch, group, dtype, res, code):
    c = inputs(dev, ch, dtype, res, ch + group)
    gr = m.rms_norm(c["x"], c["w"], res=c["res"], eps=EPS, want_rstd=True)[2]
    h, r = norm_definition(c, EPS)
    assert rounds_to(gr, r).all()
    codes, scales = norm_codes_definition((h.float() * gr[:, None]) * c["w"], code, group)
    got, gs, gh = m.rms_norm_codes(c["x"], c["w"], res=c["res"], eps=EPS, code=code, group=group)
    assert torch.equal(gs, scales) and torch.equal(gh, h)
    assert torch.equal(got.view(torch.int8), codes.view(torch.int8))
