"""Gradients of the convolution at padding where a weight is infinite or a NaN: 0 as anywhere in padding (a tap's
weight times no gradient is no product to form there), and elsewhere what they are without the padding."""
import pytest
import torch

import mamba_selective_scan_04_amd as m
from layer_util import conv_inputs


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("ch", [8, 5])
@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("starts", [False, True])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_padding_has_no_gradient(dev, dtype, ch, width, starts, bad):
    T, lens = 41, [0, 1, 2, 7, 30, 40, 41]
    c = conv_inputs(len(lens), T, ch, width, dtype, seed=30 + width, device=dev, lens=lens, starts=[(4, 9), (4, 29)] if starts else None)
    clean = m.conv_scan_bwd(c["u"], c["w"], c["dy"], bias=c["bias"], lens=c["lens"], starts=c["starts"], c_init=c["c_init"],
                            dc_final=c["dc"], want_dc_init=True)
    for j in range(width):
        w = c["w"].clone()
        w[2, j] = bad
        kw = dict(bias=c["bias"], lens=c["lens"], starts=c["starts"], c_init=c["c_init"], dc_final=c["dc"])
        for want_dc_init in (False, True):
            g = m.conv_scan_bwd(c["u"], w, c["dy"], want_dc_init=want_dc_init, **kw)
            for b, n in enumerate(lens):
                assert (g["du"][b, n:] == 0).all(), (j, b)
                one = {k: x if x is None or k == "bias" else x[b:b + 1, :n].clone() if k == "starts" else x[b:b + 1].clone()
                       for k, x in kw.items() if k != "lens"}
                alone = m.conv_scan_bwd(c["u"][b:b + 1, :n].clone(), w, c["dy"][b:b + 1, :n].clone(), want_dc_init=True, **one)
                assert torch.equal(g["du"][b, :n].isnan(), alone["du"][0].isnan())
                assert torch.equal(g["du"][b, :n].nan_to_num(7.0), alone["du"][0].nan_to_num(7.0))
                if want_dc_init:
                    assert torch.equal(g["dc_init"][b].nan_to_num(7.0), alone["dc_init"][0].nan_to_num(7.0))
        rest = [i for i in range(ch) if i != 2]
        assert torch.equal(g["du"][..., rest], clean["du"][..., rest]) and torch.equal(g["dw"][rest], clean["dw"][rest])
