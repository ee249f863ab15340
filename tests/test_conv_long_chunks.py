"""The convolution against its formula in 64 bits where a lane takes many tokens, as in long prompts and training:
its loops over whole groups of tokens, and lengths, documents and states at every place in a chunk.

Few channels make such sizes cheap.  Additions behind each other in dw and dbias (layer_util's 700): a lane's tokens,
at most 66 and the rows it goes round, 128 lanes of a workgroup, 48 parts of a wave and 16 waves."""
import ctypes

import pytest
import torch

import mamba_selective_scan_04_amd as m
from large_util import conv_reference, near

# batch, T, then tokens of a lane forward and backward
SIZES = [(61, 16393, 8, 12), (53, 37633, 16, 24), (29, 107021, 24, 36), (7, 900001, 24, 66)]


def inputs(dev, batch, T, ch, width, dtype, seed, starts, extra=0, at=0):
    gen = torch.Generator(device=dev).manual_seed(7000 + seed)
    rn = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    lens = T - torch.randint(0, 200, (batch,), generator=gen, device=dev)
    lens[0] = T
    lens[1] = 0
    lens[2::5] = torch.randint(0, T + 1, (len(lens[2::5]),), generator=gen, device=dev)
    c = dict(w=rn(ch, width), bias=rn(ch) * 0.3, c_init=rn(batch, width - 1, ch).to(dtype), dy=rn(batch, T, ch).to(dtype),
             dc=rn(batch, width - 1, ch).to(dtype), lens=lens.to(torch.int32), starts=None, u=rn(batch, T, ch + extra).to(dtype)[..., at:at + ch])
    padding = torch.arange(T, device=dev) >= lens[:, None]
    c["u"][padding] = float("nan")
    c["dy"][padding] = float("nan")
    if starts:      # rows of short documents, of long ones and of one alone; at the last tokens of a row
        often = torch.tensor([1 / 5, 1 / 300, 0.0], device=dev)[torch.arange(batch, device=dev) % 3]
        c["starts"] = torch.rand(batch, T, generator=gen, device=dev) < often[:, None]
        c["starts"][3, max(int(lens[3]) - 1, 0)] = True
        c["starts"][4, max(int(lens[4]) - 2, 0)] = True
    return c


def plan(batch, T, ch, width):
    """Tokens of a lane forward and backward by the plans' rules, and the parts of the parameters' gradients."""
    lanes = -(-ch // 4)
    forward = min(24, max(4, -(-batch * T * lanes // (256 * 16 * 64))))
    assert lanes <= 64
    row_lanes = 1 << (lanes - 1).bit_length()
    per, most = 256 // row_lanes, 256 * 3
    chunks = max(1, most * per // batch)
    backward = -(-(-(-T // chunks)) // 6) * 6
    return forward, backward, min(most, -(-batch * -(-T // backward) // per))


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("ch", [8, 5])
def test_plans(size, ch):
    """The sizes have the chunks that they stand for (the gradients' parts, which the library tells, say so too)."""
    batch, T, forward, backward = size
    for width in (2, 3, 4):
        got = plan(batch, T, ch, width)
        assert got[:2] == (forward, backward)
        s = m.ConvShape(batch, ch, width, ch, T * ch, 0)
        parts = m.load().bdssm_conv_workspace_bytes(ctypes.byref(s), T) // ((width + 1) * ch * 4)
        assert parts == got[2]
        # of all chunk lengths this one alone has that many parts, but where there are as many as there may be
        same = [k for k in range(6, 96, 6) if min(768, -(-batch * -(-T // k) // 128)) == parts]
        assert same == [backward] or parts == 768


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("starts", [False, True])
@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("ch", [8, 5])
@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("size", SIZES)
def test_long_chunks(dev, size, width, ch, silu, starts, dtype):
    batch, T = size[:2]
    c = inputs(dev, batch, T, ch, width, dtype, sum(size) + width + ch, starts, *((3, 1) if ch == 5 else (0, 0)))
    r = conv_reference(c, silu)
    kw = dict(bias=c["bias"], silu=silu, lens=c["lens"], starts=c["starts"], c_init=c["c_init"])
    y, last = m.conv_scan(c["u"], c["w"], **kw)
    near(y, r["y"], "y")
    assert torch.equal(last.double(), r["c"][0])
    g = m.conv_scan_bwd(c["u"], c["w"], c["dy"], dc_final=c["dc"], want_dc_init=True, **kw)
    for n in ("du", "dw", "dbias", "dc_init"):
        near(g[n], r[n], n)
    # without the state's gradient the row's first group goes as the others do
    alone = m.conv_scan_bwd(c["u"], c["w"], c["dy"], dc_final=c["dc"], **kw)
    for n in ("du", "dw", "dbias"):
        near(alone[n], r[n], n)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("width", [2, 3, 4])
def test_commit_in_place_of_long_rows(dev, dtype, width):
    batch, T = SIZES[1][:2]
    c = inputs(dev, batch, T, 8, width, dtype, 9 + width, False)
    r = conv_reference(c, True)
    state = c["c_init"].clone()
    y = m.conv_step(state, c["u"], c["w"], bias=c["bias"], lens=c["lens"], c_out=state)
    near(y, r["y"], "y")
    assert torch.equal(state.double(), r["c"][0])


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("starts", [False, True])
def test_references_agree(silu, starts):
    """The reference of all tokens at once and the one token by token."""
    import layer_util
    for width, lens in ((2, [9, 0, 1, 8]), (3, [1, 9, 2, 5]), (4, [3, 2, 9, 1])):
        at = [(0, 0), (0, 7), (0, 8), (1, 1), (2, 3), (2, 4), (3, 0), (3, 7)] if starts else None
        c = layer_util.conv_inputs(4, 9, 5, width, torch.float32, seed=width, lens=lens, starts=at)
        a, b = conv_reference(c, silu), layer_util.conv_reference(c, silu)
        assert a.keys() == b.keys()
        for n in a:
            for x, y in zip(a[n], b[n]):
                assert (x - y).abs().max() <= 1e-12 * (1 + y.abs().max()), n
