"""The short causal convolution against its formula in 64 bits."""
import pytest
import torch

import mamba_selective_scan_04_amd as m
from layer_util import conv_inputs, conv_reference, near

DTYPES = [torch.float32, torch.bfloat16]
# batch, T, channels, width: one token to several chunks, channels below and beside a vector, one to several waves
SIZES = [(1, 1, 1, 4), (2, 1, 8, 2), (1, 2, 3, 4), (3, 3, 16, 3), (1, 5, 130, 4), (2, 17, 9, 3), (2, 64, 40, 4), (1, 65, 264, 2),
         (1, 200, 7, 4), (2, 131, 1021, 4)]


def forward(c, **kw):
    return m.conv_scan(c["u"], c["w"], bias=c["bias"], lens=c["lens"], starts=c["starts"], c_init=c["c_init"], **kw)


def backward(c, **kw):
    return m.conv_scan_bwd(c["u"], c["w"], c["dy"], bias=c["bias"], lens=c["lens"], starts=c["starts"], c_init=c["c_init"],
                           dc_final=c["dc"], want_dc_init=True, **kw)


def check_all(c, silu=True):
    r = conv_reference(c, silu)
    y, last = forward(c, silu=silu)
    near(y, r["y"], "y")
    assert torch.equal(last.cpu().double(), r["c"][0])
    g = backward(c, silu=silu)
    for n in ("du", "dw", "dc_init") + (("dbias",) if c["bias"] is not None else ()):
        near(g[n], r[n], n)
    assert (g["dbias"] is None) == (c["bias"] is None)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size", SIZES)
def test_sizes(dev, dtype, size):
    check_all(conv_inputs(*size, dtype, seed=sum(size), device=dev))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("silu,bias,init", [(False, True, True), (True, False, False), (False, False, False)])
def test_options(dev, dtype, silu, bias, init):
    check_all(conv_inputs(2, 37, 24, 4, dtype, seed=1, device=dev, bias=bias, init=init), silu)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("width", [2, 3, 4])
def test_lengths(dev, dtype, width):
    """Rows of no token, fewer than the state holds, one chunk and part of one, values outside 0..T; padding is NaN."""
    lens = [0, 1, 2, 3, 4, 33, 40, 41, -5, 1000]
    c = conv_inputs(len(lens), 41, 20, width, dtype, seed=2, device=dev, lens=lens)
    for b, n in enumerate(lens):
        c["u"][b, max(0, n):] = float("nan")
        c["dy"][b, max(0, n):] = float("nan")
    check_all(c)
    y, _ = forward(c)
    g = backward(c)
    for b, n in enumerate(lens):
        assert (y[b, max(0, n):] == 0).all() and (g["du"][b, max(0, n):] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("width", [2, 3, 4])
def test_documents(dev, dtype, width):
    """Starts at the first token, next to each other, on both sides of a chunk's end, at the row's last tokens, in padding."""
    starts = [(0, 0), (0, 5), (0, 6), (0, 8), (0, 63), (0, 64), (0, 65), (1, 62), (1, 67), (1, 89), (2, 87), (2, 88), (2, 40), (3, 2), (3, 30)]
    check_all(conv_inputs(4, 90, 12, width, dtype, seed=3, device=dev, starts=starts, lens=[90, 90, 89, 3]))


@pytest.mark.gpu
def test_a_document_hides_what_lies_in_front_of_it(dev):
    """Infinities and NaN in front of a start reach neither its outputs nor its gradients nor the state."""
    c = conv_inputs(1, 40, 16, 4, torch.bfloat16, seed=4, device=dev, starts=[(0, 20), (0, 38)])
    clean = {n: x.clone() if isinstance(x, torch.Tensor) else x for n, x in c.items()}
    for t, v in ((17, float("inf")), (18, float("nan")), (19, float("-inf"))):
        c["u"][0, t] = v
        clean["u"][0, t] = 0
    y, last = forward(c)
    want, last2 = forward(clean)
    assert torch.equal(y[:, 20:], want[:, 20:]) and torch.equal(last, last2)
    assert torch.equal(y[:, :17], want[:, :17])
    assert (last[:, 0] == 0).all() and (last[:, 1:] != 0).any()
    assert torch.equal(backward(c)["du"][:, 20:], backward(clean)["du"][:, 20:])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("extra,at", [(8, 0), (24, 16), (5, 3), (1, 1)])
def test_slices(dev, dtype, extra, at):
    """u and du as channels of a wider tensor, from any channel on: the rest is neither used nor written."""
    c = conv_inputs(2, 50, 24, 4, dtype, seed=5, device=dev, extra=extra, at=at, lens=[50, 21])
    whole = dict(c, u=c["u"].contiguous())
    y, last = forward(c)
    assert all(torch.equal(a, b) for a, b in zip((y, last), forward(whole)))
    wide = torch.full_like(c["wide"], 7)
    g, w = backward(c, du=wide[..., at:at + 24]), backward(whole)
    assert all(torch.equal(g[n], w[n]) for n in w)
    wide[..., at:at + 24] = 7
    assert (wide == 7).all()
    # rows of a longer tensor, and every other row
    t = conv_inputs(4, 60, 24, 4, dtype, seed=6, device=dev)
    part = dict(t, u=t["u"][::2, 10:47], c_init=t["c_init"][:2].clone(), dy=t["dy"][:2, :37].contiguous(), dc=t["dc"][:2].clone())
    check_all(part)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [1, 2, 3, 16, 70])
def test_step(dev, dtype, T):
    """The step is the scan behind a cache; read only, to another state, and in place."""
    c = conv_inputs(3, T, 48, 4, dtype, seed=7, device=dev, lens=[T, T // 2, 0])
    r = conv_reference(c)
    kw = dict(bias=c["bias"], lens=c["lens"])
    before = c["c_init"].clone()
    y = m.conv_step(c["c_init"], c["u"], c["w"], **kw)
    near(y, r["y"], "y")
    assert torch.equal(c["c_init"], before)
    out = torch.empty_like(before)
    assert torch.equal(m.conv_step(c["c_init"], c["u"], c["w"], c_out=out, **kw), y)
    assert torch.equal(out.cpu().double(), r["c"][0]) and torch.equal(c["c_init"], before)
    state = before.clone()
    assert m.conv_step(state, c["u"], c["w"], c_out=state, want_y=False, **kw) is None
    assert torch.equal(state, out)
    assert torch.equal(m.conv_step(before, c["u"], c["w"], c_out=before, **kw), y) and torch.equal(before, out)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_pieces_make_the_whole(dev, dtype):
    c = conv_inputs(2, 97, 24, 4, dtype, seed=8, device=dev)
    y, last = forward(c)
    state, parts = c["c_init"].clone(), []
    for a, z in ((0, 1), (1, 3), (3, 40), (40, 97)):
        parts.append(m.conv_step(state, c["u"][:, a:z], c["w"], bias=c["bias"], c_out=state))
    assert torch.equal(torch.cat(parts, 1), y) and torch.equal(state, last)


@pytest.mark.gpu
def test_differences(dev):
    """The gradients against differences of the formula's loss in 64 bits, along random directions."""
    c = conv_inputs(2, 30, 10, 4, torch.float32, seed=9, device=dev, lens=[30, 17], starts=[(0, 11), (1, 3)])
    g = backward(c)
    grads = dict(u=g["du"], w=g["dw"], bias=g["dbias"], c_init=g["dc_init"])

    def loss(x):
        r = conv_reference(x)
        return float((r["y"][0] * c["dy"].cpu().double()).sum() + (r["c"][0] * c["dc"].cpu().double()).sum())

    gen = torch.Generator().manual_seed(10)
    cpu = {n: x.cpu().double() if isinstance(x, torch.Tensor) and x.is_floating_point() else x for n, x in c.items()}
    for n, grad in grads.items():
        d = torch.randn(grad.shape, generator=gen, dtype=torch.float64)
        h = 1e-4                 # the difference's own error is h^2 / 6 of the third derivative, below 1e-7 of it
        up, down = (loss(dict(cpu, **{n: cpu[n] + s * h * d})) for s in (1, -1))
        slope, got = (up - down) / (2 * h), float((grad.cpu().double() * d).sum())
        assert abs(got - slope) <= 1e-5 * float((grad.cpu().double() * d).abs().sum()), (n, got, slope)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_many_parts(dev, dtype):
    """More chunks than parts: workgroups go round.  Against one call for each row, summed in 64 bits."""
    c = conv_inputs(9000, 8, 260, 4, dtype, seed=11, device=dev)
    g = backward(c)
    dw, db = torch.zeros(260, 4, dtype=torch.float64), torch.zeros(260, dtype=torch.float64)
    size = torch.zeros_like(dw)
    for a in range(0, 9000, 3000):
        part = {n: x[a:a + 3000].contiguous() if x is not None and n not in ("w", "bias") else x for n, x in c.items()}
        p = backward(part)
        dw += p["dw"].cpu().double()
        db += p["dbias"].cpu().double()
        assert torch.equal(p["du"], g["du"][a:a + 3000]) and torch.equal(p["dc_init"], g["dc_init"][a:a + 3000])
        size += (part["dy"].float().abs().sum((0, 1)).cpu() * 12).double()[:, None]
    assert ((g["dw"].cpu() - dw).abs() <= 700 * 2.0 ** -24 * size).all()
    assert ((g["dbias"].cpu() - db).abs() <= 700 * 2.0 ** -24 * size[:, 0]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_large_values(dev, dtype):
    """silu where its exponential overflows and where it vanishes; infinities stay in their reach."""
    c = conv_inputs(1, 12, 8, 2, dtype, seed=12, device=dev, bias=False, init=False)
    c["w"].zero_()
    c["w"][:, 1] = 1
    v = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 88.0, -88.0, 200.0, -200.0, 3e38, -3e38, float("inf"), 1.0])
    c["u"][0] = v[:, None].to(dtype)
    y = m.conv_scan(c["u"], c["w"])[0][0, :, 0].float().cpu()
    x = c["u"][0, :, 0].float().cpu()
    want = torch.where(x == float("inf"), x, x * torch.sigmoid(x.double()).float())
    assert ((y - want).abs() <= 2.0 ** -7 * want.abs() + 1e-30)[:10].all()
    assert y[10] == float("inf") and y[11].isnan()      # 0 times infinity, one token later
    g = m.conv_scan_bwd(c["u"][:, :10].contiguous(), c["w"], torch.ones_like(c["u"][:, :10]))["du"]
    assert torch.isfinite(g).all() and (g[0, 6] == 1).all() and (g[0, 7] == 0).all()


@pytest.mark.gpu
def test_empty(dev):
    for dtype in DTYPES:
        z = torch.zeros(2, 0, 6, dtype=dtype, device=dev)
        c = conv_inputs(2, 4, 6, 4, dtype, seed=13, device=dev)
        y, last = m.conv_scan(z, c["w"], c_init=c["c_init"])
        assert y.shape == z.shape and torch.equal(last, c["c_init"])
        g = m.conv_scan_bwd(z, c["w"], z, bias=c["bias"], dc_final=c["dc"], want_dc_init=True)
        assert torch.equal(g["dc_init"], c["dc"]) and (g["dw"] == 0).all() and (g["dbias"] == 0).all()
        none = torch.zeros(0, 4, 6, dtype=dtype, device=dev)
        g = m.conv_scan_bwd(none, c["w"], none, bias=c["bias"])
        assert (g["dw"] == 0).all() and (g["dbias"] == 0).all() and m.conv_scan(none, c["w"])[0].shape == none.shape


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("starts", [False, True])
def test_whole_lanes_and_parts_of_lanes(dev, dtype, width, starts):
    """Channels that fill their lanes and that do not, with and without documents, at lengths around chunks' ends.  (The
    kernels of the two may round a product and a sum together or apart, so each is held to the formula.)"""
    for T in (4, 6, 7, 23, 24, 25, 48, 53):
        c = conv_inputs(3, T, 24, width, dtype, seed=14 + T, device=dev, lens=[T, T // 2, 1], starts=[(0, T // 2), (1, 0), (0, T - 1)] if starts else None)
        check_all(c)
        check_all({n: (x if n in ("lens", "starts") or x is None else x[:23].contiguous() if n in ("w", "bias") else x[..., :23].contiguous())
                   for n, x in c.items()})
