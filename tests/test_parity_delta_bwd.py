"""GPU parity of the gated delta rule's gradients against the recurrence's in
64 bits, and of those against differences of the forward."""
import pytest
import torch

import mamba_selective_scan_04_amd as m
from delta_util import check, inputs, reference

NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dh_init")
DTYPES = [torch.float32, torch.bfloat16]


def args(c):
    return c["q"], c["k"], c["v"], c["g"], c["beta"]


def both(c, h=True, dh=True):
    h0 = c["h"] if h else None
    _, _, chunks = m.delta_scan(*args(c), h_init=h0, lens=c["lens"], want_chunks=True)
    got = m.delta_scan_bwd(*args(c), chunks, c["do"], lens=c["lens"], dh_final=c["dh"] if dh else None,
                           want_dh_init=True)
    ref = reference({**c, "dh": c["dh"] if dh else None}, h=h0, want_grads=True)
    return got, ref


def check_all(got, ref, factor=2.0):   # a product chain and its transpose
    for n in NAMES:
        check(got[n], ref[n], n, factor)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size", [(1, 1, 1, 1, 64, 64), (1, 63, 1, 1, 64, 64), (2, 64, 2, 2, 128, 128),
                                  (1, 65, 1, 3, 128, 64), (2, 130, 2, 4, 64, 128), (2, 200, 1, 2, 128, 128)])
def test_gradients(dev, size, dtype):
    check_all(*both(inputs(*size, dtype, seed=10, device=dev)))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_from_zero_without_state_gradient(dev, dtype):
    check_all(*both(inputs(2, 100, 2, 2, 64, 64, dtype, seed=11, device=dev), h=False, dh=False))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_padded_rows(dev, dtype):
    lens = [130, 0, 1, 64, 70]
    c = inputs(5, 130, 2, 4, 64, 64, dtype, seed=12, device=dev, lens=lens)
    for b, n in enumerate(lens):
        for name in ("q", "k", "v", "g", "beta", "do"):
            c[name][b, n:] = float("nan")
    got, ref = both(c)
    for b, n in enumerate(lens):
        for name in NAMES[:5]:
            assert (got[name][b, n:] == 0).all(), name
    check_all(got, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_resets_and_idle_tokens(dev, dtype):
    """Documents' starts (g = -inf) and tokens that write nothing (beta = 0)."""
    c = inputs(1, 150, 1, 2, 64, 128, dtype, seed=13, device=dev, resets=[0, 5, 64, 100, 101])
    c["beta"][:, 20:30] = 0
    check_all(*both(c))


@pytest.mark.gpu
def test_same_bits_again(dev):
    c = inputs(2, 300, 2, 4, 128, 128, torch.bfloat16, seed=14, device=dev)
    _, _, chunks = m.delta_scan(*args(c), want_chunks=True)
    a, b = (m.delta_scan_bwd(*args(c), chunks, c["do"], want_dh_init=True) for _ in range(2))
    assert all(torch.equal(a[n], b[n]) for n in NAMES)


@pytest.mark.gpu
def test_empty(dev):
    c = inputs(2, 0, 1, 1, 64, 64, torch.bfloat16, device=dev)
    _, _, chunks = m.delta_scan(*args(c), want_chunks=True)
    got = m.delta_scan_bwd(*args(c), chunks, c["do"], dh_final=c["dh"], want_dh_init=True)
    assert torch.equal(got["dh_init"], c["dh"])


def test_reference_against_differences():
    """The 64-bit gradients themselves: central differences with step 1e-5 of
    O(1) values, whose third derivatives and roundings leave about 1e-9."""
    c = inputs(2, 70, 1, 2, 64, 64, torch.float32, seed=15, lens=[70, 5], resets=[7])
    c = {n: x.double() if x is not None and x.is_floating_point() else x for n, x in c.items()}
    grads = reference(c, h=c["h"], want_grads=True)
    live = torch.arange(70)[None, :, None, None] < c["lens"][:, None, None, None]

    def objective():
        r = reference(c, h=c["h"])
        return float((r["o"] * c["do"] * live).sum() + (r["h"] * c["dh"]).sum())

    gen = torch.Generator().manual_seed(3)
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("beta", "dbeta"), ("h", "dh_init")):
        step = torch.randn(c[name].shape, generator=gen, dtype=torch.float64)
        if name == "g":
            step[:, 7] = 0     # -inf
        base, e = c[name], 1e-5
        c[name] = base + e * step
        up = objective()
        c[name] = base - e * step
        down = objective()
        c[name] = base
        want = float((grads[grad] * step).sum())
        assert abs((up - down) / (2 * e) - want) <= 1e-6 * max(1.0, abs(want)), name


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("segs", [2, 3, 5])
@pytest.mark.parametrize("heads", [(1, 2, 64, 128), (2, 2, 128, 64)])
def test_segments(dev, heads, segs, dtype, monkeypatch):
    """The adjoint's chunks in segments that run at once; rows that end inside one, or have none."""
    monkeypatch.setenv("BDSSM_DELTA_SEGMENTS", str(segs))
    c = inputs(3, 330, *heads, dtype, seed=15, device=dev, resets=[100, 200], lens=[330, 65, 0])
    got, ref = both(c)
    check_all(got, ref, 3.0)             # as above, and each segment's map once more on the state's adjoint
    again = both(c)[0]
    assert all(torch.equal(got[n], again[n]) for n in NAMES)
    check_all(*both(c, h=False, dh=False), 3.0)


@pytest.mark.gpu
def test_long_row_is_segmented(dev, monkeypatch):
    c = inputs(1, 2100, 1, 1, 128, 64, torch.bfloat16, seed=16, device=dev)
    s = m.DeltaShape(1, 1, 1, 128, 64, 1)
    check_all(*both(c), 3.0)
    maps = m.delta_workspace_bytes(s, 2100, True)
    monkeypatch.setenv("BDSSM_DELTA_SEGMENTS", "1")
    assert maps > m.delta_workspace_bytes(s, 2100, True)   # it was: the segments' maps take room
