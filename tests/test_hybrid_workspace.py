"""Workspaces of the caller's own: any contiguous tensor of the bytes asked
for; views whose elements are not bytes in a row are refused, before any
launch."""
import ctypes

import pytest
import torch

import mamba_selective_scan_04_amd as m
import delta_util
import kv_util
from mamba_selective_scan_04_amd import hybrid


def test_a_workspace_on_the_host_is_refused():
    with pytest.raises(ValueError, match="GPU"):
        hybrid._room(torch.empty(64, dtype=torch.uint8), "bdssm_delta_workspace_bytes")


def calls(dev):
    c = delta_util.inputs(1, 100, 1, 2, 64, 64, torch.bfloat16, seed=80, device=dev)
    a = c["q"], c["k"], c["v"], c["g"], c["beta"]
    chunks = m.delta_scan(*a, want_chunks=True)[2]
    s = m.DeltaShape(1, 1, 2, 64, 64, 1)
    x = kv_util.inputs(1, [3000], 4, 4, 4, 2, 64, 16, torch.int8, torch.bfloat16, seed=81, device=dev)
    ks = m.KvShape(1, 4, 2, 64, 16, x["k"].shape[0], x["table"].shape[1], 1, 1)
    cache = m.KvCache(x["k"], x["ks"], x["v"], x["vs"])
    return [(m.delta_workspace_bytes(s, 100), lambda ws: m.delta_scan(*a, ws=ws)[0]),
            (m.delta_workspace_bytes(s, 100, True), lambda ws: m.delta_scan_bwd(*a, chunks, c["do"], ws=ws)["dk"]),
            (m.load().bdssm_kv_workspace_bytes(ctypes.byref(ks), 4),
             lambda ws: m.kv_attn_step(cache, x["q"], x["nk"], x["nv"], x["table"], x["ctx"], ws=ws))]


@pytest.mark.gpu
def test_own_workspaces(dev):
    for n, call in calls(dev):
        assert n > 0
        want = call(None)
        assert torch.equal(call(torch.empty(n, dtype=torch.uint8, device=dev)), want)
        assert torch.equal(call(torch.empty(n // 4 + 1, dtype=torch.float32, device=dev)), want)
        with pytest.raises(m.BdssmError):
            call(torch.empty(n - 1, dtype=torch.uint8, device=dev))
        with pytest.raises(ValueError, match="contiguous"):
            call(torch.empty(1, dtype=torch.uint8, device=dev).expand(n))
        with pytest.raises(ValueError, match="contiguous"):
            call(torch.empty(n, 2, dtype=torch.uint8, device=dev)[:, 0])
