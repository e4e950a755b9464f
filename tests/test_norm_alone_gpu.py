"""The first norm of a stack, without a block's output before it: the backward pass is the gradient of the forward whatever
scales the parameters hold."""
import ctypes

import pytest
import torch

import block_ref as B
from test_block_gpu import tensors, within
from w4a16_group_wise_amd import _lib

pytestmark = pytest.mark.gpu

w4q = pytest.importorskip("w4a16_group_wise_amd")


@pytest.mark.parametrize("m,d", [(5, 7), (9, 64), (300, 1001), (4, 4096), (3, 9000)])
@pytest.mark.parametrize("with_r", [False, True])
def test_the_scales_are_not_used_without_y(dev, m, d, with_r):
    t = tensors(dev, m, d, "f32", "f32", "f32", seed=m)
    hp = _lib.NormParams(1e-5, 0.25, 0.75, -1.25)     # one set of parameters for both calls
    n, gh, gw = (torch.empty_like(t[k]) for k in ("h", "h", "w_pre"))
    gr = t["grad_r"] if with_r else None
    L, s = w4q.lib(), torch.cuda.current_stream().cuda_stream
    ws = torch.empty(w4q.workspace_size("block_norm_bwd", m, d), dtype=torch.uint8, device=dev)
    assert L.block_norm_fwd(t["h"].data_ptr(), 0, None, 0, m, d, None, t["w_pre"].data_ptr(), None, 0, 0, ctypes.byref(hp), None,
                            n.data_ptr(), 0, s) == 0
    assert L.block_norm_bwd(t["grad_n"].data_ptr(), 0, gr.data_ptr() if with_r else None, t["h"].data_ptr(), 0, None, 0, m, d, None,
                            t["w_pre"].data_ptr(), None, 0, 0, ctypes.byref(hp), gh.data_ptr(), None, None, gw.data_ptr(), None,
                            ws.data_ptr(), ws.numel(), s) == 0
    opt = dict(eps=1e-5, offset=0.25)
    _, ref, _, err = B.norm_fwd(t["h"], None, None, t["w_pre"], None, **opt)
    within(n, ref, err, "n")
    ref, err = B.norm_bwd(t["grad_n"], gr, t["h"], None, None, t["w_pre"], None, rows=max(4, -(-m // 256)), **opt)
    within(gh, ref["h"], err["h"], "grad h")
    within(gw, ref["w_pre"], err["w_pre"], "grad w_pre")
    # against the differences of the 64-bit forward, which knows no scales without y
    h = t["h"].double()
    for i, j in ((0, 0), (m - 1, d - 1), (m // 2, d // 3)):
        def loss(x):
            v = h.clone()
            v[i, j] += x
            inv = 1 / torch.sqrt((v[i] * v[i]).mean() + 1e-5)
            out = (t["grad_n"][i].double() * v[i] * inv * (t["w_pre"].double() + 0.25)).sum()
            return float(out + (gr[i].double() * v[i]).sum() if with_r else out)
        step = 1e-4
        diff = (loss(step) - loss(-step)) / (2 * step)
        # third derivatives: |grad_n| w / rms^3 and d terms of it, times step^2 (below 1e-8 of values near one), and what fp32 rounds
        assert abs(float(gh[i, j]) - diff) <= float(err["h"][i, j]) + 2.0 ** -24 * abs(diff) + 1e-6


def test_the_binding_refuses_a_skip_scale_without_y(dev):
    t = tensors(dev, 4, 64, seed=1)
    with pytest.raises(ValueError, match="skip_scale"):
        w4q.block_norm_bwd(t["grad_n"], t["grad_r"], t["h"], w_pre=t["w_pre"], skip_scale=0.75)
    with pytest.raises(ValueError):
        w4q.block_norm_fwd(t["h"], w_pre=t["w_pre"], skip_scale=0.75)


@pytest.mark.parametrize("d", [40, 1001])
def test_a_branch_without_norm_and_gate_keeps_its_scales(dev, d):
    # y NULL where nothing needs it, grad_y asked for: the branch exists
    m = 6
    t = tensors(dev, m, d, "f32", "f32", "f32", seed=2)
    hp = _lib.NormParams(1e-5, 0.0, 0.75, -1.25)
    gh, gy = torch.empty_like(t["h"]), torch.empty_like(t["h"])
    ws = torch.empty(w4q.workspace_size("block_norm_bwd", m, d), dtype=torch.uint8, device=dev)
    assert w4q.lib().block_norm_bwd(None, 0, t["grad_r"].data_ptr(), None, 0, None, 0, m, d, None, None, None, 0, 0, ctypes.byref(hp),
                                    gh.data_ptr(), gy.data_ptr(), None, None, None, ws.data_ptr(), ws.numel(),
                                    torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(gh, 0.75 * t["grad_r"]) and torch.equal(gy, -1.25 * t["grad_r"])
    # a gate says so too
    assert w4q.lib().block_norm_bwd(None, 0, t["grad_r"].data_ptr(), None, 0, None, 0, m, d, None, None, t["h"].data_ptr(), 0, m,
                                    ctypes.byref(hp), gh.zero_().data_ptr(), None, None, None, None, ws.data_ptr(), ws.numel(),
                                    torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(gh, 0.75 * t["grad_r"])
