"""A NaN of any payload in the bias (memory filled with 0xFF is one) is a NaN in its column of the result,
in every kernel and both output types, and reaches no other column."""
import pytest
import torch

import layer_ref as R

pytestmark = pytest.mark.gpu

w4q = pytest.importorskip("w4a16_group_wise_amd")


@pytest.mark.parametrize("m", [1, 4, 40, 300])
@pytest.mark.parametrize("n", [512, 515])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_nan_bias(dev, m, n, dtype):
    x, w, scale, bias = (t.to(dev) for t in R.layer(m, n, 512, seed=m))
    packed, s16 = w4q.quant_pack(w, scale)
    bad = bias.clone()
    bits = bad.view(torch.int32)
    cols = torch.tensor([3, 7, 100, n - 1], device=dev)
    bits[cols] = torch.tensor([-1, 0x7FFFFFFF, 0x7FC00000, -0x7FFFFF], dtype=torch.int32, device=dev)
    fine = torch.ones(n, dtype=torch.bool, device=dev)
    fine[cols] = False
    for act in R.ACTS:
        calls = [lambda b: w4q.lsq_linear_fwd(x, w, scale, bias=b, act=act, out_dtype=dtype)[0]]
        for dq in (False, True):
            for ws in (None, torch.empty(0, dtype=torch.uint8, device=dev)):
                calls.append(lambda b, dq=dq, ws=ws: w4q.w4a16_linear(x, packed, s16, bias=b, act=act, dequant_bf16=dq,
                                                                      out_dtype=dtype, workspace=ws))
        for call in calls:
            y = call(bad)
            assert bool(torch.isnan(y[:, cols]).all())
            assert torch.equal(y[:, fine], call(bias)[:, fine])
