"""grad_clip's limit and its norm's place."""
import math

import pytest
import torch

import layer_ref as R

pytestmark = pytest.mark.gpu

w4q = pytest.importorskip("w4a16_group_wise_amd")


def test_the_limit_is_taken_in_64_bits(dev):
    # The factor is the 64-bit quotient rounded once, and a result the product rounded once: equal bit for bit.  (The norm's sums of
    # 64 bits may differ in the last places, 2^-29 of a rounding of fp32: 40 limits all on one side of a border but for one
    # chance in 10^7.)
    g = R.gen(1, dev)
    grads = [torch.randn(300, 77, generator=g, device=dev), torch.randn(5, generator=g, device=dev)]
    norm = math.sqrt(sum(float((t.double() ** 2).sum()) for t in grads))
    outs = [torch.empty_like(t) for t in grads]
    plan = w4q.GradPlan(grads, outs)
    for i in range(1, 41):
        limit, eps = 0.1 * i, 1e-6 / i
        plan.clip(limit, eps=eps)
        c = torch.tensor(limit / (norm + eps), dtype=torch.float64).float().to(dev)
        assert all(torch.equal(o, t * c) for o, t in zip(outs, grads)), limit


def test_limits_that_fp32_does_not_tell_from_the_norm(dev):
    grads = [torch.ones(9, device=dev)]          # norm 3
    outs = [torch.empty_like(grads[0])]
    for limit, clipped in ((3.0 + 1e-9, False), (3.0, False), (3.0 - 1e-6, True), (1e300, False)):
        w4q.grad_clip(grads, limit, eps=0.0, outs=outs)
        assert torch.equal(outs[0], grads[0]) != clipped, limit
    # behind fp32's last place the factor is rounded to one
    w4q.grad_clip(grads, 3.0 - 1e-9, eps=0.0, outs=outs)
    assert torch.equal(outs[0], grads[0])
