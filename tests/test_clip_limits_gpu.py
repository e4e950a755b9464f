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


def test_the_norm_may_not_lie_in_a_gradient_or_result(dev):
    buf = torch.arange(1.0, 101.0, device=dev)
    keep = buf.clone()
    outs = [torch.zeros(20, device=dev), torch.zeros(1, device=dev), torch.zeros(30, device=dev, dtype=torch.bfloat16)]
    plan = w4q.GradPlan([buf[10:30], buf[40:41], buf[60:90]], outs)
    for at in (10, 15, 29, 40, 60, 75, 89):
        for call in (lambda o: plan.norm(out=o), lambda o: plan.clip(1.0, out=o)):
            with pytest.raises(ValueError, match="overlap"):
                call(buf[at:at + 1])
    for out in (outs[0][:1], outs[0][19:], outs[1], outs[2][:2].view(torch.float32), outs[2][28:].view(torch.float32)):
        with pytest.raises(ValueError, match="overlap"):
            plan.clip(1.0, out=out)
    assert torch.equal(buf, keep) and all(float(o.float().abs().max()) == 0 for o in outs)
    # beside them it may
    want = math.sqrt(sum(float((t.double() ** 2).sum()) for t in (keep[10:30], keep[40:41], keep[60:90])))
    for at in (0, 9, 30, 39, 41, 59, 90, 99):
        got = plan.clip(1.0, out=buf[at:at + 1])
        assert got.data_ptr() == buf[at:].data_ptr() and abs(float(got) - want) <= want * (2.0 ** -24 + 1e-12)
    assert torch.equal(buf[10:30], keep[10:30]) and torch.equal(buf[60:90], keep[60:90])
