"""muon_step on weights whose rows are not multiples of 16 bytes, with tiles that end far past the last
row, and the weights at the end of their buffer."""
import pytest
import torch

import layer_ref as R

pytestmark = pytest.mark.gpu

w4q = pytest.importorskip("w4a16_group_wise_amd")


# (rows, cols): tiles of 32, 64, 128 and 256 rows with most of the last one past the matrix
@pytest.mark.parametrize("b,r,c", [(1, 65, 130), (2, 97, 201), (1, 769, 641), (1, 1281, 1301), (1, 4097, 4001)])
def test_ragged_step_equals_the_update(dev, b, r, c):
    g = R.gradient(R.gen(r, dev), b, r, c, device=dev)
    w = torch.randn(b, r, c, generator=R.gen(1, dev), device=dev)
    m = torch.zeros_like(g)
    o = w4q.newton_schulz(g)
    want = w.double() - 0.5 * (o.double() + 0.25 * w.double())
    w4q.muon_step(w, g, m, lr=0.5, momentum=0.0, nesterov=False, weight_decay=0.25, update_scale=1.0)
    # four fp32 roundings on values below |w| + |o|
    assert bool(((w.double() - want).abs() <= 4 * R.H32 * (want.abs() + o.double().abs() + w.double().abs())).all())
    assert torch.equal(m, g)
