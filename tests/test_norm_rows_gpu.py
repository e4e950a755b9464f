"""The norms' sums over rows, held to the rows that a workgroup really adds one after the other."""
import pytest

import block_ref as B
import layer_ref as R  # noqa: F401
from test_block_gpu import tensors, within

pytestmark = pytest.mark.gpu

w4q = pytest.importorskip("w4a16_group_wise_amd")


def rows_of_a_workgroup(m, d):
    """8 columns a thread in whole wavefronts; as many workgroups as the device holds at 16 wavefronts a compute unit, but up to
    four rows each before a second workgroup lies on one."""
    threads = min(1024, -(-d // 512) * 64)
    return max(-(-m // (256 * (1024 // threads))), min(-(-m // 256), 4))


def test_the_rule():
    assert [rows_of_a_workgroup(*s) for s in ((1, 4096), (9, 1001), (300, 8192), (513, 1100), (1530, 1056), (8192, 4096), (20001, 520))] == \
        [1, 1, 2, 3, 4, 16, 10]


@pytest.mark.parametrize("m,d", [(1, 4096), (2, 7), (9, 1001), (255, 72), (257, 1100), (300, 8192), (513, 1100), (700, 2050), (1100, 7168),
                                 (1530, 1056), (3001, 4104), (2000, 8200), (20001, 520)])
@pytest.mark.parametrize("types", [("bf16", "bf16", "bf16"), ("f32", "bf16", "bf16"), ("f32", "f32", "f32")])
def test_sums_over_rows(dev, m, d, types):
    groups = next(g for g in (3, 2, 5, 7, 1) if m % g == 0)
    t = tensors(dev, m, d, *types, gate="f32", groups=groups, seed=m)
    kw = dict(w_post=t["w_post"], w_pre=t["w_pre"], gate=t["gate"])
    got = dict(zip(("h", "y", "w_post", "w_pre", "gate"), w4q.block_norm_bwd(t["grad_n"], t["grad_r"], t["h"], t["y"], **kw)))
    ref, err = B.norm_bwd(t["grad_n"], t["grad_r"], t["h"], t["y"], t["w_post"], t["w_pre"], t["gate"], rows=rows_of_a_workgroup(m, d))
    for k in ("w_post", "w_pre", "gate"):
        within(got[k], ref[k], err[k], "grad " + k)
