"""No kernel of a block's operators keeps vector registers in memory, and the norms' hardly any scalars in vector registers, by the built library's own notes (no GPU needed)."""
import os
import re
import shutil
import subprocess

import pytest

from w4a16_group_wise_amd import LIB_PATH

LLVM = "/opt/rocm/llvm/bin"


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    tools = [os.path.join(LLVM, t) for t in ("llvm-objdump", "llvm-readelf")]
    if not all(os.path.exists(t) for t in tools):
        pytest.skip("no LLVM tools")
    d = tmp_path_factory.mktemp("code")
    lib = shutil.copy(LIB_PATH, d)
    subprocess.run([tools[0], "--offloading", lib], cwd=d, check=True, capture_output=True)
    found = {}
    for f in sorted(os.listdir(d)):
        if "amdgcn" not in f:
            continue
        notes = subprocess.run([tools[1], "--notes", os.path.join(d, f)], check=True, capture_output=True, text=True).stdout
        for part in re.split(r"\n  - \.", notes)[1:]:
            name = re.search(r"^ {4}\.name: +(\S+)", part, flags=re.M)
            values = [re.search(rf"\.{k}: +(\d+)", part) for k in ("private_segment_fixed_size", "vgpr_spill_count", "sgpr_spill_count")]
            if name and all(values):
                found[name.group(1)] = tuple(int(v.group(1)) for v in values)
    return found


@pytest.mark.parametrize("kind,least", [("norm_", 10), ("fp8_", 60), ("clip_", 3)])
def test_no_scratch(kernels, kind, least):
    mine = {k: v for k, v in kernels.items() if re.search(rf"w4q12_GLOBAL__N_1\d+{kind}", k)}
    assert len(mine) >= least
    assert not {k: v for k, v in mine.items() if v[:2] != (0, 0)}


def test_scalars_of_the_norms(kernels):
    # seven arguments that the kernel of ragged rows reads before and after its rows
    assert not {k: v for k, v in kernels.items() if re.search(r"w4q12_GLOBAL__N_1\d+norm_", k) and v[2] > 8}
