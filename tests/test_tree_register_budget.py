"""Register budget of the tree attention's kernels, which split their registers
between warpgroups: the counts ptxas reports have to be the ones their splits
assume (128 x 104 + 256 x 200 = 384 x 168 over 16-bit caches, 128 x (104 + 2 x 152 +
104) = 512 x 128 over FP8 ones; with another count the host refuses the kernel, since
a warpgroup that raises its share could wait forever).  It needs nvcc but no GPU."""
import pytest

from test_register_budget import NVCC, find, ptxas_report

pytestmark = pytest.mark.skipif(NVCC is None, reason="nvcc not available")


def test_tree_split(tmp_path):
    report = ptxas_report("tree_attn.cu", str(tmp_path))
    for name, (regs, _, _) in find(report, r"tree_kernelILi[01]E"):
        assert regs == 168, (name, regs)
    for name, (regs, _, _) in find(report, r"tree_kernelILi2E"):
        assert regs == 128, (name, regs)
