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


def test_tree_spills_no_more_than_measured(tmp_path):
    # bytes of spill stores and loads with which the kernels' times were taken (16-bit
    # caches of head_dim 128 and 64, FP8 caches); the merge kernels have none
    report = ptxas_report("tree_attn.cu", str(tmp_path))
    for pattern, st, ld in ((r"tree_kernelILi[01]ELi128E", 208, 296), (r"tree_kernelILi[01]ELi64E", 180, 256),
                            (r"tree_kernelILi2ELi128E", 128, 164), (r"tree_merge_kernel", 0, 0)):
        for name, (_, stores, loads) in find(report, pattern):
            assert stores <= st and loads <= ld, (name, stores, loads)
