"""Register budget of the expanded attention's kernel, which splits its registers
between warpgroups: the count ptxas reports has to be the one its split assumes
(128 x 104 + 256 x 200 = 384 x 168; with another count the host refuses the
kernel, since a warpgroup that raises its share could wait forever).  It needs
nvcc but no GPU."""
import pytest

from test_register_budget import NVCC, find, ptxas_report

pytestmark = pytest.mark.skipif(NVCC is None, reason="nvcc not available")


def test_expanded_split(tmp_path):
    for name, (regs, _, _) in find(ptxas_report("latent_expanded.cu", str(tmp_path)), r"expanded_kernelILi\dE"):
        assert regs == 168, (name, regs)
