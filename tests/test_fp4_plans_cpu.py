"""Plans of 4-bit experts without a GPU: the shapes that they refuse."""
import os
import shutil

import pytest

from pretraining_sigmoid_softmax_gb300 import build
from pretraining_sigmoid_softmax_gb300.layer import MoEPlan, MoEShape

needs_nvcc = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not installed")


@needs_nvcc
@pytest.mark.parametrize("flags", [dict(), dict(fp8=True), dict(fp8=True, fp8_dgrad=True),
                                   dict(fp4=True, fp8_dgrad=True)])
@pytest.mark.parametrize("f_shared", [0, 128])
def test_data_gradients_on_4_bits_need_4_bit_experts(flags, f_shared):
    """Without them no buffers of the data gradients' operands are there, and no backward that uses them."""
    build.build_library()
    with pytest.raises(ValueError, match="fp4_dgrad"):
        MoEPlan(MoEShape(64, 128, 4, 2, 768, f_shared, fp4_dgrad=True, **flags), "cpu", overlap_shared=False)
