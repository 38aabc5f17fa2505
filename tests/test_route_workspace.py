"""moe_route refuses a workspace that the kernel cannot use.  The other tensors
only say that they are on a GPU, so this runs without one: the refusal comes
before any CUDA call."""
import pytest
import torch

import combine_moe_layout_05_gb300 as moe
from combine_moe_layout_05_gb300 import build as moe_build


class OnGpu(torch.Tensor):
    is_cuda = True


def _gpu(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


@pytest.mark.parametrize("workspace", [
    torch.empty(1 << 16, dtype=torch.uint8),                             # host memory
    torch.empty(1 << 16, dtype=torch.uint8).as_subclass(OnGpu)[::2],     # the bytes between are not its own
])
def test_workspace_the_kernel_cannot_use(workspace):
    moe_build.build()
    i32 = torch.int32
    with pytest.raises(ValueError, match="workspace"):
        moe.moe_route(_gpu(4, 16), _gpu(4, 2, dtype=i32), _gpu(4, 2), _gpu(16, dtype=i32), _gpu(1, dtype=i32), _gpu(1),
                      workspace=workspace, stream=0)
