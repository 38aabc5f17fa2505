"""moe_expert_matmul_int8 where the average of rows an expert picks the 32-row
form and single experts have many more: their second and later tiles, full and
ragged, bit for bit as in test_gpu_expert_matmul_int8.py.  Short contractions
and many channels, so that no contraction is split over blocks."""
import pytest
import torch

import combine_moe_layout_05_gb300 as moe

from test_gpu_expert_matmul_int8 import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from combine_moe_layout_05_gb300 import build
    build.build()
    moe.load()


@pytest.mark.parametrize("H,N", [(16, 40), (1040, 1001), (1920, 520), (2064, 9744), (7168, 10001)])
@pytest.mark.parametrize("counts", [
    [33] + [0] * 31,
    [0, 300, 1, 64, 0, 65] + [2] * 40,                   # 10 tiles of one expert, the last of them short
    [97] + [1] * 20 + [96, 0, 128],
    [1] * 127 + [511] + [0] * 128,
])
def test_many_rows_of_a_few_experts(counts, H, N):
    assert sum(counts) + 2 <= 16 * len(counts)
    check(counts, H, N, seed=H + N, spare=2)
