"""Products of 32 to 65 rows on both sides of the rule that chooses their form, by N (half of the SMs
in tiles of 128 features) and by K."""
import pytest
import torch

from tests.test_gpu_fp8_block import BF, F32, check_gemm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [32, 33, 64, 65])
@pytest.mark.parametrize("block", [True, False])
def test_both_sides_of_the_few_rows_rule(lib, M, block):
    half = torch.cuda.get_device_properties(0).multi_processor_count // 2 * 128
    for N, K in ((half, 1536), (half + 1, 1536), (half - 127, 1540), (200, 1535), (200, 1536)):
        for dt in (BF, F32):
            check_gemm(M, N, K, block, dt=dt)
