"""Products by expert that take the largest tile, 256 rows x 256 columns: few experts with many
rows each.  Tolerances as in test_gpu_w8a8.py, whose cases and oracle they use."""

import pytest
import torch

import bit_quantized_gemm_qgemm_amd as qg
from test_gpu_w8a8 import experts_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    qg.lib()
    return torch.device("cuda:0")


# part-full last blocks, one of a single row, whole blocks, experts without rows; five, six,
# seven and eight K tiles, the last one part-full; columns that end inside a block (gated: of 1025,
# 1281 and 2049 outputs); rows before the first expert's and after the last's
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("gated,dtype", [(False, torch.float16), (False, torch.bfloat16), (True, torch.float16),
                                         (True, torch.bfloat16)])
@pytest.mark.parametrize("counts,N,K", [
    ([5783], 2050, 528), ([1793, 1290], 4098, 528), ([1536, 3100], 2562, 656), ([0, 2049, 1040], 4098, 784),
    ([256, 0, 1, 1755, 700], 4098, 912),
])
def test_the_largest_tile_by_expert(counts, N, K, gated, dtype, gather):
    lead, tail = 3, 14
    M = lead + sum(counts) + tail
    assert qg.qgemm_w8a8_tile(M, N, K, len(counts), gated) == (256, 256, 1)
    experts_case(counts, K, N, gated, dtype, gather, lead=lead, tail=tail)
