"""int8 codes and scales of rows on the GPU at the lengths where the kernel's shape changes, and
between them: every result is exact."""

import pytest
import torch

import bit_quantized_gemm_qgemm_amd as qg
from test_gpu_quantize_int8 import TYPES, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    qg.lib()
    return torch.device("cuda:0")


# both sides of each edge: 512, 1024, 2048, 4096, 8192, 16384, 32768 and 65536 elements
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,K", [(5, 496), (5, 528), (6, 1024), (3, 1040), (5, 2048), (2, 2064), (3, 4096),
                                    (2, 4112), (3, 8192), (2, 8208), (3, 16384), (2, 16400), (3, 32768), (2, 32784),
                                    (2, 49168), (3, 65536), (2, 65552), (2, 131056)])
def test_each_shape_matches_the_oracle(dtype, rows, K):
    print("case quantize int8 length", dtype, rows, K, flush=True)
    g = torch.Generator(device="cuda").manual_seed(rows + K)
    x = torch.randn((rows, K), generator=g, device="cuda")
    x *= torch.where(torch.rand(K, generator=g, device="cuda") < 0.02, 10.0, 1.0)
    # rows apart, and the largest of one in its last eight elements
    wide = torch.full((rows, K + 48), float("nan"), device="cuda", dtype=dtype)
    wide[:, 16:K + 16] = x.to(dtype)
    wide[rows - 1, K + 13] = -77.0
    check(wide[:, 16:K + 16])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [512, 1040, 2048, 4112, 8208, 16400, 50000, 65536, 65552])
def test_a_value_that_is_not_finite_ends_its_row_only(dtype, K):
    print("case quantize int8 length, not finite", dtype, K, flush=True)
    x = torch.randn((7, K), device="cuda").to(dtype)
    for row, at, value in ((0, K - 1, float("nan")), (2, K - 8, float("inf")), (3, K // 2, float("-inf")),
                           (6, 0, float("nan"))):
        x[row, at] = value
    codes, scale = check(x)
    assert torch.isnan(scale[[0, 2, 3, 6]]).all() and torch.isfinite(scale[[1, 4, 5]]).all()
