"""Sums of a token's expert outputs whose rows are whole waves (a multiple of 64 pieces of eight
elements): choices below, at and above the eight that are in flight, last pieces part-full, and a
last workgroup that reaches past the last token.  Tolerance as in test_gpu_experts.py."""

import numpy as np
import pytest
import torch

import bit_quantized_gemm_qgemm_amd as qg
from test_gpu_experts import HALF, combine_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    qg.lib()
    return torch.device("cuda:0")


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("tokens,top,N", [(5, 3, 512), (7, 9, 1024), (3, 17, 4096), (5, 6, 4093), (9, 2, 505),
                                          (1, 1, 512), (2, 8, 509), (6, 16, 1023), (33, 5, 2041)])
def test_rows_of_whole_waves(tokens, top, N, dtype):
    assert -(-N // 8) % 64 == 0
    rng = np.random.default_rng(tokens + N)
    rows = tokens * top + 3
    y = torch.randn((rows, N), generator=torch.Generator("cuda").manual_seed(N), device="cuda").to(dtype)
    places = rng.permutation(rows)[:tokens * top].reshape(tokens, top)
    places[rng.random(places.shape) < 0.2] = -1
    combine_case(y, places, rng.standard_normal((tokens, top)).astype(np.float32), dtype)


@pytest.mark.parametrize("dtype", HALF)
def test_nothing_is_written_past_the_last_token(dtype):
    print("case expert combine guard", dtype, flush=True)
    for tokens, N in ((1, 512), (3, 505), (5, 1021)):
        y = torch.ones((tokens, N), dtype=dtype, device="cuda")
        whole = torch.full((16 + tokens * N + 512,), 7.0, dtype=dtype, device="cuda")
        out = whole[16:16 + tokens * N].view(tokens, N)
        qg.qgemm_expert_combine(y, torch.arange(tokens, dtype=torch.int32, device="cuda").view(tokens, 1),
                                torch.full((tokens, 1), 2.0, device="cuda"), out=out)
        assert (out == 2).all() and (whole[:16] == 7).all() and (whole[16 + tokens * N:] == 7).all()
