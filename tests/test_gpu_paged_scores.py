"""Scores out of fp32's range."""

import numpy as np
import pytest
import torch

import oracle
import bit_quantized_gemm_qgemm_amd as qg

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    qg.lib()
    return torch.device("cuda:0")


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def pools(n, dtype, seed=0, dim=64, batch=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    pages = batch * -(-n // 16)
    k, v = (torch.randn((pages, 1, 16, dim), generator=g, device="cuda").to(dtype) for _ in "kv")
    return k, v, torch.arange(pages, device="cuda", dtype=torch.int32).view(batch, -1)


@pytest.mark.parametrize("n,max_len", [(1, 1), (300, 300), (40, 50000), (9000, 9000)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_scores_below_the_range(dtype, n, max_len):
    """Keys of -infinity, and dot products below fp32's range: the token weighs
    nothing, and a request of nothing else gets zeros, as in the oracle."""
    print("case scores below the range", dtype, n, max_len, flush=True)
    low = [-INF] + ([-torch.finfo(dtype).max] if dtype == torch.bfloat16 else [])
    for key in low:
        k, v, table = pools(n, dtype)
        q = torch.ones((1, 2, 64), dtype=dtype, device="cuda")
        q *= 2.0 if key == -INF else torch.finfo(dtype).max
        k.fill_(key)
        out = qg.qgemm_paged_attention(q, k, v, table, i32([n]), max_len=max_len)
        assert not out.any(), key
        with np.errstate(all="ignore"):
            args = [t.float().cpu().numpy() for t in (q, k, v)]
            args[1][args[1] < -1e38] = -INF          # what fp32 makes of the product
            ref, _, _ = oracle.paged_attention(*args, table.cpu().numpy(), [n], 64 ** -0.5)
        assert not ref.any()
        # one token in range has all the weight
        t = n // 2
        k[int(table[0, t // 16]), 0, t % 16] = 0
        out = qg.qgemm_paged_attention(q, k, v, table, i32([n]), max_len=max_len)
        assert torch.equal(out, v[int(table[0, t // 16]), 0, t % 16].expand_as(out)), key
