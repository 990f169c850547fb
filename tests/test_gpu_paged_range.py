"""Paged attention over values at the lower end of bf16's range: a weighted mean
of normal numbers keeps its relative accuracy as long as a weight times a value
does.

n equal scores weigh 1 / n each.  With values of 4 n times the smallest normal
number or more, each product is a normal fp32 number, so the result is off by
the final half step (2^-8 relative), by each weight's 2^-20 above and below the
division and by the fp32 sums' 4 sqrt(n) 2^-24."""

import numpy as np
import pytest
import torch

import bit_quantized_gemm_qgemm_amd as qg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    qg.lib()
    return torch.device("cuda:0")


@pytest.mark.parametrize("n,max_len", [(1, 1), (1, 100000), (2, 2), (17, 17), (500, 500), (5000, 5000)])
@pytest.mark.parametrize("dim,heads", [(64, 4), (128, 20)])
def test_small_values_keep_their_bits(n, max_len, dim, heads):
    print("case small values", n, max_len, dim, heads, flush=True)
    g = torch.Generator(device="cuda").manual_seed(n + dim)
    pages = -(-n // 16)
    # one value per element of the head, the same for every token: 4 n 2^-126 to 2^-90
    low = -126 + 2 + int(np.ceil(np.log2(n)))
    exponent = torch.randint(low, -89, (dim,), generator=g, device="cuda")
    row = torch.ldexp(1 + torch.rand(dim, generator=g, device="cuda"), exponent).bfloat16()
    row = torch.where(torch.rand(dim, generator=g, device="cuda") < 0.5, -row, row)
    v = row.expand(pages, 1, 16, dim).contiguous()
    k = torch.zeros_like(v)
    k[..., 0] = 1
    q = torch.randn((2, heads, dim), generator=g, device="cuda").bfloat16()
    table = torch.arange(pages, device="cuda", dtype=torch.int32).repeat(2, 1)
    lens = torch.full((2,), n, dtype=torch.int32, device="cuda")
    out = qg.qgemm_paged_attention(q, k, v, table, lens, max_len=max_len)
    ref = row.double().expand_as(out)
    err = (out.double() - ref).abs() / ref.abs()
    assert float(err.max()) <= 2.0 ** -8 + 2 * 2.0 ** -20 + 4 * np.sqrt(n) * 2.0 ** -24
    if n == 1:
        assert torch.equal(out, row.expand_as(out))
