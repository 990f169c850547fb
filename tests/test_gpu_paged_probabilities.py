"""How exactly paged attention holds its probabilities: outputs that nearly
cancel show an error of the weights that the output's own rounding hides.

Tokens of two kinds alternate, value 1 with key 1 and value -1 with a key one
step of the type above 1, so out = tanh((s0 - s1) / 2) and weight = sum p |v| =
1.  With u = 2^-24, and the scores exact products:
  - the final rounding, half a step of |out|;
  - each weight is off by 2^-20 relative at most (the exponent's rounding below
    32 and exp2's), the two kinds against each other by twice that;
  - what the probabilities' 16-bit parts leave of them: nothing in bf16 (three
    parts, 24 bits), 2^-22 in fp16 (11 bits and 11 more, rounded to nearest),
    twice for the two kinds;
  - fp32 sums over n tokens: 4 sqrt(n) u.
"""

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


@pytest.mark.parametrize("n,max_len", [(2, 2), (2, 200000), (64, 64), (300, 300), (6000, 6000)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_weights_keep_the_bits_of_fp32(dtype, n, max_len):
    print("case probabilities", dtype, n, max_len, flush=True)
    batch, heads, dim, page = 32, 12, 16, 50
    g = torch.Generator(device="cuda").manual_seed(n)
    pages = -(-n // page)
    odd = torch.arange(pages * page, device="cuda").view(pages, 1, page) % 2 == 1
    k = torch.zeros((pages, 1, page, dim), device="cuda")
    k[..., 0] = torch.where(odd, 1 + torch.finfo(dtype).eps, 1.0)
    v = torch.where(odd, -1.0, 1.0)[..., None].expand(pages, 1, page, dim).contiguous()
    q = torch.zeros((batch, heads, dim), device="cuda")
    q[..., 0] = 0.5 + 7 * torch.rand((batch, heads), generator=g, device="cuda")
    q, k, v = (t.to(dtype) for t in (q, k, v))
    table = torch.arange(pages, device="cuda", dtype=torch.int32).repeat(batch, 1)
    lens = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    out = qg.qgemm_paged_attention(q, k, v, table, lens, scale=0.125, max_len=max_len)
    ref = np.tanh(-q[..., 0].double().cpu().numpy() * 0.125 * torch.finfo(dtype).eps / 2)[..., None]
    half, u = torch.finfo(dtype).eps / 2, 2.0 ** -24
    part = 0.0 if dtype == torch.bfloat16 else 2 * 2.0 ** -22
    tol = half * np.abs(ref) * (1 + 2.0 ** -10) + 2 * 2.0 ** -20 + part + 4 * np.sqrt(n) * u + 2.0 ** -25
    err = np.abs(out.double().cpu().numpy() - ref)
    assert (err <= tol).all(), float((err / tol).max())
