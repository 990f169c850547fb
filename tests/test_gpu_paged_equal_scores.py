"""Scores that are all equal, however large: the output is the mean of the values."""

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


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def pools(n, dtype, seed=0, dim=64, batch=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    pages = batch * -(-n // 16)
    k, v = (torch.randn((pages, 1, 16, dim), generator=g, device="cuda").to(dtype) for _ in "kv")
    return k, v, torch.arange(pages, device="cuda", dtype=torch.int32).view(batch, -1)


@pytest.mark.parametrize("n,max_len", [(1, 1), (33, 33), (700, 700), (33, 50000), (9000, 9000)])
@pytest.mark.parametrize("dtype,e4m3", [(torch.float16, False), (torch.bfloat16, False),
                                        (torch.float16, True), (torch.bfloat16, True)])
def test_equal_scores_give_the_plain_mean(dtype, e4m3, n, max_len):
    """Scores of -8e4, 0 and 8e4, each the same for all tokens: an error of the
    score is theirs in common and drops out, so the output is the mean of the
    values to half a step of it, 2^-20 of the mean size for each weight above and
    below the division, 2^-22 for parts of 16 bits, 4 sqrt(n) 2^-24 for sums, and
    2^-25, half the smallest fp16 step."""
    print("case equal scores", dtype, e4m3, n, max_len, flush=True)
    for key in (-100.0, 0.0, 100.0):
        k, v, table = pools(n, dtype, seed=n)
        k.fill_(key)
        q = torch.full((1, 2, 64), 100.0, dtype=dtype, device="cuda")
        scales = (None, None)
        values = v.double()
        if e4m3:
            scales = (torch.full((1,), 100 / 96, device="cuda"), torch.full((1,), 0.01, device="cuda"))
            k = torch.full_like(k, 96.0 * np.sign(key)).to(torch.float8_e4m3fn)
            v = (v.float() * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
            values = v.double() * scales[1].double()
        out = qg.qgemm_paged_attention(q, k, v, table, i32([n]), *scales, max_len=max_len)
        rows = values[table[0].long()].reshape(-1, 64)[:n]
        mean, size = rows.mean(0), rows.abs().mean(0)
        tol = (torch.finfo(dtype).eps / 2 * mean.abs() * (1 + 2.0 ** -10) + 2.0 ** -25
               + size * (2 * 2.0 ** -20 + 2.0 ** -22 + 4 * n ** 0.5 * 2.0 ** -24))
        err = (out.double() - mean).abs()
        assert (err <= tol).all(), (key, float((err / tol).max()))
