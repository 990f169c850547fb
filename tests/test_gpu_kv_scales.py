"""e4m3 codes of the cache append at many scales: every 16-bit value over each
of a spread of scales, exactly the code of the fp32 quotient."""

import numpy as np
import pytest
import torch

import oracle
import bit_quantized_gemm_qgemm_amd as qg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    qg.lib()
    return torch.device("cuda:0")


def scales(kind, n):
    rng = np.random.default_rng(7)
    if kind == "plain":          # mantissas of every kind, the exponents of real scales
        return (rng.uniform(1, 2, n) * 2.0 ** rng.integers(-12, 4, n)).astype(np.float32)
    if kind == "near one":       # next to powers of two, where quotients come close to ties
        steps = rng.integers(-40, 41, n)
        return ((1 + steps * 2.0 ** -23) * 2.0 ** rng.integers(-8, 3, n)).astype(np.float32)
    if kind == "edges":          # both sides of the borders of the short division, and negative
        ends = [2.0 ** -60, 2.0 ** 60]
        out = [f(np.float32(e), np.float32(t)) for e in ends for t in (0, np.inf)
               for f in (np.nextafter, lambda e, t: e)]
        return np.array((out + [-x for x in out] + [-0.37, -1.0, np.inf, np.nan, 1e-38])[:n], np.float32)
    return (rng.uniform(1, 2, n) * 2.0 ** rng.integers(-62, 62, n)).astype(np.float32)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("kind", ["plain", "near one", "edges", "wide"])
def test_codes_of_every_value_over_many_scales(dtype, kind):
    print("case append scales", dtype, kind, flush=True)
    s = scales(kind, 48)
    heads, dim, tokens = len(s), 256, 256
    allv = torch.arange(65536, device="cuda").to(torch.int32).to(torch.int16).view(dtype)
    x = allv.view(tokens, 1, dim).expand(tokens, heads, dim)
    caches = [torch.zeros((16, heads, 16, dim), dtype=torch.uint8, device="cuda") for _ in range(2)]
    ks = torch.from_numpy(s).cuda()
    qg.qgemm_kv_append(x, x, torch.arange(tokens, device="cuda"), *caches, k_scale=ks,
                       v_scale=ks.flip(0).contiguous())
    values = allv.float().cpu().numpy()
    for cache, order in ((caches[0], s), (caches[1], s[::-1])):
        got = cache.transpose(1, 2).reshape(tokens, heads, dim).cpu().numpy()
        for h, scale in enumerate(order):
            with np.errstate(all="ignore"):
                f = values / np.float32(scale)
                ref = np.where(np.isnan(f), 0x7F, oracle.e4m3fn_encode(np.nan_to_num(
                    np.clip(f, np.float32(-448), np.float32(448))))).astype(np.uint8)
            code = got[:, h].reshape(-1)
            nan = np.isnan(f)
            np.testing.assert_array_equal((code & 0x7F) == 0x7F, nan, err_msg=str(scale))
            np.testing.assert_array_equal(code[~nan], ref[~nan], err_msg=str(scale))
