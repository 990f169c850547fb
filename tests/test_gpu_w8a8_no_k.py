"""Int8 products without K on the GPU: the sums are empty, so the outputs are 0 times the
scales, and nothing of the weight or the codes is read.  Few rows take workgroups of 16 of
them, more rows the larger tiles."""

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


def i8(*shape):
    return torch.zeros(shape, dtype=torch.int8, device="cuda")


def expected(M, N, gated, scales, owned):
    """0 of every row that an expert has, NaN where its scale is; 7 of the others."""
    ref = np.full((M, N // 2 if gated else N), 7.0)
    ref[owned] = 0
    ref[owned & np.isnan(scales)] = np.nan
    return ref


def same(out, ref):
    np.testing.assert_array_equal(np.abs(out.double().cpu().numpy()), ref)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,N", [(1, 2), (1, 4098), (16, 66), (40, 34), (300, 130), (2049, 514)])
def test_dense(M, N, gated, dtype):
    print("case w8a8 no k", M, N, gated, dtype, flush=True)
    scales = np.linspace(0.5, 2, M).astype(np.float32)
    scales[M // 2] = np.nan
    out = torch.full((M, N // 2 if gated else N), 7.0, dtype=dtype, device="cuda")
    qg.qgemm_w8a8(i8(M, 0), torch.from_numpy(scales).cuda(), qg.qgemm_prepack_w8a8(i8(0, N), gated=gated),
                  torch.ones(N, device="cuda"), N, gated=gated, out=out)
    same(out, expected(M, N, gated, scales, np.ones(M, bool)))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("counts,N", [([1], 2), ([3, 0, 17, 1], 66), ([1] * 130, 18), ([0] * 60 + [300, 2], 258),
                                      ([700, 1, 600], 514)])
def test_by_expert(counts, N, gated, dtype):
    print("case w8a8 experts no k", len(counts), sum(counts), N, gated, dtype, flush=True)
    lead, tail, E = 3, 20, len(counts)
    M = lead + sum(counts) + tail
    scales = np.linspace(0.5, 2, M).astype(np.float32)
    scales[lead] = np.nan
    offsets = torch.from_numpy((lead + np.concatenate([[0], np.cumsum(counts)])).astype(np.int32)).cuda()
    out = torch.full((M, N // 2 if gated else N), 7.0, dtype=dtype, device="cuda")
    qg.qgemm_w8a8_experts(i8(M, 0), torch.from_numpy(scales).cuda(),
                          qg.qgemm_prepack_w8a8(i8(E, 0, N), gated=gated), torch.ones((E, N), device="cuda"),
                          offsets, N, gated=gated, out=out)
    owned = np.zeros(M, bool)
    owned[lead:M - tail] = True
    same(out, expected(M, N, gated, scales, owned))


def test_many_rows_of_many_experts():
    """65536 rows of 1024 experts by 32767 columns: of the smallest tile the launch would have
    2^32 threads and more."""
    print("case w8a8 no k, many", flush=True)
    M, N, E = 65536, 32767, 1024
    out = torch.full((M, N), 7.0, dtype=torch.float16, device="cuda")
    offsets = torch.arange(E + 1, device="cuda", dtype=torch.int32) * (M // E)
    qg.qgemm_w8a8_experts(i8(M, 0), torch.ones(M, device="cuda"), qg.qgemm_prepack_w8a8(i8(E, 0, N)),
                          torch.ones((E, N), device="cuda"), offsets, N, out=out)
    assert (out == 0).all()
