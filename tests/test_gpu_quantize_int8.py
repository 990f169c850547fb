"""int8 codes and scales of rows on the GPU, against the oracle: every result is exact."""

import numpy as np
import pytest
import torch

import oracle
import bit_quantized_gemm_qgemm_amd as qg

pytestmark = pytest.mark.gpu
TYPES = [torch.float16, torch.bfloat16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    qg.lib()
    return torch.device("cuda:0")


def check(x, out=None):
    codes, scale = qg.qgemm_quantize_int8(x, out=out)
    want_codes, want_scale = oracle.quantize_int8(x.double().cpu().numpy())
    np.testing.assert_array_equal(scale.cpu().numpy(), want_scale)
    np.testing.assert_array_equal(codes.cpu().numpy(), want_codes)
    return codes, scale


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,K", [(1, 16), (5, 48), (64, 512), (3, 528), (7, 2032), (2, 2064), (16, 4096),
                                    (33, 8192), (5, 11008), (2, 16400), (3, 32768), (1, 131056)])
def test_matches_the_oracle(dtype, rows, K):
    print("case quantize int8", dtype, rows, K, flush=True)
    g = torch.Generator(device="cuda").manual_seed(rows + K)
    x = torch.randn((rows, K), generator=g, device="cuda")
    x *= torch.where(torch.rand(K, generator=g, device="cuda") < 0.02, 10.0, 1.0)
    check(x.to(dtype))


@pytest.mark.parametrize("dtype", TYPES)
def test_every_magnitude_and_ties(dtype):
    print("case quantize int8 magnitudes", dtype, flush=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    # rows from the type's smallest values to its largest
    low, high = (-24, 15) if dtype == torch.float16 else (-149, 127)
    e = torch.arange(low, high + 1, device="cuda", dtype=torch.float32)
    x = torch.randn((len(e), 256), generator=g, device="cuda").clamp(-1.9, 1.9).double() * 2.0 ** e[:, None].double()
    check(x.to(dtype))
    # rows whose largest is 127 steps of a power of two: half of the quotients are ties
    x = torch.arange(-254, 255, device="cuda").double() / 2
    x = torch.nn.functional.pad(x, (0, 512 - 509)) * 2.0 ** e[: len(e) - 8, None].double()
    check(x.to(dtype))
    check(torch.zeros((4, 64), device="cuda", dtype=dtype))


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_that_are_not_finite(dtype):
    print("case quantize int8 not finite", dtype, flush=True)
    x = torch.randn((9, 4112), device="cuda").to(dtype)
    for row, at, value in ((0, 0, float("inf")), (2, 4111, float("-inf")), (3, 2048, float("nan")),
                           (5, 77, float("nan")), (5, 78, float("inf")), (8, 4096, float("inf"))):
        x[row, at] = value
    codes, scale = check(x)
    assert torch.isnan(scale[[0, 2, 3, 5, 8]]).all() and (codes[[0, 2, 3, 5, 8]] == 0).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_strided_rows_and_given_outputs(dtype):
    print("case quantize int8 strided", dtype, flush=True)
    wide = torch.randn((13, 3 * 1040), device="cuda").to(dtype)
    codes = torch.full((15, 1040), 55, dtype=torch.int8, device="cuda")
    scale = torch.full((15,), 9.0, device="cuda")
    got = check(wide[:, 1040:2080], out=(codes[1:14], scale[1:14]))
    assert got[0].data_ptr() == codes[1:14].data_ptr()
    assert (codes[[0, 14]] == 55).all() and (scale[[0, 14]] == 9).all()
    check(wide[:1, 16:32].expand(5, 16))                 # one row read five times
    check(wide.t().contiguous().t()[:, :0])              # no columns
    codes, scale = qg.qgemm_quantize_int8(wide[:0, :64])
    assert codes.shape == (0, 64) and scale.shape == (0,)


def test_more_rows_than_one_dimension_holds():
    """2^26 rows of 16 and 2^24 of 2064: workgroups of 256 threads, 2^32 and more of them together."""
    print("case quantize int8 many rows", flush=True)
    pattern = torch.randn((1025, 16), device="cuda").bfloat16()
    want = qg.qgemm_quantize_int8(pattern)
    times = 2 ** 26 // 1025 + 2
    codes, scale = qg.qgemm_quantize_int8(pattern.repeat(times, 1))
    assert torch.equal(codes.view(times, -1), want[0].view(1, -1).expand(times, -1))
    assert torch.equal(scale.view(times, -1), want[1].view(1, -1).expand(times, -1))
    del codes, scale
    row, rows = torch.randn((1, 2064), device="cuda").bfloat16(), 2 ** 24 + 3
    want = qg.qgemm_quantize_int8(row)
    out = (torch.empty((rows, 2064), dtype=torch.int8, device="cuda"), torch.zeros(rows, device="cuda"))
    qg.qgemm_quantize_int8(row.expand(rows, 2064), out=out)
    assert (out[1] == want[1]).all()
    for r in (0, 1, 2 ** 20 - 1, 2 ** 20, 2 ** 23 + 5, 2 ** 24 - 1, 2 ** 24, rows - 1):
        assert torch.equal(out[0][r], want[0][0])


def test_on_another_stream_and_in_a_graph():
    print("case quantize int8 graph", flush=True)
    x = torch.randn((31, 4096), device="cuda").to(torch.bfloat16)
    out = (torch.empty((31, 4096), dtype=torch.int8, device="cuda"), torch.empty(31, device="cuda"))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        check(x, out=out)
    torch.cuda.current_stream().wait_stream(stream)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qg.qgemm_quantize_int8(x, out=out)
    for i in range(3):
        x.mul_(1.5 + i)
        want = oracle.quantize_int8(x.double().cpu().numpy())
        g.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(out[0].cpu().numpy(), want[0])
        np.testing.assert_array_equal(out[1].cpu().numpy(), want[1])


def test_refusals():
    x = torch.randn((4, 64), device="cuda")
    with pytest.raises(qg.QgemmError):                   # K is no multiple of 16
        qg.qgemm_quantize_int8(torch.randn((4, 40), device="cuda"))
    with pytest.raises(qg.QgemmError):                   # rows not 16 bytes apart
        qg.qgemm_quantize_int8(torch.randn((4, 66), device="cuda")[:, :64])
    with pytest.raises(qg.QgemmError):                   # the codes lie in x
        qg.qgemm_quantize_int8(x, out=(x.view(torch.int8).view(-1)[:256].view(4, 64),
                                       torch.empty(4, device="cuda")))
    with pytest.raises(TypeError):
        qg.qgemm_quantize_int8(x.double())
    with pytest.raises(ValueError):
        qg.qgemm_quantize_int8(x, out=(torch.empty((4, 48), dtype=torch.int8, device="cuda"),
                                       torch.empty(4, device="cuda")))
