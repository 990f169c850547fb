"""Products of 8-bit integers with token and channel scales on the GPU, dense and
grouped by expert, against the oracle in fp64.

Tolerance.  The sum is exact; its conversion to fp32 and the two scales round once
each: 3 * 2^-24 of |Y|.  The gated form adds, per unit of 2^-24, at most 6 of the
output (the up value's 3, the sum 1 + exp, the quotient, the product) and 6 of
sigmoid(gate) (1 + |gate|) |gate| |up| (the gate's own 3, the exponent's argument 1,
the exponential 2): 2^-21 of the oracle's bound covers both.  The last rounding is
off by half a step: 2^-11 (fp16) or 2^-8 (bf16) of the value, 2^-25 below fp16's
normal range.
"""

import numpy as np
import pytest
import torch

import oracle
import bit_quantized_gemm_qgemm_amd as qg

pytestmark = pytest.mark.gpu
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    qg.lib()
    return torch.device("cuda:0")


def operands(M, K, N, experts=None, seed=0):
    """Codes over the whole range and scales that leave outputs of about 1."""
    rng = np.random.default_rng([M, K, N, experts or 0, seed])
    a = rng.integers(-128, 128, (M, K), dtype=np.int8)
    shape = (K, N) if experts is None else (experts, K, N)
    w = rng.integers(-128, 128, shape, dtype=np.int8)
    sa = rng.uniform(0.3, 1, M).astype(np.float32) / 74
    sw = rng.uniform(0.3, 1, N if experts is None else (experts, N)).astype(np.float32) / (74 * K ** 0.5)
    return a, sa, w, sw


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def close(got, ref, bound, dtype):
    got = got.double().cpu().numpy()
    limit = HALF[dtype] * np.abs(ref) + 2.0 ** -21 * bound + 2.0 ** -25
    bad = np.argwhere(~(np.abs(got - ref) <= limit))
    assert len(bad) == 0, (len(bad), bad[:5].tolist(), got[tuple(bad[0])], ref[tuple(bad[0])])


def dense(M, K, N, gated, dtype, seed=0):
    print("case w8a8", M, K, N, gated, dtype, flush=True)
    a, sa, w, sw = operands(M, K, N, seed=seed)
    packed = qg.qgemm_prepack_w8a8(dev(w), gated=gated)
    out = qg.qgemm_w8a8(dev(a), dev(sa), packed, dev(sw), N, gated=gated, dtype=dtype)
    ref, bound = oracle.gemm_w8a8(a, sa, w, sw, gated)
    close(out, ref, bound, dtype)


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,K,N", [
    (1, 16, 2), (1, 1024, 1024), (2, 144, 34), (15, 4096, 130), (16, 128, 16), (17, 272, 66),
    (31, 512, 258), (32, 640, 32), (33, 1040, 100), (64, 2048, 190), (65, 128, 640), (100, 400, 514),
    (127, 1152, 66), (128, 512, 256), (129, 96, 1030), (255, 256, 258), (256, 1024, 512), (257, 784, 386),
    (400, 2048, 64), (513, 640, 770), (1000, 144, 1026),
])
def test_dense(M, K, N, gated, dtype):
    dense(M, K, N, gated, dtype)


@pytest.mark.parametrize("M,K,N", [(1, 4096, 11008), (16, 4096, 4097), (48, 4096, 2049), (300, 4096, 5505),
                                   (1040, 1024, 2305), (2049, 512, 2047)])
def test_dense_of_ordinary_sizes_and_odd_columns(M, K, N):
    dense(M, K, N, False, torch.bfloat16)


TILES = [(16, 16, 8), (16, 32, 4), (16, 64, 4), (32, 32, 4), (32, 64, 4), (32, 128, 1), (64, 64, 2), (64, 128, 1),
         (96, 256, 1), (128, 128, 1), (128, 256, 1), (256, 256, 1)]


def sizes_of(tile, experts, most):
    """Sizes that take this tile, the cheapest of a grid first, with K tiles of every remainder."""
    found = []
    for M in (1, 17, 70, 129, 200, 300, 385, 513, 700, 1000, 1500, 2049):
        for N in (34, 130, 258, 642, 1282, 2050, 4098, 8194):
            for K in (16, 272, 400, 528, 1040, 2064, 4112):
                if M * N * K <= 1.25e10 and qg.qgemm_w8a8_tile(M, N, K, experts) == tile:
                    found.append((M * N * K + 3 * K * N * max(1, experts) + 20 * M * N, M, N, K))
    out = []
    for _, M, N, K in sorted(found)[:most]:
        out += [(M, N, k) for k in (K, K + 128, K + 256, K + 400)
                if qg.qgemm_w8a8_tile(M, N, k, experts) == tile]
    return out


@pytest.mark.parametrize("tile", TILES)
def test_dense_of_each_tile(tile):
    sizes = sizes_of(tile, 0, 2)
    assert sizes
    for i, (M, N, K) in enumerate(sizes):
        print("tile", tile, flush=True)
        dense(M, K, N, gated=i % 2 == 1 and tile != (16, 16, 8), dtype=list(HALF)[i % 2])


def test_dense_without_k_rows_or_columns():
    print("case w8a8 empty", flush=True)
    f32 = lambda *s: torch.ones(s, device="cuda")
    i8 = lambda *s: torch.zeros(s, dtype=torch.int8, device="cuda")
    for gated, cols in ((False, 6), (True, 3)):
        p = qg.qgemm_prepack_w8a8(i8(0, 6), gated=gated)
        out = torch.full((5, cols), 7.0, dtype=torch.float16, device="cuda")
        assert (qg.qgemm_w8a8(i8(5, 0), f32(5), p, f32(6), 6, gated=gated, out=out) == 0).all()
    p = qg.qgemm_prepack_w8a8(i8(32, 6))
    assert qg.qgemm_w8a8(i8(0, 32), f32(0), p, f32(6), 6).shape == (0, 6)
    p = qg.qgemm_prepack_w8a8(i8(32, 0))
    assert qg.qgemm_w8a8(i8(4, 32), f32(4), p, f32(0), 0).shape == (4, 0)


def test_largest_sums_are_exact():
    """|sum| up to 131056 * 2^14 just below 2^31, for the longest K."""
    print("case w8a8 longest K", flush=True)
    K = 131056
    for M in (3, 70):
        a, w = np.full((M, K), -128, np.int8), np.full((K, 4), -128, np.int8)
        w[:, 1] = 127
        a[1], w[0, 2] = 127, 127
        out = qg.qgemm_w8a8(dev(a), dev(np.full(M, 2.0 ** -16, np.float32)), qg.qgemm_prepack_w8a8(dev(w)),
                            dev(np.full(4, 2.0 ** -14, np.float32)), 4, dtype=torch.bfloat16)
        ref, bound = oracle.gemm_w8a8(a, np.full(M, 2.0 ** -16), w, np.full(4, 2.0 ** -14))
        close(out, ref, bound, torch.bfloat16)


@pytest.mark.parametrize("M", [3, 40, 300])
def test_rows_of_nan_scales_stay_their_own(M):
    """A row whose scale is NaN is NaN; no other row is touched by it.  A weight scale of infinity
    makes its column infinite where the sum is not zero."""
    print("case w8a8 nan", M, flush=True)
    a, sa, w, sw = operands(M, 256, 70)
    sa[1], sw[5] = np.nan, np.inf
    out = qg.qgemm_w8a8(dev(a), dev(sa), qg.qgemm_prepack_w8a8(dev(w)), dev(sw), 70).double().cpu().numpy()
    assert np.isnan(out[1]).all()
    sums = a.astype(np.int64) @ w.astype(np.int64)
    rest = np.arange(M) != 1
    assert (out[rest, 5] == np.where(sums[rest, 5] == 0, np.nan, np.sign(sums[rest, 5]) * np.inf)).all()
    keep = np.ix_(rest, np.arange(70) != 5)
    ref, bound = oracle.gemm_w8a8(a[rest], sa[rest], w[:, np.arange(70) != 5], sw[np.arange(70) != 5])
    close(torch.from_numpy(out[keep]), ref, bound, torch.bfloat16)


def test_gates_far_from_zero():
    """Gates from -2000 to 2000: silu goes to 0 and to the gate itself."""
    print("case w8a8 far gates", flush=True)
    a = np.ones((40, 16), np.int8)
    w = np.zeros((16, 254), np.int8)
    w[0, :127], w[0, 127:] = np.arange(-63, 64) * 2, 3
    sa = np.linspace(0.01, 16, 40).astype(np.float32)
    sw = np.ones(254, np.float32)
    out = qg.qgemm_w8a8(dev(a), dev(sa), qg.qgemm_prepack_w8a8(dev(w), gated=True), dev(sw), 254, gated=True,
                        dtype=torch.bfloat16)
    ref, bound = oracle.gemm_w8a8(a, sa, w, sw, True)
    close(out, ref, bound, torch.bfloat16)


# ---- by expert ----------------------------------------------------------------

def experts_case(counts, K, N, gated, dtype, gather, lead=0, tail=0, seed=0):
    """Experts with counts[e] rows, `lead` rows before the first and `tail` after the last that must
    stay; gathered rows come from fewer tokens, some of them outside."""
    print("case w8a8 experts", len(counts), sum(counts), K, N, gated, dtype, gather, flush=True)
    rng = np.random.default_rng([sum(counts), K, N, seed])
    M = lead + sum(counts) + tail
    tokens = max(1, M // 3) if gather else M
    a, sa, w, sw = operands(tokens, K, N, len(counts), seed)
    rows = rng.integers(0, tokens, M).astype(np.int32) if gather else None
    if gather and M > 8:
        rows[[2, M // 2]] = [-1, tokens]
    offsets = (lead + np.concatenate([[0], np.cumsum(counts)])).astype(np.int32)
    cols = N // 2 if gated else N
    out = torch.full((M, cols), 7.0, dtype=dtype, device="cuda")
    packed = qg.qgemm_prepack_w8a8(dev(w), gated=gated)
    got = qg.qgemm_w8a8_experts(dev(a), dev(sa), packed, dev(sw), dev(offsets), N,
                                rows=None if rows is None else dev(rows), gated=gated, out=out)
    assert got.data_ptr() == out.data_ptr()
    ref, bound, touched = oracle.gemm_w8a8_experts(a, sa, w, sw, offsets, rows, np.full((M, cols), 7.0), gated)
    close(out, ref, bound, dtype)
    assert (out.cpu()[torch.from_numpy(~touched)] == 7).all()
    assert (~touched).sum() == lead + tail


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("gated,dtype", [(False, torch.float16), (True, torch.bfloat16)])
@pytest.mark.parametrize("counts,K,N", [
    ([1], 16, 2), ([0, 5, 0], 256, 50), ([3, 0, 17, 1, 16, 0, 0, 40], 400, 130),
    ([33] * 5, 128, 66), ([0] * 60 + [1, 2, 3], 272, 34), ([1] * 130, 144, 18), ([300, 1, 257, 0, 64], 512, 258),
    ([700, 20], 144, 514), ([2] * 63 + [0, 9], 1040, 96),
])
def test_experts(counts, K, N, gated, dtype, gather):
    experts_case(counts, K, N, gated, dtype, gather)


def test_experts_leave_rows_outside_as_they_were():
    for gather in (False, True):
        experts_case([5, 0, 21], 256, 66, False, torch.bfloat16, gather, lead=3, tail=14)
        experts_case([0, 0], 256, 66, True, torch.float16, gather, lead=2, tail=5)
        experts_case([150, 0, 90], 256, 66, True, torch.float16, gather, lead=2, tail=300)


@pytest.mark.parametrize("tile", TILES[:-1])    # the largest is for single weights
def test_experts_of_each_tile(tile):
    sizes = sizes_of(tile, 3, 1) + sizes_of(tile, 20, 1)
    assert sizes
    rng = np.random.default_rng(5)
    for i, (M, N, K) in enumerate(sizes):
        experts = 3 if qg.qgemm_w8a8_tile(M, N, K, 3) == tile else 20
        cuts = np.sort(rng.integers(0, M + 1, experts - 1))
        counts = np.diff(np.concatenate([[0], cuts, [M]]))
        print("tile", tile, flush=True)
        experts_case(list(counts), K, N, i % 2 == 1 and tile != (16, 16, 8), list(HALF)[i % 2], i % 3 != 1)


@pytest.mark.parametrize("experts", [63, 64, 65, 127, 128, 257, 1024])
def test_many_experts_of_few_rows(experts):
    rng = np.random.default_rng(experts)
    experts_case(list(rng.integers(0, 4, experts)), 32, 18, False, torch.float16, True)


def test_offsets_outside_the_rows():
    """Offsets below 0 and past M are held to the rows that there are."""
    print("case w8a8 experts offsets", flush=True)
    a, sa, w, sw = operands(20, 64, 24, 3)
    offsets = np.array([-5, 4, 4, 1000], np.int32)
    out = torch.full((20, 24), 7.0, dtype=torch.bfloat16, device="cuda")
    qg.qgemm_w8a8_experts(dev(a), dev(sa), qg.qgemm_prepack_w8a8(dev(w)), dev(sw), dev(offsets), 24, out=out)
    ref, bound, touched = oracle.gemm_w8a8_experts(a, sa, w, sw, offsets, None, np.full((20, 24), 7.0))
    assert touched.all()
    close(out, ref, bound, torch.bfloat16)
    # falling offsets: nothing is written
    guard = torch.full((40, 24), 7.0, dtype=torch.bfloat16, device="cuda")
    qg.qgemm_w8a8_experts(dev(a), dev(sa), qg.qgemm_prepack_w8a8(dev(w)), dev(sw),
                          dev(np.array([15, 3, 20, 0], np.int32)), 24, out=guard[10:30])
    torch.cuda.synchronize()
    assert (guard == 7).all()


def test_falling_offsets_of_many_experts():
    """Row counts that add up to more than 2^31 items."""
    print("case w8a8 falling offsets", flush=True)
    experts, M, K, N = 1024, 60000, 16, 32768
    zeros = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device="cuda")
    offsets = torch.arange(experts + 1, dtype=torch.int32, device="cuda") % 2 * M
    out = torch.full((M, N), 7.0, dtype=torch.float16, device="cuda")
    packed = zeros(qg.qgemm_prepack_w8a8_bytes(experts, K, N), dtype=torch.uint8)
    qg.qgemm_w8a8_experts(zeros(M, K, dtype=torch.int8), zeros(M), packed, zeros(experts, N), offsets, N, out=out)
    assert (out == 7).all()


def test_expert_weights_past_four_gigabytes():
    """Each expert's weight is found by a 64-bit offset."""
    print("case w8a8 experts large", flush=True)
    experts, K, N = 40, 16384, 8192        # 5.4 GB packed
    w = torch.zeros((experts, K, N), dtype=torch.int8, device="cuda")
    w[:, 5, :] = torch.arange(experts, device="cuda", dtype=torch.int8)[:, None] + 1
    packed = qg.qgemm_prepack_w8a8(w)
    del w
    a = torch.ones((experts, K), dtype=torch.int8, device="cuda")
    one = torch.ones(experts, device="cuda")
    out = qg.qgemm_w8a8_experts(a, one, packed, torch.ones((experts, N), device="cuda"),
                                torch.arange(experts + 1, dtype=torch.int32, device="cuda"), N)
    assert (out == torch.arange(1, experts + 1, device="cuda")[:, None]).all()


def test_repeated_calls_are_bit_identical_on_two_streams():
    print("case w8a8 repeat", flush=True)
    a, sa, w, sw = operands(200, 1024, 770, 4)
    args = (dev(a), dev(sa), qg.qgemm_prepack_w8a8(dev(w), gated=True), dev(sw),
            dev(np.array([0, 90, 91, 91, 200], np.int32)), 770)
    first = qg.qgemm_w8a8_experts(*args, gated=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for i in range(4):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(qg.qgemm_w8a8_experts(*args, gated=True))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o.view(torch.int16), first.view(torch.int16))


def test_products_in_a_graph_follow_their_inputs():
    print("case w8a8 graph", flush=True)
    a, sa, w, sw = operands(96, 512, 130, 5)
    A, SA, P, SW = dev(a), dev(sa), qg.qgemm_prepack_w8a8(dev(w)), dev(sw)
    offsets, rows = dev(np.array([0, 50, 50, 60, 61, 96], np.int32)), dev(np.arange(96, dtype=np.int32))
    out = torch.zeros((96, 130), dtype=torch.float16, device="cuda")
    call = lambda: qg.qgemm_w8a8_experts(A, SA, P, SW, offsets, 130, rows=rows, out=out)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for new in ([0, 1, 2, 3, 4, 96], [0, 0, 0, 0, 0, 0], [0, 20, 40, 60, 80, 90]):
        offsets.copy_(torch.tensor(new, dtype=torch.int32))
        rows.copy_(rows.flip(0))
        out.fill_(7)
        ref, bound, _ = oracle.gemm_w8a8_experts(a, sa, w, sw, new, rows.cpu().numpy(), np.full((96, 130), 7.0))
        g.replay()
        torch.cuda.synchronize()
        close(out, ref, bound, torch.float16)
