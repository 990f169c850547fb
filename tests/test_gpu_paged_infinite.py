"""Paged attention over values that are not finite, and over the largest finite
ones, at tokens of any weight.

A softmax weight is above 0 wherever the score is finite, so an infinite value
gives an infinite output however far its score lies below the largest, two of
opposite signs NaN, and a score of -infinity, whose weight is 0, NaN.  Other
elements of the head do not see any of it.  A finite value whose weight is out
of fp32's range adds nothing."""

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


class Line:
    """One request of n tokens of value 1 and score 0, over one kv head; tokens
    are changed one by one.  Head 0 has scores of k, head 1 of k / 2."""

    def __init__(self, n, dtype, dim=64):
        pages = -(-n // 16) + 1
        self.k, self.v = (torch.zeros((pages, 1, 16, dim), dtype=dtype, device="cuda") for _ in "kv")
        self.v += 1
        self.q = torch.zeros((1, 2, dim), dtype=dtype, device="cuda")
        self.q[0, :, 0] = torch.tensor([1.0, 0.5])
        self.table = torch.arange(pages, device="cuda", dtype=torch.int32).flip(0)[None].contiguous()
        self.n = n

    def set(self, t, score, value, at):
        page = int(self.table[0, t // 16])
        self.k[page, 0, t % 16, 0] = score
        self.v[page, 0, t % 16, at] = value

    def run(self):
        lens = torch.tensor([self.n], dtype=torch.int32, device="cuda")
        return qg.qgemm_paged_attention(self.q, self.k, self.v, self.table, lens, max_len=self.n,
                                        scale=1.0).float()

    def others(self, out, *at):
        keep = [d for d in range(out.shape[2]) if d not in at]
        return out[:, :, keep]


# where the token lies: in the tile of token 0, in other waves' tiles, in later
# tiles of the same waves, and in other workgroups' shares
PLACES = [(1, 0), (33, 5), (300, 31), (300, 32), (300, 100), (300, 140), (300, 299), (9000, 3),
          (9000, 4500), (9000, 8999)]


@pytest.mark.parametrize("n,t", PLACES)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_infinite_values_stay_infinite_at_any_weight(dtype, n, t):
    print("case infinite values", dtype, n, t, flush=True)
    for gap in (0, 10, 25, 30, 45, 70, 100, 200, 1000):
        line = Line(n, dtype)
        line.set(t, -gap, INF, 5)
        line.set(t, -gap, -INF, 50)
        out = line.run()
        assert (out[:, :, 5] == INF).all() and (out[:, :, 50] == -INF).all(), gap
        assert (line.others(out, 5, 50) == 1).all(), gap


@pytest.mark.parametrize("n", [300, 9000])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_what_infinite_values_add_up_to(dtype, n):
    print("case infinite sums", dtype, n, flush=True)
    for a, b in ((3, 4), (3, 40), (3, n - 1), (n // 2, n - 1)):
        line = Line(n, dtype)
        line.set(a, -30, INF, 5)      # the same sign twice, at very different weights
        line.set(b, -300, INF, 5)
        line.set(a, -30, INF, 6)      # opposite signs
        line.set(b, -300, -INF, 6)
        line.set(a, -30, float("nan"), 7)
        line.set(a, -30, INF, 8)      # with a NaN
        line.set(b, -300, float("nan"), 8)
        out = line.run()
        assert (out[:, :, 5] == INF).all() and torch.isnan(out[:, :, 6:9]).all(), (a, b)
        assert (line.others(out, 5, 6, 7, 8) == 1).all(), (a, b)
    # a weight of 0 times infinity
    line = Line(n, dtype)
    line.set(2, -INF, INF, 5)
    line.set(n - 1, -5, INF, 5)
    line.set(n - 2, -5, INF, 6)
    out = line.run()
    assert torch.isnan(out[:, :, 5]).all() and (out[:, :, 6] == INF).all()
    assert (line.others(out, 5, 6) == 1).all()


@pytest.mark.parametrize("n,t", PLACES[1:])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_largest_values_at_small_weights(dtype, n, t):
    """Zeros everywhere but in one token of the largest value, far down: what it
    adds is its weight times its value, 0 where the weight is out of range."""
    print("case largest values far down", dtype, n, t, flush=True)
    most = torch.finfo(dtype).max
    for gap in (4, 10, 60, 400, 1000):
        line = Line(n, dtype)
        line.v.zero_()
        line.set(t, -gap, most, 5)
        out = line.run()
        s = torch.zeros((2, n), dtype=torch.float64)
        s[:, t] = torch.tensor([-gap, -gap / 2], dtype=torch.float64)
        ref = torch.softmax(s, 1)[:, t] * most
        got = out[0, :, 5].double().cpu()
        # half a step; a weight's relative error: its exponent (below 2048, in steps of 2^-13 at
        # most, each operation off by half a one) and the rest by 2^-20
        slack = 2 * (3 * max(gap, 1) * 2.0 ** -23 + 2.0 ** -20) + 4 * n ** 0.5 * 2.0 ** -24
        tol = ref * (torch.finfo(dtype).eps / 2 + slack) + (2.0 ** -23 if dtype == torch.float16 else 0)
        tiny = ref < 2.0 ** -20     # of a weight near or below 2^-126: any part of it may be left
        assert (torch.where(tiny, (got >= 0) & (got <= 2 * ref + tol), (got - ref).abs() <= tol)).all(), \
            (gap, got, ref)
        assert (line.others(out, 5) == 0).all()


@pytest.mark.parametrize("heads,kv_heads,dim,page,order", [
    (4, 2, 16, 3, "phtd"), (6, 2, 80, 24, "pthd"), (20, 1, 96, 16, "phtd"), (3, 3, 112, 16, "phtd"),
    (8, 2, 192, 40, "pthd"), (34, 2, 256, 16, "phtd"), (5, 5, 240, 100, "phtd"),
])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("max_len,window", [(150, 0), (70000, 0), (70000, 97)])
def test_infinite_values_in_all_shapes(heads, kv_heads, dim, page, order, dtype, max_len, window):
    """Infinite and NaN values at random places, in tokens that count and in
    those that do not (past the end, before the window, of missing pages): the
    oracle's infinities and NaN, and everything else within the tolerance of
    test_gpu_paged_attention.py's derivation, here with whole probabilities."""
    print("case infinite shapes", heads, kv_heads, dim, page, order, dtype, max_len, window, flush=True)
    g = torch.Generator(device="cuda").manual_seed(dim + page)
    lens = [150, 0, 1, 33, 149, 64] + ([4000] if max_len > 150 else [])
    blocks = [-(-n // page) for n in lens]
    pages, width = sum(blocks) + 2, max(blocks)
    shape = {"phtd": (pages, 2, kv_heads, page, dim), "pthd": (pages, 2, page, kv_heads, dim)}[order]
    pool = torch.randn(shape, generator=g, device="cuda").to(dtype)
    k, v = (pool[:, j] if order == "phtd" else pool[:, j].transpose(1, 2) for j in (0, 1))
    odd = torch.rand(v.shape, generator=g, device="cuda")
    few = 0.5 / 150
    v[odd < few] = INF
    v[odd > 1 - few] = -INF
    v[(odd > 0.5) & (odd < 0.5 + few / 8)] = float("nan")
    q = (3 * torch.randn((len(lens), heads, dim), generator=g, device="cuda")).to(dtype)
    order = torch.randperm(pages, generator=g, device="cuda").cpu().numpy()
    table, at = np.full((len(lens), width), -1), 0
    for b, n in enumerate(blocks):
        table[b, :n] = order[at:at + n]
        at += n
    table[0, 1] = -1
    scale = 2.0 * dim ** -0.5            # scores some tens apart
    out = qg.qgemm_paged_attention(
        q, k, v, torch.tensor(table, dtype=torch.int32, device="cuda"),
        torch.tensor(lens, dtype=torch.int32, device="cuda"), scale=scale, max_len=max_len,
        window=window).double().cpu().numpy()
    with np.errstate(all="ignore"):
        ref, weight, reach = oracle.paged_attention(*(t.float().cpu().numpy() for t in (q, k, v)), table,
                                                    lens, scale, window=window, max_len=max_len)
    assert (np.isnan(out) == np.isnan(ref)).all()
    assert ((out == INF) == (ref == INF)).all() and ((out == -INF) == (ref == -INF)).all()
    assert np.isinf(ref).any() and np.isfinite(ref).any()
    fine = np.isfinite(ref)
    u = 2.0 ** -24
    part = 0.0 if dtype == torch.bfloat16 else 2.0 ** -22
    tol = (torch.finfo(dtype).eps / 2 * np.abs(ref) * (1 + 2.0 ** -10) + weight *
           (2 * ((dim + 8) * u * reach[..., None] + 2.0 ** -20) + part + 4 * np.sqrt(max(lens)) * u)
           + 2.0 ** -25)
    err = np.abs(out[fine] - ref[fine])
    assert (err <= tol[fine]).all(), float((err / tol[fine]).max())
