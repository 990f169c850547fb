"""Routing around the products grouped by expert on the GPU: the order of the rows
(exact) and the sum of each token's expert outputs, and the whole layer."""

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


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def plan_case(ids, experts, dtype=torch.int64):
    print("case expert plan", ids.shape, experts, dtype, flush=True)
    T, top = ids.shape
    # outputs within larger buffers: nothing around them may change
    offsets = torch.full((experts + 3,), -7, dtype=torch.int32, device="cuda")
    rows = torch.full((T * top + 2,), -7, dtype=torch.int32, device="cuda")
    places = torch.full((T * top + 2,), -7, dtype=torch.int32, device="cuda")
    got = qg.qgemm_expert_plan(dev(ids).to(dtype), experts,
                               out=(offsets[1:-1], rows[1:-1], places[1:-1].view(T, top)))
    for part, want, name in zip(got, oracle.expert_plan(ids, experts), ("offsets", "rows", "places")):
        np.testing.assert_array_equal(part.cpu().numpy(), want, err_msg=name)
    for whole in (offsets, rows, places):
        assert whole[0] == -7 and whole[-1] == -7


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens,top,experts", [
    (1, 1, 1), (1, 8, 64), (7, 3, 5), (32, 8, 128), (64, 1, 2), (65, 2, 63), (100, 6, 64), (513, 4, 65),
    (1000, 8, 256), (1024, 8, 257), (1025, 8, 60), (2049, 8, 1024), (5000, 5, 1000), (9000, 8, 16), (600, 8, 300), (33000, 8, 20), (40000, 7, 1024),
    (70000, 8, 40), (70000, 9, 257), (2 ** 20 // 8 + 1, 8, 256), (150000, 7, 1000),
])
def test_plan_matches_the_oracle(tokens, top, experts, dtype):
    rng = np.random.default_rng(tokens + experts)
    plan_case(rng.integers(0, experts, (tokens, top)), experts, dtype)
    if tokens > 1:
        # an uneven choice, some ids outside
        ids = np.minimum(rng.integers(0, experts, (tokens, top)), rng.integers(-2, experts + 3, (tokens, top)))
        plan_case(ids, experts, dtype)


def test_plan_edges():
    plan_case(np.full((300, 7), 3), 9)                           # all of one expert
    plan_case(np.full((3000, 4), 0), 1)
    plan_case(np.full((50, 4), -1), 6)                           # none at all
    plan_case(np.full((5000, 4), 6), 6)
    plan_case(np.array([[2 ** 40 + 1, -2 ** 62, 1, 2 ** 31]]), 4)   # ids far outside 32 bits
    plan_case(np.zeros((0, 4), np.int64), 6)                     # no tokens, no choices
    plan_case(np.zeros((5, 0), np.int64), 6)
    plan_case(np.array([[1, 1], [1, 1]]), 2)                     # the same expert twice


def test_plan_in_a_graph_follows_its_ids():
    print("case expert plan graph", flush=True)
    rng = np.random.default_rng(3)
    T, top, experts = 3000, 4, 100
    ids = dev(rng.integers(0, experts, (T, top)))
    ws = torch.empty(qg.qgemm_expert_plan_workspace_bytes(T * top, experts), dtype=torch.uint8, device="cuda")
    out = qg.qgemm_expert_plan(ids, experts, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qg.qgemm_expert_plan(ids, experts, out=out, workspace=ws)
    for i in range(3):
        new = rng.integers(-1, experts // (i + 1) + 2, (T, top))
        ids.copy_(dev(new))
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        for got, want in zip(out, oracle.expert_plan(new, experts)):
            np.testing.assert_array_equal(got.cpu().numpy(), want)


def combine_case(y, places, gates, dtype):
    print("case expert combine", tuple(y.shape), places.shape, dtype, flush=True)
    got = qg.qgemm_expert_combine(y, dev(places.astype(np.int32)), dev(gates))
    ref, weight = oracle.expert_combine(y.double().cpu().numpy(), places, gates)
    # each of the top products and sums rounds once in fp32, then the output by half a step
    limit = HALF[dtype] * np.abs(ref) + 2 * places.shape[1] * 2.0 ** -24 * weight + 2.0 ** -25
    assert (np.abs(got.double().cpu().numpy() - ref) <= limit).all()
    return got


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("tokens,top,N", [(1, 1, 1), (3, 2, 7), (16, 8, 4096), (5, 3, 2049), (77, 6, 1030),
                                          (300, 8, 128), (9, 17, 264), (2, 8, 11008), (1000, 1, 15),
                                          (40, 9, 2056)])
def test_combine_matches_the_oracle(tokens, top, N, dtype):
    rng = np.random.default_rng(tokens + N)
    rows = tokens * top + 3
    y = torch.randn((rows, N), generator=torch.Generator("cuda").manual_seed(N), device="cuda").to(dtype)
    places = rng.permutation(rows)[:tokens * top].reshape(tokens, top)
    places[rng.random(places.shape) < 0.2] = -1
    gates = rng.standard_normal((tokens, top)).astype(np.float32)
    combine_case(y, places, gates, dtype)


def test_combine_edges():
    y = torch.randn((6, 40), device="cuda").half()
    y[4] = float("nan")
    y[5] = float("inf")
    # places outside are left out whatever their gate; the same row twice
    places = np.array([[-1, 0], [6, 1], [-1, -2 ** 31], [2, 2], [2 ** 31 - 1, 3]])
    gates = np.array([[np.nan, 1], [np.inf, 2], [1, np.nan], [1, 2], [np.nan, 0]], np.float32)
    got = combine_case(y, places, gates, torch.float16)
    assert (got[2] == 0).all()
    out = qg.qgemm_expert_combine(y, dev(np.array([[4, 0], [5, 0]], np.int32)), torch.ones((2, 2), device="cuda"))
    assert torch.isnan(out[0]).all() and torch.isinf(out[1]).all()
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    assert (qg.qgemm_expert_combine(y[:0], i32(3, 2), torch.ones((3, 2), device="cuda")) == 0).all()
    assert (qg.qgemm_expert_combine(y, i32(3, 0), torch.ones((3, 0), device="cuda")) == 0).all()
    assert qg.qgemm_expert_combine(y, i32(0, 2), torch.ones((0, 2), device="cuda")).shape == (0, 40)
    # cancelling terms keep fp32's accuracy: 1000 - 1000 + 2^-10
    y = torch.tensor([[1000.0] * 9, [-1000.0] * 9, [2.0 ** -10] * 9], device="cuda").bfloat16()
    got = qg.qgemm_expert_combine(y, dev(np.array([[0, 1, 2]], np.int32)), torch.ones((1, 3), device="cuda"))
    assert (got == 2.0 ** -10).all()


def layer(x, ids, gates, weights, F, held):
    """A mixture-of-experts layer as a serving loop runs it."""
    (p1, s1), (p2, s2) = weights
    codes, scale = qg.qgemm_quantize_int8(x)
    offsets, rows, places = qg.qgemm_expert_plan(ids, held)
    h = torch.zeros((rows.shape[0], F), dtype=x.dtype, device="cuda")
    qg.qgemm_w8a8_experts(codes, scale, p1, s1, offsets, 2 * F, rows=rows, gated=True, out=h)
    codes, scale = qg.qgemm_quantize_int8(h)
    y = torch.zeros((rows.shape[0], x.shape[1]), dtype=x.dtype, device="cuda")
    qg.qgemm_w8a8_experts(codes, scale, p2, s2, offsets, x.shape[1], out=y)
    return qg.qgemm_expert_combine(y, places, gates)


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("tokens", [1, 9, 200])
def test_a_whole_layer(tokens, dtype):
    """Against the layer in fp64 with the same weights and unquantized activations.

    Each quantizer is off by half a step of its row's largest value over 127 (2^-8 of it); over
    normal activations, whose largest of 256 is below 5 deviations, that is 5 * 2^-8 / sqrt(3) of a
    deviation, 2^-6.4, and a product of independent errors keeps the ratio.  Activations behind a
    gate have heavier tails: their largest is below 30 of their root mean square (a product of two
    such normals), 30 * 2^-8 / sqrt(3) = 2^-3.9 at most.  Together below 2^-3."""
    print("case expert layer", tokens, dtype, flush=True)
    K, F, E, held, top = 256, 160, 12, 9, 4
    g = torch.Generator("cuda").manual_seed(tokens)
    x = torch.randn((tokens, K), generator=g, device="cuda").to(dtype)
    ids = torch.stack([torch.randperm(E, generator=g, device="cuda")[:top] for _ in range(tokens)])
    gates = torch.rand((tokens, top), generator=g, device="cuda") + 0.1

    def weight(k, n):
        w = torch.randint(-127, 128, (held, k, n), generator=g, device="cuda", dtype=torch.int8)
        return w, (torch.rand((held, n), generator=g, device="cuda") + 0.5) / (74 * k ** 0.5)

    (w1, s1), (w2, s2) = weight(K, 2 * F), weight(F, K)
    packed = ((qg.qgemm_prepack_w8a8(w1, gated=True), s1), (qg.qgemm_prepack_w8a8(w2), s2))
    got = layer(x, ids, gates, packed, F, held).double().cpu()
    d1, d2 = (w1.double() * s1.double()[:, None]).cpu(), (w2.double() * s2.double()[:, None]).cpu()
    ref = torch.zeros(tokens, K, dtype=torch.float64)
    for t in range(tokens):
        for j in range(top):
            e = int(ids[t, j])
            if e < held:
                y = x[t].double().cpu() @ d1[e]
                ref[t] += float(gates[t, j]) * ((torch.nn.functional.silu(y[:F]) * y[F:]) @ d2[e])
    assert float((got - ref).norm()) <= 2.0 ** -3 * float(ref.norm())


def layer_inputs(tokens, seed):
    K, F, E, top, dtype = 256, 96, 10, 3, torch.bfloat16
    g = torch.Generator("cuda").manual_seed(seed)
    weights = []
    for k, n, gated in ((K, 2 * F, True), (F, K, False)):
        w = torch.randint(-127, 128, (E, k, n), generator=g, device="cuda", dtype=torch.int8)
        s = torch.rand((E, n), generator=g, device="cuda") / (74 * k ** 0.5)
        weights.append((qg.qgemm_prepack_w8a8(w, gated=gated), s))
    x = torch.randn((tokens, K), generator=g, device="cuda").to(dtype)
    ids = torch.randint(0, E + 2, (tokens, top), generator=g, device="cuda")
    return x, ids, torch.rand((tokens, top), generator=g, device="cuda"), weights, F, E


@pytest.mark.parametrize("tokens", [2, 2000])
def test_a_captured_layer_follows_its_inputs(tokens):
    """One graph for any routing: the sizes of the experts are read on the device."""
    print("case captured layer", tokens, flush=True)
    x, ids, gates, weights, F, E = layer_inputs(tokens, 1)
    layer(x, ids, gates, weights, F, E)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = layer(x, ids, gates, weights, F, E)
    for i in range(4):
        ids.copy_(torch.randint(-1, E // (i + 1) + 1, ids.shape, device="cuda"))
        x.copy_(torch.randn(x.shape, device="cuda"))
        want = layer(x, ids, gates, weights, F, E)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        out.zero_()


def test_layers_on_two_streams():
    """Calls on different streams with storage of their own do not disturb each other."""
    print("case layers on two streams", flush=True)
    inputs = [layer_inputs(tokens, tokens) for tokens in (1500, 37)]
    want = [layer(*i) for i in inputs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in inputs]
    got = [[], []]
    for _ in range(5):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got[i].append(layer(*inputs[i]))
    torch.cuda.synchronize()
    for outs, ref in zip(got, want):
        assert all(torch.equal(o, ref) for o in outs)
