"""Block tables, slots and cache writes on the GPU, against the oracle.

Every result here is exact: whole numbers, copies, and e4m3 codes of a
correctly rounded quotient.
"""

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


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def plan_case(batch, width, page, cached, added, free, seed, tokens=None):
    """Run one plan and compare all five results with the oracle's."""
    rng = np.random.default_rng(seed)
    table = np.full((batch, width), -1)
    pool = rng.permutation(batch * width + free + 1)
    at = 0
    for b in range(batch):
        have = min(-(-max(int(cached[b]), 0) // page), width)
        table[b, :have] = pool[at:at + have]
        at += have
    free_pages = pool[len(pool) - free:]
    total = int(np.maximum(added, 0).sum())
    tokens = total if tokens is None else tokens
    ref = oracle.kv_plan(table, cached, added, free_pages, page, tokens)
    wide = i32(np.full((batch, width + 3), -7))
    t = wide[:, :width]                      # a view: rows further apart than they are wide
    t.copy_(i32(table))
    out = qg.qgemm_kv_plan(t, i32(cached), i32(added), i32(free_pages), page, tokens)
    for got, want, name in zip((t, *out), ref, ("table", "lens", "cu_tokens", "cu_pages", "slots")):
        np.testing.assert_array_equal(got.cpu().numpy(), want, err_msg=name)
    assert (wide[:, width:] == -7).all()
    return out


@pytest.mark.parametrize("batch,width,page,most,gain", [
    (1, 1, 1, 0, 1), (1, 5, 16, 40, 1), (8, 260, 16, 4000, 1), (13, 9, 24, 100, 70),
    (255, 4, 32, 90, 3), (256, 4, 7, 20, 2), (257, 3, 128, 300, 40), (1000, 40, 16, 600, 1),
    (3, 600, 16, 5, 4000),
])
def test_plan_matches_the_oracle(batch, width, page, most, gain):
    print("case plan", batch, width, page, most, gain, flush=True)
    rng = np.random.default_rng(batch + page)
    cached = rng.integers(0, most + 1, batch)
    added = rng.integers(0, gain + 1, batch)
    plan_case(batch, width, page, cached, added, batch * width + 1, seed=page)


def test_plan_edges():
    print("case plan edges", flush=True)
    # negative counts, a free list that ends early, tables that end before the tokens do, more and
    # fewer slots than tokens, requests that gain nothing
    cached, added = [-3, 0, 17, 64, 5, 0], [4, -1, 40, 3, 0, 33]
    plan_case(6, 4, 16, cached, added, 3, seed=1)
    plan_case(6, 4, 16, cached, added, 0, seed=2)
    plan_case(6, 4, 16, cached, added, 9, seed=3, tokens=120)
    plan_case(6, 4, 16, cached, added, 9, seed=4, tokens=41)
    plan_case(6, 4, 16, cached, added, 9, seed=5, tokens=0)
    plan_case(300, 2, 16, np.zeros(300, int), np.zeros(300, int), 4, seed=6)
    # an empty batch: sums of nothing, slots of no token
    lens, cu_tokens, cu_pages, slots = qg.qgemm_kv_plan(i32(np.zeros((0, 4))), i32([]), i32([]),
                                                        i32([1, 2]), 16, 5)
    assert lens.numel() == 0 and cu_tokens.tolist() == [0] and cu_pages.tolist() == [0]
    assert slots.tolist() == [-1] * 5
    # a page that a request should hold is missing in its table
    t = i32([[4, -1, 6, -1]])
    out = qg.qgemm_kv_plan(t, i32([18]), i32([20]), i32([9]), 16, 20)
    assert out[3].tolist() == [-1] * 14 + [144 + i for i in range(6)]
    assert t.tolist() == [[4, -1, 9, -1]]      # two pages are held, the third is a new one


def test_plan_in_a_graph_follows_its_inputs():
    print("case plan graph", flush=True)
    batch, width, page = 40, 30, 16
    cached, added = i32(np.arange(batch) * 9), i32(np.ones(batch))
    table, free = i32(np.zeros((batch, width))), i32(np.arange(100))
    out = qg.qgemm_kv_plan(table, cached, added, free, page, batch)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qg.qgemm_kv_plan(table, cached, added, free, page, batch, out=out)
    for i in range(3):
        cached.add_(1 + i)
        free.add_(1)
        table.zero_()
        ref = oracle.kv_plan(table.cpu().numpy(), cached.cpu().numpy(), added.cpu().numpy(),
                             free.cpu().numpy(), page, batch)
        g.replay()
        torch.cuda.synchronize()
        for got, want in zip((table, *out), ref):
            np.testing.assert_array_equal(got.cpu().numpy(), want)


def bits(t):
    """The elements as integers (torch compares NaN unequal)."""
    return t.contiguous().view(torch.uint8 if t.element_size() == 1 else torch.int16)


def append_case(tokens, kv_heads, dim, page, pages, dtype, e4m3, order="phtd", seed=0, x=None,
                slots=None, scales=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    width = (3 * kv_heads) * dim                    # the k and v parts of a fused product's rows
    fused = torch.randn((tokens, width), generator=g, device="cuda").to(dtype) if x is None else x
    k, v = fused[:, :2 * kv_heads * dim].split(kv_heads * dim, dim=1)
    k, v = k.unflatten(1, (kv_heads, dim)), v.unflatten(1, (kv_heads, dim))
    if slots is None:
        slots = torch.randperm(pages * page, generator=g, device="cuda")[:tokens]
    shape = {"phtd": (pages, 2, kv_heads, page, dim), "pthd": (pages, 2, page, kv_heads, dim)}[order]
    pool = torch.randint(0, 100, shape, generator=g, device="cuda").to(torch.uint8)
    pool = pool if e4m3 else pool.to(dtype)
    caches = [pool[:, j] if order == "phtd" else pool[:, j].transpose(1, 2) for j in (0, 1)]
    if scales is None:
        scales = (0.5 + torch.rand((2, kv_heads), generator=g, device="cuda")) / 40
    ks, vs = (scales[0].contiguous(), scales[1].contiguous()) if e4m3 else (None, None)
    before = [c.clone() for c in caches]
    args = caches if not e4m3 else [c.view(torch.float8_e4m3fn) for c in caches]
    qg.qgemm_kv_append(k, v, slots, *args, k_scale=ks, v_scale=vs)
    host = slots.cpu().numpy()
    ok = (host >= 0) & (host < pages * page)
    for part, cache, was, scale in zip((k, v), caches, before, (ks, vs)):
        want = bits(was).clone() if not e4m3 else was.clone()
        if e4m3:
            ref = oracle.kv_append(part.float().cpu().numpy(), host, was.cpu().numpy(),
                                   scale.cpu().numpy())
            got = cache.cpu().numpy()
            nan = (ref & 0x7F) == 0x7F
            np.testing.assert_array_equal((got & 0x7F) == 0x7F, nan)
            np.testing.assert_array_equal(got[~nan], ref[~nan])
        else:
            idx = torch.from_numpy(host[ok]).cuda()
            want[idx // page, :, idx % page] = bits(part)[torch.from_numpy(ok).cuda()]
            assert torch.equal(bits(cache), want)
    return caches


@pytest.mark.parametrize("tokens,kv_heads,dim,page,order", [
    (1, 1, 16, 1, "phtd"), (1, 8, 128, 16, "phtd"), (3, 2, 48, 5, "pthd"), (64, 8, 128, 16, "phtd"),
    (97, 8, 80, 24, "phtd"), (130, 3, 112, 16, "pthd"), (257, 1, 256, 128, "phtd"),
    (33, 32, 64, 32, "pthd"), (19, 5, 208, 48, "phtd"),
])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("e4m3", [False, True])
def test_append_matches_the_oracle(tokens, kv_heads, dim, page, order, dtype, e4m3):
    print("case append", tokens, kv_heads, dim, page, order, dtype, e4m3, flush=True)
    append_case(tokens, kv_heads, dim, page, -(-tokens // page) + 3, dtype, e4m3, order, seed=tokens)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("scale", [1.0, 1 / 32, 0.3, 1e-3, 37.0, 1e-30, 1e30, 1e-42, 0.0])
def test_append_codes_of_every_16_bit_value(dtype, scale):
    """All 65536 bit patterns, infinities and NaN among them, at plain and at
    extreme scales."""
    print("case append all values", dtype, scale, flush=True)
    tokens, dim = 1024, 64
    allv = torch.arange(65536, device="cuda").to(torch.int32).to(torch.int16).view(dtype)
    x = torch.cat([allv.view(tokens, dim), allv.flip(0).view(tokens, dim),
                   torch.zeros((tokens, dim), dtype=dtype, device="cuda")], dim=1)
    scales = torch.tensor([[scale], [scale]], dtype=torch.float32, device="cuda")
    append_case(tokens, 1, dim, 16, 70, dtype, True, x=x, scales=scales)


def test_append_skips_slots_outside_the_pool():
    print("case append skipped slots", flush=True)
    s = torch.tensor([3, -1, 160, 161, -2 ** 62, 2 ** 62, 159, 0, 2 ** 32], device="cuda")
    for e4m3 in (False, True):
        append_case(9, 2, 64, 16, 10, torch.float16, e4m3, slots=s)


def test_append_past_4_gib():
    """A pool of more than 2^32 bytes: rows on both sides of that offset."""
    print("case append past 4 GiB", flush=True)
    kv_heads, page, dim = 8, 16, 128
    pages = (1 << 32) // (kv_heads * page * dim * 2) + 600
    caches = [torch.empty((pages, kv_heads, page, dim), dtype=torch.bfloat16, device="cuda")
              for _ in range(2)]
    far = pages - 500
    x = torch.randn((4, 2 * kv_heads, dim), device="cuda").to(torch.bfloat16)
    slots = torch.tensor([far * page + 5, 7, (pages - 1) * page + 15, 1 << 20], device="cuda")
    for p in (far, 0, pages - 1, (1 << 20) // page):
        for c in caches:
            c[p].zero_()
    qg.qgemm_kv_append(x[:, :kv_heads], x[:, kv_heads:], slots, *caches)
    for j, c in enumerate(caches):
        for i, s in enumerate(slots.tolist()):
            assert torch.equal(c[s // page, :, s % page], x[i, j * kv_heads:(j + 1) * kv_heads])
            assert int((c[s // page] != 0).any(-1).sum()) == kv_heads
    table = i32([[0, far], [far, pages - 1]])
    q = torch.randn((2, kv_heads, dim), device="cuda").to(torch.bfloat16)
    out = qg.qgemm_paged_attention(q, *caches, table, i32([32, 32]))
    rows = [[c[t].double().permute(0, 2, 1, 3).reshape(-1, kv_heads, dim) for c in caches]
            for t in table.long()]
    for b, (kd, vd) in enumerate(rows):
        s = (kd * q[b].double()).sum(-1) * dim ** -0.5
        ref = (torch.softmax(s, 0)[:, :, None] * vd).sum(0)
        size = (torch.softmax(s, 0)[:, :, None] * vd.abs()).sum(0)
        # half a bf16 step of the result, and 2^-14 of the weighted sizes for fp32 arithmetic
        assert ((out[b].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -14 * size).all()
