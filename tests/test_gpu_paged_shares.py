"""Paged attention where workgroups share items: many parts of one item, more
requests than workgroups, empty ones among them, and values at the end of the
type's range.  Tolerances as derived in test_gpu_paged_attention.py."""

import numpy as np
import pytest
import torch

import oracle
import bit_quantized_gemm_qgemm_amd as qg

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    qg.lib()
    return torch.device("cuda:0")


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def check(lens, heads, kv_heads, dim, page, dtype, seed=0, **kw):
    g = torch.Generator(device="cuda").manual_seed(seed)
    batch, blocks = len(lens), [-(-n // page) for n in lens]
    pages = sum(blocks) + 1
    pools = [torch.randn((pages, kv_heads, page, dim), generator=g, device="cuda").to(dtype)
             for _ in range(2)]
    q = torch.randn((batch, heads, dim), generator=g, device="cuda").to(dtype)
    perm = torch.randperm(pages, generator=g, device="cuda").cpu().numpy()
    table, at = np.full((batch, max(1, max(blocks))), -1), 0
    for b, n in enumerate(blocks):
        table[b, :n] = perm[at:at + n]
        at += n
    out = qg.qgemm_paged_attention(q, *pools, i32(table), i32(lens), **kw)
    assert torch.isfinite(out).all()
    ref, weight, reach = oracle.paged_attention(
        q.float().cpu().numpy(), *(p.float().cpu().numpy() for p in pools), table, lens,
        dim ** -0.5, window=kw.get("window", 0))
    half = torch.finfo(dtype).eps / 2
    part = 2.0 ** -16 if dtype == torch.bfloat16 else 2.0 ** -21
    tol = (half * np.abs(ref) * (1 + 2.0 ** -10) + weight *
           (2 * ((dim + 8) * U * reach[..., None] + 2.0 ** -20) + part + 4 * np.sqrt(max(lens)) * U)
           + 2.0 ** -25)
    err = np.abs(out.double().cpu().numpy() - ref)
    assert (err <= tol).all(), float((err / tol).max())
    return out


@pytest.mark.parametrize("lens,heads,kv_heads,dim", [
    ([200000], 2, 1, 16),          # about a thousand parts of one item
    ([100000], 20, 1, 32),         # two items: the heads of one kv head in two chunks
    ([40000, 1, 0, 40000], 3, 3, 80), ([30000], 4, 1, 256), ([70000, 3], 1, 1, 128),
])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_many_parts(lens, heads, kv_heads, dim, dtype):
    print("case many parts", lens, heads, kv_heads, dim, dtype, flush=True)
    check(lens, heads, kv_heads, dim, 64, dtype, seed=dim)


def test_more_requests_than_workgroups():
    print("case more requests than workgroups", flush=True)
    lens = [0 if i % 3 == 1 else (37 * i) % 130 for i in range(1500)]
    lens[1400] = 4000
    out = check(lens, 4, 2, 64, 16, torch.bfloat16, max_len=4100)
    assert not out[[i for i, n in enumerate(lens) if n == 0]].any()
    check(lens, 2, 2, 64, 16, torch.float16, max_len=4100, window=1700)


def test_nothing_to_attend_to_on_the_shared_path():
    print("case all empty", flush=True)
    pools = torch.full((4, 2, 16, 64), float("nan"), device="cuda").half()
    q = torch.randn((900, 4, 64), device="cuda").half()
    out = torch.full_like(q, 7)
    qg.qgemm_paged_attention(q, pools, pools, i32(np.full((900, 400), -1)), i32(np.zeros(900)),
                             max_len=6000, out=out)
    assert not out.any()
    # lengths, but no page: every part is empty
    out.fill_(7)
    qg.qgemm_paged_attention(q, pools, pools, i32(np.full((900, 400), -1)), i32(np.full(900, 5000)),
                             max_len=6000, out=out)
    assert not out.any()


@pytest.mark.parametrize("n", [3, 700, 5000])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_values_at_the_end_of_the_range(n, dtype):
    """Equal scores over the largest values: their mean is that value, though
    their sum is far past the range."""
    print("case largest values", n, dtype, flush=True)
    pages = -(-n // 16)
    k = torch.ones((pages, 1, 16, 128), dtype=dtype, device="cuda")
    v = torch.full_like(k, torch.finfo(dtype).max)
    q = torch.randn((1, 4, 128), device="cuda").to(dtype)
    out = qg.qgemm_paged_attention(q, k, v, i32(np.arange(pages)[None]), i32([n]))
    assert (out == torch.finfo(dtype).max).all()


def test_shared_path_in_a_graph():
    """Lengths that change between replays move the shares about; every replay
    equals the eager call, which runs in between."""
    print("case shares in a graph", flush=True)
    g = torch.Generator(device="cuda").manual_seed(3)
    pools = [torch.randn((400, 2, 16, 80), generator=g, device="cuda").bfloat16() for _ in range(2)]
    q = torch.randn((5, 6, 80), generator=g, device="cuda").bfloat16()
    table = torch.randint(0, 400, (5, 300), generator=g, device="cuda", dtype=torch.int32)
    lens, out = i32([4800, 0, 17, 900, 2600]), torch.empty_like(q)
    ws = torch.empty(qg.qgemm_paged_attention_workspace_bytes(5, 6, 2, 80, 4800), dtype=torch.uint8,
                     device="cuda")

    def call():
        qg.qgemm_paged_attention(q, *pools, table, lens, max_len=4800, out=out, workspace=ws)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(4):
        lens.copy_(lens.roll(1) // (i + 1) + i)
        call()
        torch.cuda.synchronize()
        want = out.clone()
        out.fill_(9)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
