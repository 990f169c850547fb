"""The plan of a routing with the most pairs that it takes, 2^22, and just above 2^21, where a
workgroup's share grows to 8192 pairs.  Exact, against a stable sort on the CPU."""

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


def sorted_pairs(ids, experts):
    flat = ids.reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < experts), flat, experts)
    order = np.argsort(key, kind="stable")
    offsets = np.searchsorted(key[order], np.arange(experts + 1))
    held = np.arange(flat.size) < offsets[-1]
    places = np.empty(flat.size, np.int64)
    places[order] = np.where(held, np.arange(flat.size), -1)
    return offsets, np.where(held, order // ids.shape[1], -1), places.reshape(ids.shape)


def test_the_sort_is_the_oracle():
    import oracle
    ids = np.random.default_rng(0).integers(-1, 9, (100, 3))
    for got, want in zip(sorted_pairs(ids, 7), oracle.expert_plan(ids, 7)):
        np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("experts", [3, 256, 257, 1024])
@pytest.mark.parametrize("tokens,top", [(1 << 19, 8), (1 << 22, 1), ((1 << 21) // 7 + 1, 7), (419430, 10)])
def test_plan(tokens, top, experts, dtype):
    print("case expert plan", tokens, top, experts, dtype, flush=True)
    pairs = tokens * top
    assert 1 << 21 < pairs <= 1 << 22
    rng = np.random.default_rng([tokens, experts])
    # uneven, some ids outside
    ids = np.minimum(rng.integers(-1, experts + 2, (tokens, top)), rng.integers(0, experts + 2, (tokens, top)))
    guarded = lambda n: torch.full((n + 2,), -7, dtype=torch.int32, device="cuda")
    whole = [guarded(experts + 1), guarded(pairs), guarded(pairs)]
    # a workspace of exactly the size, in a larger buffer too
    size = qg.qgemm_expert_plan_workspace_bytes(pairs, experts)
    workspace = torch.full((size + 32,), 0xa5, dtype=torch.uint8, device="cuda")
    out = (whole[0][1:-1], whole[1][1:-1], whole[2][1:-1].view(tokens, top))
    qg.qgemm_expert_plan(torch.from_numpy(ids).cuda().to(dtype), experts, out=out, workspace=workspace[16:size + 16])
    for got, want, name in zip(out, sorted_pairs(ids, experts), ("offsets", "rows", "places")):
        np.testing.assert_array_equal(got.cpu().numpy(), want, err_msg=name)
    for t in whole:
        assert t[0] == -7 and t[-1] == -7
    assert (workspace[:16] == 0xa5).all() and (workspace[-16:] == 0xa5).all()
