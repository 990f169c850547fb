"""Plans whose device counts and the host's count of tokens disagree, up to
counts far past any table: the pages are still given, in bounded time."""

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


def check(cached, added, width, page, free, tokens):
    rng = np.random.default_rng(len(cached) + width)
    batch = len(cached)
    pool = rng.permutation(batch * width + free)
    table, at = np.full((batch, width), -1), 0
    for b in range(batch):
        have = min(-(-max(int(cached[b]), 0) // page), width)
        table[b, :have] = pool[at:at + have]
        at += have
    free_pages = pool[at:at + free]
    ref = oracle.kv_plan(table, cached, added, free_pages, page, tokens)
    t = i32(table)
    out = qg.qgemm_kv_plan(t, i32(cached), i32(added), i32(free_pages), page, tokens)
    for got, want, name in zip((t, *out), ref, ("table", "lens", "cu_tokens", "cu_pages", "slots")):
        np.testing.assert_array_equal(got.cpu().numpy(), want, err_msg=name)


@pytest.mark.parametrize("batch,tokens", [(1, 0), (7, 40), (255, 3), (256, 256), (300, 0), (300, 1500),
                                          (1024, 100), (1030, 1), (2500, 2049), (2500, 90000)])
def test_counts_that_disagree(batch, tokens):
    print("case plan counts", batch, tokens, flush=True)
    rng = np.random.default_rng(batch + tokens)
    cached, added = rng.integers(0, 70, batch), rng.integers(-3, 60, batch)
    check(cached, added, 6, 16, batch * 3, tokens)
    check(cached, np.where(rng.random(batch) < 0.9, 0, added), 6, 16, batch, tokens)
    check(cached, np.ones(batch, int), 9, 7, batch, tokens)


def test_counts_past_the_table():
    print("case plan counts past the table", flush=True)
    check([0, 50, 3, 0], [70000, 3, 100000, 1], 4, 16, 9, 60)
    check([0, 50, 3, 0], [70000, 3, 100000, 1], 4, 16, 9, 0)


def test_the_largest_counts():
    """2^31 - 1 tokens for each of 1100 requests: every sum needs 64 bits."""
    print("case plan largest counts", flush=True)
    batch, width, page, tokens, most = 1100, 3, 16, 5000, 2 ** 31 - 1
    table = i32(np.full((batch, width), -1))
    free = torch.randperm(batch * width - 5, device="cuda", dtype=torch.int32)
    cached = i32(np.zeros(batch))
    cached[1] = most                 # holds more than the table can name: gains nothing
    lens, _, cu_pages, slots = qg.qgemm_kv_plan(table, cached, i32(np.full(batch, most)), free, page,
                                                tokens)
    assert (lens == width * page).all()
    want = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
    rows = [0] + list(range(2, batch))
    flat = torch.full((len(rows) * width,), -1, dtype=torch.int32, device="cuda")
    n = min(len(free), len(flat))
    flat[:n] = free[:n]
    want[rows] = flat.view(-1, width)
    assert torch.equal(table, want)
    assert int(cu_pages[-1]) == len(rows) * width
    at = torch.arange(width * page, device="cuda")
    assert torch.equal(slots[:width * page], free[at // page].long() * page + at % page)
    assert (slots[width * page:] == -1).all()
