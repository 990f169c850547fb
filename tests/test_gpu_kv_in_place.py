"""Plans that update the lengths in place, as a decode loop does, over one
workgroup and over several."""

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


@pytest.mark.parametrize("batch,most", [(1, 1), (8, 1), (200, 1), (300, 1), (40, 100), (1000, 9),
                                        (3000, 1), (64, 3000), (1, 50000)])
def test_lengths_in_place(batch, most):
    print("case plan in place", batch, most, flush=True)
    rng = np.random.default_rng(batch + most)
    page, steps = 16, 4
    added = rng.integers(0 if most > 1 else 1, most + 1, batch)
    width = -(-steps * most // page)
    tokens = int(added.sum())
    order = rng.permutation(batch * width + 1)
    table, lens, taken = np.full((batch, width), -1), np.zeros(batch, int), 0
    t, n, a = i32(table), i32(lens), i32(added)
    free = i32(order)
    out = (n, i32(np.zeros(batch + 1)), i32(np.zeros(batch + 1)),
           torch.zeros(tokens, dtype=torch.int64, device="cuda"))
    graph = None
    for step in range(steps):
        table, lens, cu_tokens, cu_pages, slots = oracle.kv_plan(table, lens, added, order[taken:], page,
                                                                 tokens)
        if step == 0:
            qg.qgemm_kv_plan(t, n, a, free, page, tokens, out=out)
        else:
            if graph is None:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    qg.qgemm_kv_plan(t, n, a, free, page, tokens, out=out)
            graph.replay()
        torch.cuda.synchronize()
        for got, want, name in zip((t, *out), (table, lens, cu_tokens, cu_pages, slots),
                                   ("table", "lens", "cu_tokens", "cu_pages", "slots")):
            np.testing.assert_array_equal(got.cpu().numpy(), want, err_msg=f"{name} {step}")
        taken += int(cu_pages[-1])
        free.copy_(i32(np.concatenate([order[taken:], np.full(taken, -1)])))


def test_other_overlaps_are_refused():
    print("case plan overlaps", flush=True)
    buf = i32(np.zeros(64))
    t = i32(np.full((4, 8), -1))
    free, added = i32(np.arange(9)), i32(np.ones(4))
    slots = torch.zeros(4, dtype=torch.int64, device="cuda")
    for lens, cu_tokens, cu_pages in ((buf[1:5], buf[8:13], buf[16:21]), (buf[24:28], buf[3:8], buf[16:21]),
                                      (buf[24:28], buf[8:13], buf[10:15]), (added, buf[8:13], buf[16:21])):
        with pytest.raises(qg.QgemmError, match="share"):
            qg.qgemm_kv_plan(t, buf[:4], added, free, 16, 4, out=(lens, cu_tokens, cu_pages, slots))
