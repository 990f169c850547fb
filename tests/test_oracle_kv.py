"""Pins of the key-value cache oracle: hand-written cases, torch's e4m3fn cast
and a dense softmax formulation."""

import numpy as np
import torch

import oracle


def test_plan_by_hand():
    # pages of 4; request 0 holds 3 tokens and gains 3, 1 holds 8 and gains 1 (a full last page),
    # 2 gains nothing, 3 starts with 9 tokens in a table of 2 pages (8 tokens at most)
    table = np.full((4, 2), -1)
    table[0, 0], table[1] = 7, (5, 6)
    table, lens, cu_tokens, cu_pages, slots = oracle.kv_plan(
        table, [3, 8, 0, 0], [3, 1, 0, 9], [10, 11], 4, 14)
    assert lens.tolist() == [6, 8, 0, 8]
    assert cu_tokens.tolist() == [0, 3, 4, 4, 13]
    assert cu_pages.tolist() == [0, 1, 1, 1, 3]
    # the free list of two ends inside request 3
    assert table.tolist() == [[7, 10], [5, 6], [-1, -1], [11, -1]]
    assert slots.tolist() == [31, 40, 41, -1, 44, 45, 46, 47, -1, -1, -1, -1, -1, -1]


def test_append_matches_the_e4m3_cast():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((6, 2, 16)) * 3).astype(np.float16)
    x[0, 0, :4] = (np.inf, -np.inf, np.nan, 6e4)
    scale = np.array([0.37, 1e-3], np.float32)
    cache = np.zeros((3, 2, 4, 16), np.uint8)
    got = oracle.kv_append(x, [0, 5, -1, 11, 12, 2], cache, scale)
    f = torch.from_numpy(x).float() / torch.from_numpy(scale)[None, :, None]
    want = f.clamp(-448, 448).to(torch.float8_e4m3fn).float().numpy()
    for t, slot in ((0, 0), (1, 5), (3, 11), (5, 2)):
        np.testing.assert_array_equal(oracle.e4m3fn_decode(got[slot // 4, :, slot % 4]), want[t])
    assert np.count_nonzero(got[0, :, 1]) == 0       # slots nobody names, and the skipped ones
    plain = oracle.kv_append(x, [3, 4, 5, 6, 7, 8], np.zeros((3, 2, 4, 16), np.float16))
    np.testing.assert_array_equal(plain[0, :, 3], x[0])
    np.testing.assert_array_equal(plain[2, :, 0], x[5])


def test_attention_matches_a_dense_softmax():
    rng = np.random.default_rng(1)
    batch, heads, kv_heads, dim, page, n = 2, 6, 2, 16, 4, 10
    q = rng.standard_normal((batch, heads, dim))
    k, v = rng.standard_normal((2, 8, kv_heads, page, dim))
    table = rng.permutation(8)[:6].reshape(2, 3)
    out, weight, reach = oracle.paged_attention(q, k, v, table, [n, 0], 0.25)
    assert not out[1].any() and not weight[1].any()
    kd = torch.from_numpy(k[table[0]]).transpose(0, 1).reshape(kv_heads, 12, dim)[:, :n]
    vd = torch.from_numpy(v[table[0]]).transpose(0, 1).reshape(kv_heads, 12, dim)[:, :n]
    qd = torch.from_numpy(q[0]).reshape(kv_heads, 3, dim)
    p = torch.softmax(qd @ kd.transpose(1, 2) * 0.25, -1)
    np.testing.assert_allclose(out[0], (p @ vd).reshape(heads, dim).numpy(), rtol=1e-12)
    assert (weight[0] >= np.abs(out[0]) - 1e-12).all() and (reach[0] > 0).all()
    # a window of 5 (tokens 5 .. 9) over a missing middle page leaves tokens 8 and 9
    table[0, 1] = -1
    out, _, _ = oracle.paged_attention(q, k, v, table, [n, 0], 0.25, window=5)
    p = torch.softmax(qd @ kd.transpose(1, 2)[..., 8:] * 0.25, -1)
    np.testing.assert_allclose(out[0], (p @ vd[:, 8:]).reshape(heads, dim).numpy(), rtol=1e-12)
