"""Pins of the int8 oracle: hand-written cases and independent formulations."""

import numpy as np

import oracle


def test_quantize_by_hand():
    x = np.array([[127.0, -63.5, 0.5, 1.5, -2.5, 0.0], [0.0] * 6, [254.0, -3.0, 1.0, 5.0, -254.0, 253.0]])
    codes, scale = oracle.quantize_int8(x)
    assert scale.tolist() == [1.0, 2.0 ** -126, 2.0]
    # ties go to the even code: 63.5 -> 64, 0.5 -> 0, 1.5 -> 2, 2.5 -> 2, 126.5 -> 126
    assert codes.tolist() == [[127, -64, 0, 2, -2, 0], [0] * 6, [127, -2, 0, 2, -127, 126]]


def test_quantize_of_rows_that_are_not_finite_and_of_tiny_ones():
    x = np.array([[1.0, np.inf], [np.nan, 2.0], [2.0 ** -126, 127 * 2.0 ** -126], [2.0 ** -149, 0.0]])
    codes, scale = oracle.quantize_int8(x)
    assert np.isnan(scale[:2]).all() and (scale[2:] == np.float32(2.0 ** -126)).all()
    assert codes.tolist() == [[0, 0], [0, 0], [1, 127], [0, 0]]


def test_quantize_agrees_with_fp32_division():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((200, 64)) * np.exp(rng.uniform(-30, 30, (200, 1)))).astype(np.float32)
    codes, scale = oracle.quantize_int8(x)
    want = np.abs(x).max(1) / np.float32(127)
    assert (scale == want).all()
    assert (codes == np.rint(x / want[:, None])).all()


def test_products_by_hand():
    a, w = np.array([[1, -128], [127, 2]], np.int8), np.array([[3, -128], [-128, 1]], np.int8)
    y, bound = oracle.gemm_w8a8(a, [0.5, 2.0], w, [1.0, 0.25])
    assert y.tolist() == [[0.5 * (3 + 16384), 0.125 * -256], [2.0 * (381 - 256), 0.5 * (-16256 + 2)]]
    assert (bound == np.abs(y)).all()
    h, _ = oracle.gemm_w8a8(a, [0.0, 2.0], w, [1.0, 0.25], gated=True)
    gate, up = 250.0, -8127.0
    np.testing.assert_allclose(h[:, 0], [0.0, gate / (1 + np.exp(-gate)) * up], rtol=1e-15)


def test_experts_take_their_rows_and_leave_the_others():
    rng = np.random.default_rng(1)
    a, w = rng.integers(-128, 128, (5, 4), dtype=np.int8), rng.integers(-128, 128, (3, 4, 2), dtype=np.int8)
    sa, sw = rng.uniform(0.5, 1, 5), rng.uniform(0.5, 1, (3, 2))
    before = np.full((7, 2), 9.0)
    rows = np.array([4, 0, 0, -1, 3, 5, 2])
    out, _, touched = oracle.gemm_w8a8_experts(a, sa, w, sw, [1, 3, 3, 6], rows, before)
    assert touched.tolist() == [False, True, True, True, True, True, False]
    assert (out[[0, 6]] == 9).all() and (out[[3, 5]] == 0).all()       # rows -1 and 5 name none
    for m, e in ((1, 0), (2, 0), (4, 2)):
        want = [sum(int(a[rows[m], k]) * int(w[e, k, n]) for k in range(4)) * sa[rows[m]] * sw[e, n]
                for n in range(2)]
        np.testing.assert_allclose(out[m], want, rtol=1e-15)


def test_plan_by_hand_and_by_sorting():
    offsets, rows, places = oracle.expert_plan([[2, 0], [7, 2], [-1, 0], [2, 1]], 3)
    assert offsets.tolist() == [0, 2, 3, 6]
    assert rows.tolist() == [0, 2, 3, 0, 1, 3, -1, -1]
    assert places.tolist() == [[3, 0], [-1, 4], [-1, 1], [5, 2]]
    ids = np.random.default_rng(2).integers(-2, 12, (50, 4))
    offsets, rows, places = oracle.expert_plan(ids, 10)
    flat = np.where((ids < 0) | (ids >= 10), 10, ids).ravel()
    order = np.argsort(flat, kind="stable")
    n = int((flat < 10).sum())
    assert rows[:n].tolist() == (order[:n] // 4).tolist()
    assert offsets.tolist() == np.searchsorted(np.sort(flat), np.arange(11)).tolist()
    assert places.ravel()[order[:n]].tolist() == list(range(n))


def test_combine_by_hand():
    y = np.array([[1.0, 2.0], [10.0, 20.0]])
    out, weight = oracle.expert_combine(y, [[1, 0], [-1, 2], [1, 1]], [[0.5, -1.0], [np.nan, 3.0], [1.0, 2.0]])
    assert out.tolist() == [[4.0, 8.0], [0.0, 0.0], [30.0, 60.0]]
    assert weight.tolist() == [[6.0, 12.0], [0.0, 0.0], [30.0, 60.0]]
