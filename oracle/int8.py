"""Products of 8-bit integers with scales for each token and channel, dense and
grouped by expert, and the routing around them.

TEST INFRASTRUCTURE (oracle).  Importable only by the tests, the smoke check
and the benchmark's CPU-baseline leg.

Exact integers and fp64, no code shared with the HIP library.
tests/test_oracle_int8.py pins each function against hand-written cases and an
independent formulation.
"""

import numpy as np


def quantize_int8(x):
    """Rows of x (fp16, fp32, or fp64 holding bf16 values) -> (codes int8, scales
    float32).  Both quotients are fp32 numbers: formed in fp64 and rounded, which
    equals a correctly rounded fp32 division."""
    x = np.asarray(x, dtype=np.float64)
    codes = np.zeros(x.shape, dtype=np.int8)
    scales = np.full(x.shape[0], np.float32(2.0 ** -126), dtype=np.float32)
    for r, row in enumerate(x):
        if not np.isfinite(row).all():
            scales[r] = np.nan
            continue
        if row.size:
            scales[r] = max(np.float32(np.abs(row).max() / 127), np.float32(2.0 ** -126))
        codes[r] = np.rint(np.float32(row / np.float64(scales[r])))
    return codes, scales


def gemm_w8a8(a, a_scale, w, w_scale, gated=False):
    """(out, bound) in fp64; the sum is exact (integers below 2^53).  bound is the
    size that the roundings on the way act on: |Y|, or where gated
    |silu(gate) up| + |sigmoid(gate)| (1 + |gate|) |gate| |up| for an error of the
    gate and one of the up value."""
    sums = a.astype(np.float64) @ w.astype(np.float64)
    y = sums * np.asarray(a_scale, np.float64)[:, None] * np.asarray(w_scale, np.float64)[None, :]
    if not gated:
        return y, np.abs(y)
    half = y.shape[1] // 2
    gate, up = y[:, :half], y[:, half:]
    with np.errstate(over="ignore"):
        sig = 1 / (1 + np.exp(-gate))
    out = gate * sig * up
    return out, np.abs(out) + sig * (1 + np.abs(gate)) * np.abs(gate) * np.abs(up)


def gemm_w8a8_experts(a, a_scale, w, w_scale, offsets, rows, before, gated=False):
    """Rows of each expert in turn; rows that none has keep `before`'s.  Returns
    (out, bound, touched)."""
    out, bound = np.array(before, dtype=np.float64), np.zeros(before.shape)
    touched = np.zeros(len(before), dtype=bool)
    for e in range(len(w)):
        lo = min(max(int(offsets[e]), 0), len(before))
        hi = min(max(int(offsets[e + 1]), lo), len(before))
        for m in range(lo, hi):
            touched[m] = True
            row = m if rows is None else int(rows[m])
            if not 0 <= row < len(a):
                out[m] = 0
        at = np.arange(lo, hi)
        src = at if rows is None else np.asarray(rows)[at]
        ok = (src >= 0) & (src < len(a))
        if ok.any():
            out[at[ok]], bound[at[ok]] = gemm_w8a8(a[src[ok]], np.asarray(a_scale)[src[ok]], w[e],
                                                   w_scale[e], gated)
    return out, bound, touched


def expert_plan(ids, experts):
    """(offsets, rows, places) by a plain walk over the experts."""
    ids = np.asarray(ids)
    tokens, top = ids.shape
    rows, places, offsets = np.full(tokens * top, -1), np.full((tokens, top), -1), [0]
    at = 0
    for e in range(experts):
        for t, j in np.argwhere(ids == e):
            rows[at], places[t, j] = t, at
            at += 1
        offsets.append(at)
    return np.array(offsets), rows, places


def expert_combine(y, places, gates):
    """(out, weight) in fp64; weight = sum_j |gate| |y|, the size that errors act on."""
    y, gates = np.asarray(y, np.float64), np.asarray(gates, np.float64)
    out = np.zeros((len(places), y.shape[1]))
    weight = np.zeros(out.shape)
    for t, row in enumerate(places):
        for j, place in enumerate(row):
            if 0 <= place < len(y):
                out[t] += gates[t, j] * y[place]
                weight[t] += abs(gates[t, j]) * np.abs(y[place])
    return out, weight
