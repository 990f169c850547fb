"""Paged key-value cache: plan, append and attention of one new token.

TEST INFRASTRUCTURE (oracle).  Importable only by the tests, the smoke check
and the benchmark's CPU-baseline leg.

Plain loops over requests and tokens in fp64 (exact integers for the plan), no
code shared with the HIP library.  tests/test_oracle_kv.py pins each function
against hand-written cases and an independent formulation.
"""

import numpy as np

from .formats import e4m3fn_decode, e4m3fn_encode


def kv_plan(table, cached, added, free_pages, page_size, tokens):
    """Returns (table, lens, cu_tokens, cu_pages, slots); the table is a copy."""
    table = np.array(table, dtype=np.int64)
    batch, width = table.shape
    lens, cu_tokens, cu_pages = [], [0], [0]
    slots = np.full(tokens, -1, dtype=np.int64)
    taken = 0
    at = 0
    for b in range(batch):
        c, a = max(int(cached[b]), 0), max(int(added[b]), 0)
        n = min(c + a, width * page_size)
        for page in range(min(-(-c // page_size), width), -(-n // page_size)):
            table[b, page] = free_pages[taken] if taken < len(free_pages) else -1
            taken += 1
        for pos in range(c, c + a):
            if at < tokens and pos < width * page_size and table[b, pos // page_size] >= 0:
                slots[at] = table[b, pos // page_size] * page_size + pos % page_size
            at += 1
        lens.append(n)
        cu_tokens.append(at)
        cu_pages.append(taken)
    return table, np.array(lens), np.array(cu_tokens), np.array(cu_pages), slots


def kv_append(x, slots, cache, scale=None):
    """x [tokens, kv_heads, dim] into a copy of cache [pages, kv_heads,
    page_size, dim] (uint8 e4m3fn codes when scale is given: the fp32 quotient
    rounded to nearest even, saturated)."""
    cache = np.array(cache)
    pages, _, page_size, _ = cache.shape
    for t, slot in enumerate(slots):
        if not 0 <= slot < pages * page_size:
            continue
        row = x[t]
        if scale is not None:
            with np.errstate(all="ignore"):
                f = (row.astype(np.float32) / np.asarray(scale, np.float32)[:, None])
            row = np.where(np.isnan(f), 0x7F, e4m3fn_encode(np.nan_to_num(
                np.clip(f, np.float32(-448), np.float32(448))))).astype(np.uint8)
        cache[slot // page_size, :, slot % page_size] = row
    return cache


def paged_attention(q, k_cache, v_cache, table, lens, scale, window=0, max_len=None,
                    k_scale=None, v_scale=None):
    """q [batch, heads, dim], pools [pages, kv_heads, page_size, dim] (uint8
    codes when the scales are given).  A request without tokens, and a head all
    of whose scores are -infinity, gets zeros.  Returns (out, weight, reach) in fp64:
    weight = sum_t p[t] |v[t]| (the size that errors of p and of the sum act
    on) and reach [batch, heads] = max_t scale * sum_d |q[d] k[t, d]| (the size
    that errors of a score act on)."""
    batch, heads, dim = q.shape
    pages, kv_heads, page_size, _ = k_cache.shape
    group = heads // kv_heads
    out, weight = np.zeros((batch, heads, dim)), np.zeros((batch, heads, dim))
    reach = np.zeros((batch, heads))
    most = table.shape[1] * page_size
    if max_len is not None:
        most = min(most, max_len)
    for b in range(batch):
        n = min(max(int(lens[b]), 0), most)
        seen = [t for t in range(max(0, n - window) if window else 0, n)
                if 0 <= table[b, t // page_size] < pages]
        if not seen:
            continue
        page = np.array([table[b, t // page_size] for t in seen])
        off = np.array([t % page_size for t in seen])
        for h in range(kv_heads):
            k, v = k_cache[page, h, off], v_cache[page, h, off]
            if k_scale is not None:
                k = e4m3fn_decode(k) * float(k_scale[h])
                v = e4m3fn_decode(v) * float(v_scale[h])
            k, v = k.astype(np.float64), v.astype(np.float64)
            for j in range(h * group, (h + 1) * group):
                qj = q[b, j].astype(np.float64)
                s = k @ qj * scale
                if s.max() == -np.inf:      # nothing weighs anything: zeros
                    continue
                p = np.exp(s - s.max())
                p /= p.sum()
                out[b, j] = p @ v
                weight[b, j] = p @ np.abs(v)
                reach[b, j] = np.max(np.abs(k) @ np.abs(qj)) * abs(scale)
    return out, weight, reach
