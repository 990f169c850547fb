"""Host-side refusals of the key-value cache entry points: the C ABI's status
codes and the binding's argument checks.  Nothing here launches a kernel."""

import ctypes
import os

import pytest
import torch

import bit_quantized_gemm_qgemm_amd as qg

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_ARCH, ERR_FORMAT = 0, -1, -2, -3, -4, -6
P = ctypes.c_void_p
GOOD, TWO, FOUR, EIGHT = P(0x10000), P(0x10002), P(0x10004), P(0x10008)   # never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(qg.LIB_PATH):
        from bit_quantized_gemm_qgemm_amd import build
        build.build()
    return qg.lib()


PLAN = dict(table=GOOD, cached=GOOD, added=GOOD, free=GOOD, lens=GOOD, cu_tokens=GOOD,
            cu_pages=GOOD, slots=GOOD, batch=4, width=8, table_stride=8, num_free=9, page_size=16,
            tokens=4)
APPEND = dict(dtype=1, cache_dtype=1, k=GOOD, v=GOOD, slots=GOOD, k_cache=GOOD, v_cache=GOOD,
              k_scale=None, v_scale=None, tokens=4, kv_heads=2, dim=64, k_token=128, k_head=64,
              v_token=128, v_head=64, pages=5, page_size=16, page_stride=2048, head_stride=1024,
              token_stride=64)
ATTEND = dict(dtype=1, cache_dtype=1, q=GOOD, k_cache=GOOD, v_cache=GOOD, table=GOOD, lens=GOOD,
              k_scale=None, v_scale=None, out=GOOD, workspace=GOOD, batch=3, heads=8, kv_heads=2,
              dim=64, q_batch=512, q_head=64, pages=5, page_size=16, page_stride=2048,
              head_stride=1024, token_stride=64, width=8, table_stride=8, max_len=128, window=0,
              scale=0.125)
BIG = 1 << 31


def call(fn, base, **change):
    assert set(change) <= set(base)
    return fn(*{**base, **change}.values(), P(0))


@pytest.mark.parametrize("change,status", [
    (dict(batch=-1), ERR_SHAPE), (dict(width=-1), ERR_SHAPE), (dict(page_size=0), ERR_SHAPE),
    (dict(tokens=-1), ERR_SHAPE), (dict(tokens=BIG), ERR_SHAPE), (dict(num_free=-1), ERR_SHAPE),
    (dict(table_stride=7), ERR_SHAPE), (dict(batch=BIG), ERR_SHAPE),
    (dict(table=None), ERR_NULL), (dict(cached=None), ERR_NULL), (dict(added=None), ERR_NULL),
    (dict(free=None), ERR_NULL), (dict(lens=None), ERR_NULL), (dict(cu_tokens=None), ERR_NULL),
    (dict(cu_pages=None, batch=0), ERR_NULL), (dict(slots=None), ERR_NULL),
    (dict(table=TWO), ERR_ALIGN), (dict(slots=FOUR), ERR_ALIGN),
])
def test_plan_refusals(lib, change, status):
    assert call(lib.qgemm_kv_plan, PLAN, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(dtype=3, cache_dtype=3), ERR_FORMAT), (dict(dtype=0), ERR_FORMAT),
    (dict(cache_dtype=2), ERR_FORMAT), (dict(k_scale=GOOD), ERR_FORMAT),
    (dict(cache_dtype=3), ERR_NULL), (dict(cache_dtype=3, k_scale=GOOD), ERR_NULL),
    (dict(cache_dtype=3, k_scale=TWO, v_scale=GOOD), ERR_ALIGN),
    (dict(dim=72), ERR_SHAPE), (dict(dim=0), ERR_SHAPE), (dict(dim=272), ERR_SHAPE),
    (dict(tokens=-1), ERR_SHAPE), (dict(pages=-1), ERR_SHAPE), (dict(page_size=0), ERR_SHAPE),
    (dict(k_token=132), ERR_SHAPE), (dict(v_head=-64), ERR_SHAPE),
    (dict(page_stride=2040), ERR_SHAPE), (dict(head_stride=-64), ERR_SHAPE),
    (dict(pages=BIG - 1), ERR_SHAPE),             # 2^36 rows
    (dict(k=None), ERR_NULL), (dict(slots=None), ERR_NULL), (dict(v_cache=None), ERR_NULL),
    (dict(v=EIGHT), ERR_ALIGN), (dict(k_cache=EIGHT), ERR_ALIGN), (dict(slots=FOUR), ERR_ALIGN),
    (dict(tokens=0, k=None, v=None, slots=None), OK), (dict(pages=0, k_cache=None), OK),
])
def test_append_refusals(lib, change, status):
    assert call(lib.qgemm_kv_append, APPEND, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(dtype=3), ERR_FORMAT), (dict(cache_dtype=2), ERR_FORMAT), (dict(v_scale=GOOD), ERR_FORMAT),
    (dict(cache_dtype=3, v_scale=GOOD), ERR_NULL),
    (dict(heads=9), ERR_SHAPE), (dict(kv_heads=0), ERR_SHAPE), (dict(batch=-1), ERR_SHAPE),
    (dict(dim=24), ERR_SHAPE), (dict(dim=512), ERR_SHAPE), (dict(max_len=-1), ERR_SHAPE),
    (dict(window=-1), ERR_SHAPE), (dict(width=-1), ERR_SHAPE), (dict(table_stride=7), ERR_SHAPE),
    (dict(q_head=68), ERR_SHAPE), (dict(q_batch=-8), ERR_SHAPE), (dict(token_stride=72), ERR_SHAPE),
    (dict(pages=1 << 28), ERR_SHAPE), (dict(max_len=BIG), ERR_SHAPE),
    (dict(q=None), ERR_NULL), (dict(table=None), ERR_NULL), (dict(lens=None), ERR_NULL),
    (dict(out=None), ERR_NULL), (dict(k_cache=None), ERR_NULL),
    (dict(q=EIGHT), ERR_ALIGN), (dict(out=EIGHT), ERR_ALIGN), (dict(v_cache=EIGHT), ERR_ALIGN),
    (dict(workspace=EIGHT), ERR_ALIGN), (dict(lens=TWO), ERR_ALIGN),
    (dict(batch=0, q=None, out=None, lens=None, table=None), OK), (dict(heads=0), OK),
])
def test_attention_refusals(lib, change, status):
    assert call(lib.qgemm_paged_attention, ATTEND, **change) == status


def test_workspace_size(lib):
    fn = lib.qgemm_paged_attention_workspace_bytes
    assert fn(3, 8, 2, 64, 128, 0) >= 0
    for bad in ((-1, 8, 2, 64, 128, 0), (3, 9, 2, 64, 128, 0), (3, 8, 0, 64, 128, 0),
                (3, 8, 2, 40, 128, 0), (3, 8, 2, 64, -1, 0), (3, 8, 2, 64, 128, -1),
                (1 << 20, 1 << 12, 2, 64, 128, 0)):
        assert fn(*bad) == ERR_SHAPE
    with pytest.raises(qg.QgemmError):
        qg.qgemm_paged_attention_workspace_bytes(3, 9, 2, 64, 128)


def test_other_architectures_are_refused(lib, monkeypatch):
    monkeypatch.setenv("QGEMM_ARCH_OVERRIDE", "gfx942")
    for fn, base in ((lib.qgemm_kv_plan, PLAN), (lib.qgemm_kv_append, APPEND),
                     (lib.qgemm_paged_attention, ATTEND)):
        assert call(fn, base) == ERR_ARCH


# ---- the binding ------------------------------------------------------------

class Recorder:
    """Answers the size query from the library and records every other call."""

    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name.endswith("_bytes") or name == "qgemm_status_string":
            return getattr(self.real, name)
        return lambda *args: self.calls.append((name, args)) or 0


@pytest.fixture
def fake(lib, monkeypatch):
    rec = Recorder(lib)
    monkeypatch.setattr(qg, "lib", lambda: rec)
    monkeypatch.setattr(qg, "_stream", lambda t: None)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda self: True), raising=False)
    return rec


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def f16(*shape, dtype=torch.float16):
    return torch.zeros(shape, dtype=dtype)


def plan_args():
    return dict(table=i32(4, 8), cached=i32(4), added=i32(4), free_pages=i32(9), page_size=16,
                tokens=4, out=(i32(4), i32(5), i32(5), torch.zeros(4, dtype=torch.int64)))


def append_args():
    return dict(k=f16(4, 2, 64), v=f16(4, 2, 64), slots=torch.zeros(4, dtype=torch.int64),
                k_cache=f16(5, 2, 16, 64), v_cache=f16(5, 2, 16, 64), k_scale=None, v_scale=None)


def attend_args():
    return dict(q=f16(3, 8, 64), k_cache=f16(5, 2, 16, 64), v_cache=f16(5, 2, 16, 64),
                table=i32(3, 8), lens=i32(3), k_scale=None, v_scale=None, window=0, max_len=100,
                out=f16(3, 8, 64),
                workspace=torch.zeros(max(16, qg.qgemm_paged_attention_workspace_bytes(
                    3, 8, 2, 64, 100)), dtype=torch.uint8))


CODES = torch.zeros((5, 2, 16, 64), dtype=torch.uint8)
HEADS = torch.ones(2)


@pytest.mark.parametrize("change,error", [
    (dict(table=i32(4, 16)[:, ::2]), ValueError), (dict(table=torch.zeros(4, 8)), TypeError),
    (dict(cached=i32(3)), ValueError), (dict(added=i32(8)[::2]), ValueError),
    (dict(free_pages=torch.zeros(9, dtype=torch.int64)), TypeError),
    (dict(page_size=0), ValueError), (dict(tokens=-1), ValueError), (dict(tokens=5), ValueError),
    (dict(out=(i32(4), i32(4), i32(5), torch.zeros(4, dtype=torch.int64))), ValueError),
    (dict(out=(i32(4), i32(5), i32(5), i32(4))), TypeError), (dict(out=(i32(4),)), ValueError),
])
def test_plan_binding_refusals(fake, change, error):
    with pytest.raises(error):
        qg.qgemm_kv_plan(**{**plan_args(), **change})
    assert not fake.calls


@pytest.mark.parametrize("change,error", [
    (dict(k=f16(4, 2, 128)[:, :, ::2]), ValueError), (dict(k=f16(4, 3, 64)), ValueError),
    (dict(v=f16(4, 2, 64, dtype=torch.bfloat16)), TypeError), (dict(v=f16(3, 2, 64)), ValueError),
    (dict(slots=i32(4)), TypeError), (dict(k_cache=f16(5, 2, 16, 80)), ValueError),
    (dict(v_cache=f16(5, 16, 2, 64).transpose(1, 2)), ValueError),      # other strides than k_cache
    (dict(k_cache=CODES, v_cache=CODES), ValueError),                   # no scales
    (dict(k_cache=CODES, v_cache=CODES, k_scale=HEADS, v_scale=torch.ones(3)), ValueError),
    (dict(k_cache=CODES, v_cache=CODES, k_scale=HEADS, v_scale=HEADS.double()), TypeError),
    (dict(k_scale=HEADS), ValueError),
    (dict(k=f16(4, 2, 64, dtype=torch.bfloat16), v=f16(4, 2, 64, dtype=torch.bfloat16)), TypeError),
])
def test_append_binding_refusals(fake, change, error):
    with pytest.raises(error):
        qg.qgemm_kv_append(**{**append_args(), **change})
    assert not fake.calls


@pytest.mark.parametrize("change,error", [
    (dict(q=f16(3, 9, 64)), ValueError), (dict(q=f16(3, 8, 32)), ValueError),
    (dict(q=f16(3, 8, 64).float()), TypeError), (dict(q=f16(8, 64)), ValueError),
    (dict(table=i32(2, 8)), ValueError), (dict(lens=i32(4)), ValueError),
    (dict(lens=torch.zeros(3, dtype=torch.int64)), TypeError),
    (dict(out=f16(3, 8, 128)[:, :, ::2]), ValueError), (dict(out=f16(3, 4, 64)), ValueError),
    (dict(out=f16(3, 8, 64, dtype=torch.bfloat16)), TypeError),
    (dict(k_cache=CODES, v_cache=CODES, k_scale=HEADS), ValueError),
    (dict(max_len=-1), qg.QgemmError), (dict(window=-1), qg.QgemmError),
    (dict(workspace=i32(16)), TypeError),
])
def test_attention_binding_refusals(fake, change, error):
    with pytest.raises(error):
        qg.qgemm_paged_attention(**{**attend_args(), **change})
    assert not fake.calls


def test_attention_refuses_a_short_workspace(fake, monkeypatch):
    args = attend_args()
    monkeypatch.setattr(qg, "qgemm_paged_attention_workspace_bytes", lambda *a: 4096)
    with pytest.raises(ValueError, match="4096"):
        qg.qgemm_paged_attention(**{**args, "workspace": torch.zeros(4095, dtype=torch.uint8)})
    assert not fake.calls


def test_binding_passes_views_by_their_strides(fake):
    fused = f16(4, (8 + 2 + 2) * 64)
    q, k, v = fused.split([512, 128, 128], dim=1)
    pools = f16(5, 2, 16, 2, 64)                       # [pages, k or v, page_size, kv_heads, dim]
    kc, vc = pools[:, 0].transpose(1, 2), pools[:, 1].transpose(1, 2)
    qg.qgemm_kv_append(k.unflatten(1, (2, 64)), v.unflatten(1, (2, 64)),
                       torch.zeros(4, dtype=torch.int64), kc, vc)
    name, args = fake.calls[-1]
    assert name == "qgemm_kv_append"
    #                     tokens heads dim  k strides  v strides  pages page  pool strides
    assert args[9:21] == (4, 2, 64, 768, 64, 768, 64, 5, 16, 4096, 64, 128)
    qg.qgemm_paged_attention(q.unflatten(1, (8, 64)), kc, vc, i32(4, 9)[:, :8], i32(4))
    name, args = fake.calls[-1]
    assert name == "qgemm_paged_attention"
    assert args[11:26] == (4, 8, 2, 64, 768, 64, 5, 16, 4096, 64, 128, 8, 9, 128, 0)
    # an axis of one entry: its stride is whatever torch left there, and is not used
    qg.qgemm_paged_attention(f16(1, 8, 64).as_strided((1, 8, 64), (3, 64, 1)), kc, vc, i32(1, 8),
                             i32(1))
    assert fake.calls[-1][1][15:17] == (0, 64)
