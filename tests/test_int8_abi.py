"""Host-side refusals of the int8 and expert entry points: the C ABI's status codes
and the binding's argument checks.  Nothing here launches a kernel."""

import ctypes
import os

import pytest
import torch

import bit_quantized_gemm_qgemm_amd as qg

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_ARCH, ERR_FORMAT, ERR_OVERLAP = 0, -1, -2, -3, -4, -6, -9
P = ctypes.c_void_p
BIG = 1 << 31


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(qg.LIB_PATH):
        from bit_quantized_gemm_qgemm_amd import build
        build.build()
    return qg.lib()


def at(i, off=0):
    """An address of its own, never dereferenced."""
    return P((i << 44) + off)


QUANT = dict(dtype=1, x=at(1), codes=at(2), scale=at(3), rows=4, K=64, stride=64)
PREPACK = dict(w=at(1), packed=at(2), experts=3, K=64, N=32, gated=0)
DENSE = dict(dtype=1, a=at(1), a_scale=at(2), packed=at(3), w_scale=at(4), out=at(5), M=4, N=32, K=64, gated=0)
EXPERTS = dict(dtype=2, a=at(1), a_scale=at(2), packed=at(3), w_scale=at(4), offsets=at(5), rows=at(6),
               out=at(7), a_rows=4, M=9, N=32, K=64, experts=3, gated=1)
PLAN = dict(id_bytes=8, ids=at(1), offsets=at(2), rows=at(3), places=at(4), ws=at(5), tokens=5, top=2,
            experts=6)
COMBINE = dict(dtype=1, y=at(1), places=at(2), gates=at(3), out=at(4), rows=9, tokens=5, top=2, N=24)


def call(fn, base, **change):
    assert set(change) <= set(base)
    return fn(*{**base, **change}.values(), P(0))


def refused(base, *changes):
    return [(base, change, status) for change, status in changes]


@pytest.mark.parametrize("name,base,change,status", [
    ("qgemm_quantize_int8", *r) for r in refused(
        QUANT, (dict(dtype=3), ERR_FORMAT), (dict(dtype=0), ERR_FORMAT), (dict(rows=-1), ERR_SHAPE),
        (dict(K=40), ERR_SHAPE), (dict(K=-16), ERR_SHAPE), (dict(K=131072), ERR_SHAPE),
        (dict(rows=BIG), ERR_SHAPE), (dict(stride=-64), ERR_SHAPE), (dict(stride=68), ERR_SHAPE),
        (dict(dtype=4, stride=66), ERR_SHAPE), (dict(stride=1 << 40), ERR_SHAPE),
        (dict(rows=BIG - 1, stride=(1 << 40) - 8), ERR_SHAPE),        # 2^71 elements
        (dict(x=None), ERR_NULL), (dict(codes=None), ERR_NULL), (dict(scale=None), ERR_NULL),
        (dict(x=at(1, 8)), ERR_ALIGN), (dict(codes=at(2, 8)), ERR_ALIGN), (dict(scale=at(3, 2)), ERR_ALIGN),
        (dict(codes=at(1, 256)), ERR_OVERLAP), (dict(scale=at(1, 508)), ERR_OVERLAP),
        (dict(scale=at(2, 252)), ERR_OVERLAP),
        (dict(rows=0, x=None, codes=None, scale=None), OK))] + [
    ("qgemm_prepack_w8a8", *r) for r in refused(
        PREPACK, (dict(experts=0), ERR_SHAPE), (dict(experts=1025), ERR_SHAPE), (dict(K=24), ERR_SHAPE),
        (dict(K=131072), ERR_SHAPE), (dict(N=-1), ERR_SHAPE), (dict(gated=2), ERR_SHAPE),
        (dict(gated=1, N=33), ERR_SHAPE), (dict(K=65536, N=32768), ERR_SHAPE), (dict(w=None), ERR_NULL),
        (dict(packed=None), ERR_NULL), (dict(w=at(1, 4)), ERR_ALIGN), (dict(packed=at(2, 8)), ERR_ALIGN),
        (dict(packed=at(1, 6128)), ERR_OVERLAP), (dict(K=0, w=None, packed=None), OK))] + [
    ("qgemm_w8a8", *r) for r in refused(
        DENSE, (dict(dtype=4), ERR_FORMAT), (dict(dtype=3), ERR_FORMAT), (dict(M=-1), ERR_SHAPE),
        (dict(N=-2), ERR_SHAPE), (dict(K=72), ERR_SHAPE), (dict(K=131072), ERR_SHAPE),
        (dict(gated=1, N=31), ERR_SHAPE), (dict(gated=-1), ERR_SHAPE), (dict(M=BIG), ERR_SHAPE),
        (dict(M=1 << 20, K=2048), ERR_SHAPE), (dict(M=1 << 16, N=1 << 15), ERR_SHAPE),
        (dict(a=None), ERR_NULL), (dict(a_scale=None), ERR_NULL), (dict(packed=None), ERR_NULL),
        (dict(w_scale=None), ERR_NULL), (dict(out=None), ERR_NULL), (dict(a=at(1, 4)), ERR_ALIGN),
        (dict(out=at(5, 8)), ERR_ALIGN), (dict(a_scale=at(2, 2)), ERR_ALIGN), (dict(w_scale=at(4, 1)), ERR_ALIGN),
        (dict(out=at(1, 240)), ERR_OVERLAP), (dict(out=at(4, 112)), ERR_OVERLAP),
        (dict(out=at(3, 4080)), ERR_OVERLAP),
        (dict(M=0, a=None, a_scale=None, out=None), OK), (dict(N=0, packed=None, w_scale=None, out=None), OK))] + [
    ("qgemm_w8a8_experts", *r) for r in refused(
        EXPERTS, (dict(dtype=0), ERR_FORMAT), (dict(experts=0), ERR_SHAPE), (dict(experts=-3), ERR_SHAPE),
        (dict(experts=1025), ERR_SHAPE), (dict(N=33), ERR_SHAPE), (dict(a_rows=-1), ERR_SHAPE),
        (dict(a_rows=BIG // 64), ERR_SHAPE), (dict(rows=None), ERR_SHAPE),      # M is not a_rows
        (dict(offsets=None), ERR_NULL), (dict(a=None), ERR_NULL), (dict(out=None), ERR_NULL),
        (dict(offsets=at(5, 2)), ERR_ALIGN), (dict(rows=at(6, 2)), ERR_ALIGN),
        (dict(out=at(6, 32)), ERR_OVERLAP), (dict(offsets=at(7, 272)), ERR_OVERLAP),
        (dict(w_scale=at(7, 284)), ERR_OVERLAP), (dict(M=0, rows=None, out=None), OK))] + [
    ("qgemm_expert_plan", *r) for r in refused(
        PLAN, (dict(id_bytes=2), ERR_FORMAT), (dict(tokens=-1), ERR_SHAPE), (dict(top=-1), ERR_SHAPE),
        (dict(experts=0), ERR_SHAPE), (dict(experts=1025), ERR_SHAPE), (dict(tokens=1 << 21, top=3), ERR_SHAPE),
        (dict(tokens=BIG - 1, top=BIG - 1), ERR_SHAPE), (dict(ids=None), ERR_NULL),
        (dict(offsets=None), ERR_NULL), (dict(rows=None), ERR_NULL), (dict(places=None), ERR_NULL),
        (dict(tokens=4097, ws=None), ERR_NULL), (dict(ids=at(1, 4)), ERR_ALIGN),
        (dict(offsets=at(2, 2)), ERR_ALIGN), (dict(ws=at(5, 8)), ERR_ALIGN), (dict(rows=at(1, 72)), ERR_OVERLAP),
        (dict(places=at(3, 36)), ERR_OVERLAP), (dict(offsets=at(4, 16)), ERR_OVERLAP),
        (dict(tokens=4097, ws=at(4, 16)), ERR_OVERLAP))] + [
    ("qgemm_expert_combine", *r) for r in refused(
        COMBINE, (dict(dtype=4), ERR_FORMAT), (dict(rows=-1), ERR_SHAPE), (dict(tokens=-1), ERR_SHAPE),
        (dict(top=-1), ERR_SHAPE), (dict(N=-1), ERR_SHAPE), (dict(rows=1 << 16, N=1 << 15), ERR_SHAPE),
        (dict(tokens=1 << 16, N=1 << 15), ERR_SHAPE), (dict(tokens=1 << 16, top=1 << 15), ERR_SHAPE),
        (dict(y=None), ERR_NULL), (dict(places=None), ERR_NULL), (dict(gates=None), ERR_NULL),
        (dict(out=None), ERR_NULL), (dict(y=at(1, 8)), ERR_ALIGN), (dict(out=at(4, 8)), ERR_ALIGN),
        (dict(gates=at(3, 2)), ERR_ALIGN), (dict(out=at(1, 416)), ERR_OVERLAP), (dict(out=at(3, 32)), ERR_OVERLAP),
        (dict(tokens=0, places=None, gates=None, out=None), OK), (dict(N=0, y=None, out=None), OK))])
def test_refusals(lib, name, base, change, status):
    assert call(getattr(lib, name), base, **change) == status


def test_other_architectures_are_refused(lib, monkeypatch):
    monkeypatch.setenv("QGEMM_ARCH_OVERRIDE", "gfx942")
    for name, base in (("qgemm_quantize_int8", QUANT), ("qgemm_prepack_w8a8", PREPACK), ("qgemm_w8a8", DENSE),
                       ("qgemm_w8a8_experts", EXPERTS), ("qgemm_expert_plan", PLAN),
                       ("qgemm_expert_combine", COMBINE)):
        assert call(getattr(lib, name), base) == ERR_ARCH


def test_most_rows(lib, monkeypatch):
    """A launch holds a product's rows in one dimension of its grid."""
    monkeypatch.setenv("QGEMM_ARCH_OVERRIDE", "gfx942")    # what passes the checks ends there
    for M, status in (((1 << 28) - 1, ERR_ARCH), (1 << 28, ERR_SHAPE)):
        assert call(lib.qgemm_w8a8, DENSE, M=M, K=0, N=2) == status
        assert call(lib.qgemm_w8a8_experts, EXPERTS, M=M, N=2) == status


def test_sizes(lib):
    n = lib.qgemm_prepack_w8a8_bytes
    assert n(1, 4096, 11008, 0) == 4096 * 11008
    assert n(3, 144, 33, 0) == 3 * 3 * 2 * 2048            # three column groups, two K tiles
    assert n(1, 128, 34, 1) == 2 * 2 * 2048                # 17 columns twice, each half padded
    assert n(7, 0, 5, 0) == 0 and n(7, 16, 0, 0) == 0
    for bad in ((0, 16, 16, 0), (1, 8, 16, 0), (1, 16, -1, 0), (1, 16, 15, 1), (1, 16, 16, 2), (1, 131072, 16, 0)):
        assert n(*bad) == ERR_SHAPE
    assert n(1, 0, (1 << 24) - 33, 0) == 0 and n(1, 0, (1 << 24) - 32, 0) == ERR_SHAPE
    w = lib.qgemm_expert_plan_workspace_bytes
    assert w(0, 1) == 0 and w(2048, 1024) == 0 and w(2049, 7) == 3 * 7 * 4
    assert w(1 << 22, 1024) == (1 << 22) // 8192 * 1024 * 4
    # a workspace for the most pairs serves fewer
    sizes = [w(n, 7) for n in range(0, (1 << 22) + 1, 1024)] + [w(1 << 22, 7)]
    assert sizes == sorted(sizes)
    for bad in ((-1, 4), ((1 << 22) + 1, 4), (5, 0), (5, 1025)):
        assert w(*bad) == ERR_SHAPE
    with pytest.raises(qg.QgemmError):
        qg.qgemm_prepack_w8a8_bytes(1, 24, 16)
    with pytest.raises(qg.QgemmError):
        qg.qgemm_expert_plan_workspace_bytes(5, 0)


def test_tiles_follow_the_sizes(lib):
    """Few rows take tiles of 16, a full grid the largest ones, whatever is between something between."""
    assert qg.qgemm_w8a8_tile(1, 11008, 4096)[0] == 16
    assert qg.qgemm_w8a8_tile(8192, 8192, 8192) == (256, 256, 1)
    assert qg.qgemm_w8a8_tile(64, 2048, 4096, experts=64)[0] == 16
    assert qg.qgemm_w8a8_tile(65536, 2048, 4096, experts=64) == (128, 256, 1)
    rows = [qg.qgemm_w8a8_tile(M, 8192, 8192)[0] for M in (1, 16, 64, 256, 1024, 4096)]
    assert rows == sorted(rows)
    assert qg.qgemm_w8a8_tile(1, 32, 4096, gated=True)[1] >= 32          # both halves of an output
    for bad in ((-1, 8, 16), (1, 8, 24), (1, 7, 16, 0, True), (1 << 20, 1 << 11, 16), (1, 8, 16, -1)):
        with pytest.raises(qg.QgemmError):
            qg.qgemm_w8a8_tile(*bad)
    assert lib.qgemm_w8a8_tile(1, 8, 16, 0, 0, None, None, None) == ERR_NULL


# ---- the binding ------------------------------------------------------------

class Recorder:
    """Answers the size queries from the library and records every other call."""

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


def i8(*shape):
    return torch.zeros(shape, dtype=torch.int8)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def f16(*shape):
    return torch.zeros(shape, dtype=torch.float16)


def packed(experts, K, N, gated=False):
    return torch.zeros(qg.qgemm_prepack_w8a8_bytes(experts, K, N, gated), dtype=torch.uint8)


def quantize_args():
    return dict(x=f16(4, 64), out=(i8(4, 64), torch.zeros(4)))


def dense_args():
    return dict(a=i8(4, 64), a_scale=torch.zeros(4), w_packed=packed(1, 64, 32), w_scale=torch.zeros(32), N=32,
                gated=False, out=f16(4, 32))


def experts_args():
    return dict(a=i8(4, 64), a_scale=torch.zeros(4), w_packed=packed(3, 64, 32, True),
                w_scale=torch.zeros(3, 32), offsets=i32(4), N=32, rows=i32(9), gated=True, out=f16(9, 16))


def plan_args():
    return dict(ids=torch.zeros((5, 2), dtype=torch.int64), experts=6, out=(i32(7), i32(10), i32(5, 2)),
                workspace=torch.zeros(16, dtype=torch.uint8))


def combine_args():
    return dict(y=f16(9, 24), places=i32(5, 2), gates=torch.zeros(5, 2), out=f16(5, 24))


CALLS = {qg.qgemm_quantize_int8: quantize_args, qg.qgemm_w8a8: dense_args, qg.qgemm_w8a8_experts: experts_args,
         qg.qgemm_expert_plan: plan_args, qg.qgemm_expert_combine: combine_args}


@pytest.mark.parametrize("fn", CALLS)
def test_the_plain_call_is_made(fake, fn):
    fn(**CALLS[fn]())
    assert [name for name, _ in fake.calls] == [fn.__name__]


@pytest.mark.parametrize("fn,change,error", [
    (qg.qgemm_quantize_int8, dict(x=torch.zeros(4, 64).double()), TypeError),
    (qg.qgemm_quantize_int8, dict(x=f16(4, 128)[:, ::2]), ValueError),
    (qg.qgemm_quantize_int8, dict(x=f16(64)), ValueError),
    (qg.qgemm_quantize_int8, dict(out=(i8(4, 64),)), ValueError),
    (qg.qgemm_quantize_int8, dict(out=(i8(4, 48), torch.zeros(4))), ValueError),
    (qg.qgemm_quantize_int8, dict(out=(i8(4, 64), torch.zeros(5))), ValueError),
    (qg.qgemm_quantize_int8, dict(out=(torch.zeros(4, 64), torch.zeros(4))), TypeError),
    (qg.qgemm_quantize_int8, dict(out=(i8(4, 128)[:, :64], torch.zeros(4))), ValueError),
    (qg.qgemm_w8a8, dict(a=f16(4, 64)), TypeError), (qg.qgemm_w8a8, dict(a=i8(4, 128)[:, :64]), ValueError),
    (qg.qgemm_w8a8, dict(a=None), TypeError), (qg.qgemm_w8a8, dict(a_scale=torch.zeros(5)), ValueError),
    (qg.qgemm_w8a8, dict(a_scale=f16(4)), TypeError), (qg.qgemm_w8a8, dict(w_scale=torch.zeros(31)), ValueError),
    (qg.qgemm_w8a8, dict(w_packed=torch.zeros(16, dtype=torch.uint8)), ValueError),
    (qg.qgemm_w8a8, dict(w_packed=i8(4096)), TypeError), (qg.qgemm_w8a8, dict(out=f16(4, 16)), ValueError),
    (qg.qgemm_w8a8, dict(out=torch.zeros(4, 32)), TypeError), (qg.qgemm_w8a8, dict(N=48), ValueError),
    (qg.qgemm_w8a8, dict(out=None, dtype=torch.float32), TypeError),
    (qg.qgemm_w8a8, dict(a=i8(4, 40)), qg.QgemmError),
    (qg.qgemm_w8a8_experts, dict(offsets=None), TypeError),
    (qg.qgemm_w8a8_experts, dict(offsets=torch.zeros(4, dtype=torch.int64)), TypeError),
    (qg.qgemm_w8a8_experts, dict(offsets=i32(3)), ValueError),       # two experts
    (qg.qgemm_w8a8_experts, dict(offsets=i32(1)), qg.QgemmError),    # none
    (qg.qgemm_w8a8_experts, dict(w_scale=torch.zeros(32)), ValueError),
    (qg.qgemm_w8a8_experts, dict(rows=torch.zeros(9, dtype=torch.int64)), TypeError),
    (qg.qgemm_w8a8_experts, dict(rows=None), ValueError),            # out has nine rows, a four
    (qg.qgemm_w8a8_experts, dict(gated=False), ValueError),
    (qg.qgemm_w8a8_experts, dict(out=f16(9, 32)), ValueError),
    (qg.qgemm_expert_plan, dict(ids=i32(5, 2).float()), TypeError),
    (qg.qgemm_expert_plan, dict(ids=i32(10)), ValueError),
    (qg.qgemm_expert_plan, dict(ids=i32(5, 4)[:, ::2]), ValueError),
    (qg.qgemm_expert_plan, dict(experts=0), qg.QgemmError),
    (qg.qgemm_expert_plan, dict(out=(i32(7), i32(10))), ValueError),
    (qg.qgemm_expert_plan, dict(out=(i32(6), i32(10), i32(5, 2))), ValueError),
    (qg.qgemm_expert_plan, dict(out=(i32(7), i32(10), i32(2, 5))), ValueError),
    (qg.qgemm_expert_plan, dict(workspace=i32(16)), TypeError),
    (qg.qgemm_expert_plan, dict(ids=torch.zeros((5000, 2), dtype=torch.int64),
                                out=(i32(7), i32(10000), i32(5000, 2))), ValueError),    # short workspace
    (qg.qgemm_expert_combine, dict(y=torch.zeros(9, 24)), TypeError),
    (qg.qgemm_expert_combine, dict(y=f16(9, 48)[:, :24]), ValueError),
    (qg.qgemm_expert_combine, dict(places=torch.zeros((5, 2), dtype=torch.int64)), TypeError),
    (qg.qgemm_expert_combine, dict(gates=torch.zeros(5, 3)), ValueError),
    (qg.qgemm_expert_combine, dict(gates=f16(5, 2)), TypeError),
    (qg.qgemm_expert_combine, dict(out=f16(9, 24)), ValueError),
])
def test_binding_refusals(fake, fn, change, error):
    with pytest.raises(error):
        fn(**{**CALLS[fn](), **change})
    assert not fake.calls


@pytest.mark.parametrize("w,error", [(f16(64, 32), TypeError), (i8(64), ValueError), (i8(2, 3, 64, 32), ValueError),
                                     (i8(64, 64)[:, :32], ValueError), (i8(24, 32), qg.QgemmError), (3, TypeError)])
def test_prepack_refusals(fake, w, error):
    with pytest.raises(error):
        qg.qgemm_prepack_w8a8(w)
    assert not fake.calls


def test_arguments_reach_the_library(fake):
    qg.qgemm_quantize_int8(torch.zeros(4, 96)[:, :64])
    assert fake.calls[-1][1][0] == 4 and fake.calls[-1][1][4:7] == (4, 64, 96)
    args = experts_args()
    qg.qgemm_w8a8_experts(**{**args, "out": None, "dtype": torch.bfloat16})
    name, sent = fake.calls[-1]
    assert sent[0] == 2 and sent[6] == args["rows"].data_ptr() and sent[8:14] == (4, 9, 32, 64, 3, 1)
    qg.qgemm_w8a8_experts(**{**args, "rows": None, "out": f16(4, 16)})
    assert fake.calls[-1][1][0] == 1 and fake.calls[-1][1][6] is None and fake.calls[-1][1][8:10] == (4, 4)
    qg.qgemm_expert_plan(i32(5, 2), 6)
    assert fake.calls[-1][1][0] == 4 and fake.calls[-1][1][6:9] == (5, 2, 6)
