"""The native half of the binding: what it takes, what it leaves to the checks
in Python, and that both make the same call."""

import os

import pytest
import torch

import bit_quantized_gemm_qgemm_amd as qg


@pytest.fixture(scope="module")
def native():
    if not (os.path.exists(qg.LIB_PATH) and qg.LIB_PATH.endswith("libqgemm.so")):
        from bit_quantized_gemm_qgemm_amd import build
        build.build()
    qg.lib()
    return qg._native


def arguments(device):
    """Plain arguments of the three calls, in the native functions' order."""
    i32 = {"dtype": torch.int32, "device": device}
    table = torch.tensor([[2, -1], [0, 1], [-1, -1]], **i32)
    plan = [table, torch.tensor([5, 20, 0], **i32), torch.tensor([14, 1, 7], **i32),
            torch.tensor([4, 3, 5], **i32), 16, 22,
            (torch.zeros(3, **i32), torch.zeros(4, **i32), torch.zeros(4, **i32),
             torch.zeros(22, dtype=torch.int64, device=device))]
    g = torch.Generator().manual_seed(1)
    fused = torch.randn((22, 12 * 64), generator=g).half().to(device)
    q, k, v = fused.split([512, 128, 128], dim=1)
    pools = torch.randn((6, 2, 16, 2, 64), generator=g).half().to(device)
    pools = [pools[:, j].transpose(1, 2) for j in (0, 1)]
    slots = torch.arange(22, device=device) + 30
    append = [k.unflatten(1, (2, 64)), v.unflatten(1, (2, 64)), slots, *pools, None, None]
    out = torch.zeros((3, 8, 64), dtype=torch.float16, device=device)
    ws = torch.zeros(4096, dtype=torch.uint8, device=device)
    full = torch.tensor([[2, 4], [0, 1], [3, 5]], **i32)
    attend = [q[:3].unflatten(1, (8, 64)), *pools, full, torch.tensor([19, 21, 7], **i32), None, None,
              0, 32, None, out, ws]
    return plan, append, attend


def changed(args, at, value):
    return [value if i == at else a for i, a in enumerate(args)]


def test_host_tensors_and_odd_arguments_are_left_to_python(native):
    plan, append, attend = arguments("cpu")
    for fn, args in ((native.kv_plan, plan), (native.kv_append, append),
                     (native.paged_attention, attend)):
        assert fn(*args) is None
        assert fn() is None and fn(*args[:-1]) is None and fn(*args, 1) is None
        for i in range(len(args)):
            for other in (None, 3, "x", 1.5, 2 ** 80, (), torch.zeros(()), torch.zeros(2, 3, 4, 5)):
                assert fn(*changed(args, i, other)) is None


@pytest.mark.gpu
def test_plain_calls_are_taken_and_agree_with_the_checked_ones(native, monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    print("case native binding", flush=True)

    def run():
        plan, append, attend = arguments("cuda")
        lens, cu_tokens, cu_pages, slots = qg.qgemm_kv_plan(*plan[:-1], out=plan[-1])
        qg.qgemm_kv_append(*append)
        names = ("q", "k_cache", "v_cache", "table", "lens", "k_scale", "v_scale", "window",
                 "max_len", "scale", "out", "workspace")
        out = qg.qgemm_paged_attention(**dict(zip(names, attend)))
        assert out is attend[-2]
        windowed = qg.qgemm_paged_attention(**dict(zip(names, attend), window=5, scale=0.25, out=None))
        torch.cuda.synchronize()
        return plan[0], lens, cu_tokens, cu_pages, slots, *append[3:5], out, windowed

    with monkeypatch.context() as m:
        m.setattr(qg, "_native", None)
        checked = run()
    fast = run()
    for a, b in zip(checked, fast):
        assert torch.equal(a, b)
    plan, append, attend = arguments("cuda")
    assert native.kv_plan(*plan) == native.kv_append(*append) == native.paged_attention(*attend) == 0
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_device_tensors_that_do_not_fit_are_not_taken(native):
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    print("case native refusals", flush=True)
    plan, append, attend = arguments("cuda")
    x = torch.zeros
    cuda = {"device": "cuda"}
    for fn, args, at, value in (
            (native.kv_plan, plan, 0, plan[0].t()), (native.kv_plan, plan, 1, plan[1].long()),
            (native.kv_plan, plan, 1, plan[1][:2]), (native.kv_plan, plan, 4, 0),
            (native.kv_plan, plan, 5, 21), (native.kv_plan, plan, 5, -1),
            (native.kv_plan, plan, 6, plan[6][:3]), (native.kv_plan, plan, 2, plan[2].cpu()),
            (native.kv_append, append, 0, append[0].float()), (native.kv_append, append, 0, append[0][:20]),
            (native.kv_append, append, 1, append[1].bfloat16()),
            (native.kv_append, append, 2, append[2].int()),
            (native.kv_append, append, 2, x(44, dtype=torch.int64, **cuda)[::2]),
            (native.kv_append, append, 4, append[4].contiguous()),
            (native.kv_append, append, 5, x(2, **cuda)),
            (native.kv_append, append, 3, append[3].to(torch.float8_e4m3fn)),
            (native.paged_attention, attend, 0, attend[0][..., :32]),
            (native.paged_attention, attend, 0, attend[0][:, :7]),
            (native.paged_attention, attend, 3, attend[3][:2]),
            (native.paged_attention, attend, 4, attend[4].long()),
            (native.paged_attention, attend, 7, -1), (native.paged_attention, attend, 8, None),
            (native.paged_attention, attend, 8, -1), (native.paged_attention, attend, 9, 1),
            (native.paged_attention, attend, 10, None),
            (native.paged_attention, attend, 10, attend[10].transpose(0, 1)),
            (native.paged_attention, attend, 10, attend[10].bfloat16()),
            (native.paged_attention, attend, 11, None),
            # contexts past one workgroup's: a workspace that is too small
            (native.paged_attention, attend, 8, 100000)):
        assert fn(*changed(args, at, value)) is None, (at, value)
