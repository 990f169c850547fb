"""The native half of the binding of the int8 and expert calls: what it takes, what it
leaves to the checks in Python, and that both make the same call."""

import os

import pytest
import torch

import bit_quantized_gemm_qgemm_amd as qg


@pytest.fixture(scope="module")
def native():
    if not os.path.exists(qg.LIB_PATH):
        from bit_quantized_gemm_qgemm_amd import build
        build.build()
    qg.lib()
    return qg._native


def arguments(device):
    """Plain arguments of the five calls, in the native functions' order."""
    g = torch.Generator().manual_seed(2)

    def codes(*shape):
        return torch.randint(-128, 128, shape, generator=g, dtype=torch.int8).to(device)

    def scales(*shape):
        return (torch.rand(shape, generator=g) / 500).to(device)

    i32 = {"dtype": torch.int32, "device": device}
    quantize = [torch.randn((6, 160), generator=g).to(device)[:, :64],
                (torch.zeros((6, 64), dtype=torch.int8, device=device), torch.zeros(6, device=device))]
    packed = torch.randint(0, 256, (qg.qgemm_prepack_w8a8_bytes(3, 64, 34, True),), generator=g,
                           dtype=torch.uint8).to(device)
    dense = [codes(6, 64), scales(6), packed, scales(34), 34, False,
             torch.zeros((6, 34), dtype=torch.bfloat16, device=device)]
    experts = [codes(6, 64), scales(6), packed, scales(3, 34), torch.tensor([0, 4, 4, 9], **i32), 34,
               torch.tensor([5, 0, 1, 3, 5, 5, 2, 4, 0], **i32), True,
               torch.zeros((9, 17), dtype=torch.float16, device=device)]
    plan = [torch.randint(0, 7, (9, 3), generator=g).to(device), 6,
            (torch.zeros(7, **i32), torch.zeros(27, **i32), torch.zeros((9, 3), **i32)),
            torch.zeros(16, dtype=torch.uint8, device=device)]
    combine = [torch.randn((9, 24), generator=g).half().to(device), torch.tensor([[3, -1], [8, 0]], **i32),
               scales(2, 2), torch.zeros((2, 24), dtype=torch.float16, device=device)]
    return {"quantize_int8": quantize, "w8a8": dense, "w8a8_experts": experts, "expert_plan": plan,
            "expert_combine": combine}


def changed(args, at, value):
    return [value if i == at else a for i, a in enumerate(args)]


def test_host_tensors_and_odd_arguments_are_left_to_python(native):
    for name, args in arguments("cpu").items():
        fn = getattr(native, name)
        assert fn(*args) is None
        assert fn() is None and fn(*args[:-1]) is None and fn(*args, 1) is None
        for i in range(len(args)):
            for other in (None, 3, "x", 1.5, 2 ** 80, (), torch.zeros(()), torch.zeros(2, 3, 4, 5)):
                assert fn(*changed(args, i, other)) is None


def outputs(args):
    return [t for a in args for t in (a if isinstance(a, tuple) else (a,)) if isinstance(t, torch.Tensor)]


@pytest.mark.gpu
def test_plain_calls_are_taken_and_agree_with_the_checked_ones(native, monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    calls = {
        "quantize_int8": lambda x, out: qg.qgemm_quantize_int8(x, out=out),
        "w8a8": lambda a, s, w, ws, N, gated, out: qg.qgemm_w8a8(a, s, w, ws, N, gated=gated, out=out),
        "w8a8_experts": lambda a, s, w, ws, o, N, rows, gated, out: qg.qgemm_w8a8_experts(
            a, s, w, ws, o, N, rows=rows, gated=gated, out=out),
        "expert_plan": lambda ids, experts, out, ws: qg.qgemm_expert_plan(ids, experts, out=out, workspace=ws),
        "expert_combine": lambda y, places, gates, out: qg.qgemm_expert_combine(y, places, gates, out=out),
    }
    for name, args in arguments("cuda").items():
        print("case native", name, flush=True)
        assert getattr(native, name)(*args) == 0
        torch.cuda.synchronize()
        taken = [t.clone() for t in outputs(args)]
        again = arguments("cuda")[name]
        with monkeypatch.context() as m:
            m.setattr(qg, "_native", None)
            calls[name](*again)
        torch.cuda.synchronize()
        for a, b in zip(taken, outputs(again)):
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
        # the public call goes the native way and returns the tensors given
        third = arguments("cuda")[name]
        got = calls[name](*third)
        assert got is (third[2] if name == "expert_plan" else third[-1])


@pytest.mark.gpu
def test_what_is_not_plain_is_refused_or_made_in_python(native):
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    args = arguments("cuda")
    wrong = {
        "quantize_int8": [(0, args["quantize_int8"][0].double()), (0, args["quantize_int8"][0].t())],
        "w8a8": [(0, args["w8a8"][0][:, :48]), (1, args["w8a8"][1][:5]), (2, args["w8a8"][2][:64]),
                 (3, args["w8a8"][3][:33]), (4, 33), (5, 1), (6, args["w8a8"][6].float())],
        "w8a8_experts": [(3, args["w8a8_experts"][3][:2]), (4, args["w8a8_experts"][4].long()),
                         (6, args["w8a8_experts"][6].long()), (7, False), (8, args["w8a8_experts"][8][:8])],
        "expert_plan": [(0, args["expert_plan"][0].float()), (1, 7), (3, args["expert_plan"][3].view(torch.int32))],
        "expert_combine": [(1, args["expert_combine"][1].long()), (2, args["expert_combine"][2][:1]),
                           (3, args["expert_combine"][3].float())],
    }
    for name, changes in wrong.items():
        for i, value in changes:
            print("case native refused", name, i, flush=True)
            assert getattr(native, name)(*changed(args[name], i, value)) is None
    # rows left out: the rows of a as they lie
    plain = args["w8a8_experts"]
    out = torch.zeros((6, 17), dtype=torch.float16, device="cuda")
    assert native.w8a8_experts(*changed(changed(plain, 6, None), 8, out)) == 0
    # the status of a refused call comes back
    x = torch.zeros((4, 40), device="cuda")
    out = (torch.zeros((4, 40), dtype=torch.int8, device="cuda"), torch.zeros(4, device="cuda"))
    assert native.quantize_int8(x, out) == -2
    with pytest.raises(qg.QgemmError):
        qg.qgemm_quantize_int8(x, out=out)
