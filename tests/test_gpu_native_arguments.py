"""The native half of the binding on device tensors, every argument right but
one: nothing is taken and nothing raised, so each check of it is reached."""

import pytest
import torch

import bit_quantized_gemm_qgemm_amd as qg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def native():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    qg.lib()
    assert qg._native is not None
    return qg._native


def arguments(e4m3=False):
    i32 = {"dtype": torch.int32, "device": "cuda"}
    plan = [torch.tensor([[2, -1], [0, 1], [-1, -1]], **i32), torch.tensor([5, 20, 0], **i32),
            torch.tensor([14, 1, 7], **i32), torch.tensor([4, 3, 5], **i32), 16, 22,
            (torch.zeros(3, **i32), torch.zeros(4, **i32), torch.zeros(4, **i32),
             torch.zeros(22, dtype=torch.int64, device="cuda"))]
    pools = [torch.zeros((6, 2, 16, 64), dtype=torch.uint8 if e4m3 else torch.float16, device="cuda")
             for _ in "kv"]
    scales = [torch.ones(2, device="cuda") if e4m3 else None for _ in "kv"]
    x = torch.zeros((22, 4, 64), dtype=torch.float16, device="cuda")
    append = [x[:, :2], x[:, 2:], torch.arange(22, device="cuda"), *pools, *scales]
    attend = [x[:3], *pools, torch.tensor([[2, 4], [0, 1], [3, 5]], **i32),
              torch.tensor([19, 21, 7], **i32), *scales, 0, 32, None,
              torch.zeros((3, 4, 64), dtype=torch.float16, device="cuda"),
              torch.zeros(4096, dtype=torch.uint8, device="cuda")]
    return plan, append, attend


# what of the odd values below is right for which argument
TAKEN = {("kv_plan", 4): (3,), ("paged_attention", 7): (3,), ("paged_attention", 8): (3,),
         ("paged_attention", 9): (None, 1.5)}


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("name,at", [("kv_plan", 0), ("kv_append", 1), ("paged_attention", 2)])
def test_each_argument_in_turn(native, name, at, e4m3):
    print("case native arguments", name, e4m3, flush=True)
    fn, args = getattr(native, name), arguments(e4m3)[at]
    assert fn(*args) == 0
    assert fn(*args[:-1]) is None and fn(*args, 1) is None
    tensors = [torch.zeros((), device="cuda"), torch.zeros((2, 3, 4, 5), device="cuda"),
               torch.zeros(7, device="cuda"), torch.zeros((3, 4, 64), device="cuda")[:, :, ::2],
               torch.zeros((9, 9), dtype=torch.int32, device="cuda").t(), torch.zeros(3),
               torch.zeros((3, 3, 3)).to_sparse()]
    for i, right in enumerate(args):
        for odd in [None, 3, -3, "x", 1.5, float("nan"), True, 2 ** 80, -2 ** 80, (), (1, 2, 3, 4), [],
                    torch.float16, *tensors]:
            if odd is right or any(odd is t for t in TAKEN.get((name, i), ())):
                continue
            if (name, i) == ("paged_attention", 9) and isinstance(odd, float):
                continue                     # any float is a scale
            assert fn(*[odd if j == i else a for j, a in enumerate(args)]) is None, (i, odd)
        if isinstance(right, torch.Tensor):
            for odd in (right.cpu(), right.double(), right[None], right.to(torch.bool)):
                assert fn(*[odd if j == i else a for j, a in enumerate(args)]) is None, (i, odd)
            if right.dim() and right.numel():
                longer = torch.cat([right, right[:1]])
                if (name, i) not in (("kv_plan", 3), ("paged_attention", 11)):   # of any length
                    assert fn(*[longer if j == i else a for j, a in enumerate(args)]) is None, i
    # each output of a plan
    if name == "kv_plan":
        for j, t in enumerate(args[6]):
            for odd in (None, 3, t.cpu(), t.float(), t[:-1], t[None], torch.stack([t, t], 1)[:, 0]):
                out = tuple(odd if x == j else y for x, y in enumerate(args[6]))
                assert fn(*args[:6], out) is None, (j, odd)
        assert fn(*args[:6], list(args[6])) is None
    assert fn(*args) == 0
    torch.cuda.synchronize()
