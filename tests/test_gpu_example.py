"""The example's layer, end to end, against fp64."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "decode_layer.py")


@pytest.mark.parametrize("cache", ["fp16", "e4m3"])
@pytest.mark.parametrize("prompts", [(5, 130, 1, 64, 47), (2100, 3)])
def test_decode_layer(cache, prompts):
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    print("case example", cache, prompts, flush=True)
    spec = importlib.util.spec_from_file_location("decode_layer", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    y, ref = example.run(steps=20, cache=cache, prompts=prompts)
    # Roundings on the way, each at most half a step of its value: the QKV product's output
    # (fp32 sums may round to the other neighbour: a whole fp16 step, 2^-10; in an e4m3 cache
    # that can move a code by its step, 2^-3, seldom and for a few elements), the attention's
    # (2^-11, a neighbour 2^-10) and the result's (2^-11).  Over a norm of independent errors
    # their sum bounds the relative error: 2^-10 + 2^-10 + 2^-11 < 2^-8.  Of the codes about
    # one in 2^6 lies within an fp16 step of a border, so they add 2^-3 * 2^-3 of one key's or
    # value's norm at most: 2^-6.
    error = float((y - ref).norm() / ref.norm())
    assert error <= (2.0 ** -8 if cache == "fp16" else 2.0 ** -8 + 2.0 ** -6), error
