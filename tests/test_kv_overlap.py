"""Buffers of a plan that must not share memory are refused before anything is
launched; lengths may be updated in place."""

import ctypes
import os

import pytest
import torch

import bit_quantized_gemm_qgemm_amd as qg

ERR_OVERLAP = -9
BATCH, WIDTH, STRIDE, FREE, TOKENS = 5, 6, 9, 7, 40
# buffers that do not touch, apart by less than their sizes
AT = dict(table=0x10000, cached=0x20000, added=0x20014, free_pages=0x20028, lens=0x20044,
          cu_tokens=0x20058, cu_pages=0x20070, slots=0x20088)
BYTES = dict(cached=4 * BATCH, added=4 * BATCH, free_pages=4 * FREE, lens=4 * BATCH,
             cu_tokens=4 * BATCH + 4, cu_pages=4 * BATCH + 4, slots=8 * TOKENS)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(qg.LIB_PATH):
        from bit_quantized_gemm_qgemm_amd import build
        build.build()
    return qg.lib()


@pytest.fixture(autouse=True)
def any_device(monkeypatch):
    if torch.cuda.is_available():
        pytest.skip("addresses that must not reach a GPU")
    monkeypatch.setenv("QGEMM_ARCH_OVERRIDE", "gfx950")


def plan(lib, **change):
    at = {**AT, **change}
    return lib.qgemm_kv_plan(*(ctypes.c_void_p(at[n]) for n in AT), BATCH, WIDTH, STRIDE, FREE, 16,
                             TOKENS, None)


OUTPUTS = ("lens", "cu_tokens", "cu_pages", "slots")


@pytest.mark.parametrize("one", OUTPUTS)
@pytest.mark.parametrize("other", ("cached", "added", "free_pages") + OUTPUTS)
def test_outputs_that_share_memory_are_refused(lib, one, other):
    if one == other:
        pytest.skip("one buffer")
    step = 8 if one == "slots" else 4
    for at in (AT[other], AT[other] + BYTES[other] - 4):     # its first entry, its last one
        if (one, at) == ("lens", AT["cached"]):
            continue                                         # in place: taken
        assert plan(lib, **{one: at - at % step}) == ERR_OVERLAP, (one, other, at)


@pytest.mark.parametrize("name", ("cached", "added", "free_pages") + OUTPUTS)
def test_the_table_shares_memory_with_nothing(lib, name):
    row = 4 * STRIDE
    for offset in (0, 4 * WIDTH - 4, row, 3 * row + 8, (BATCH - 1) * row + 4 * WIDTH - 4):
        at = AT["table"] + offset
        assert plan(lib, **{name: at - at % 8 if name == "slots" else at}) == ERR_OVERLAP, offset
    # an array that begins in the gap after a row and reaches into the next
    if name != "slots":
        assert plan(lib, **{name: AT["table"] + 4 * WIDTH}) == ERR_OVERLAP


def test_the_status_has_a_text():
    assert "share" in qg.status_string(ERR_OVERLAP)


def test_buffers_side_by_side_are_taken(lib):
    """Without a device the call then fails in the runtime, not in the checks."""
    assert plan(lib) not in (ERR_OVERLAP, -1, -2, -3)
    assert plan(lib, lens=AT["cached"]) not in (ERR_OVERLAP, -1, -2, -3)
    end = AT["table"] + 4 * (STRIDE * (BATCH - 1) + WIDTH)
    assert plan(lib, cached=end) != ERR_OVERLAP and plan(lib, cached=AT["table"] - 4 * BATCH) != ERR_OVERLAP
