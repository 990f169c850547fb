"""Limits of the key-value cache calls that keep a launch below 2^32 threads."""

import ctypes
import os

import pytest

import bit_quantized_gemm_qgemm_amd as qg

GOOD, ERR_SHAPE = ctypes.c_void_p(0x10000), -2   # never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(qg.LIB_PATH):
        from bit_quantized_gemm_qgemm_amd import build
        build.build()
    return qg.lib()


@pytest.mark.parametrize("tokens,kv_heads,dim", [
    (1 << 31, 1, 16), (1 << 30, 1, 16), (1 << 26, 1, 256), (1 << 20, 1 << 7, 128),
])
def test_append_refuses_a_grid_that_is_too_large(lib, tokens, kv_heads, dim):
    assert lib.qgemm_kv_append(1, 1, GOOD, GOOD, GOOD, GOOD, GOOD, None, None, tokens, kv_heads, dim,
                               dim, dim, dim, dim, 4, 16, 16 * dim * kv_heads, 16 * dim, dim,
                               None) == ERR_SHAPE


@pytest.mark.parametrize("batch,heads", [(1 << 23, 1), (1 << 12, 1 << 11), (1, 1 << 23)])
def test_attention_refuses_a_grid_that_is_too_large(lib, batch, heads):
    fn = lib.qgemm_paged_attention_workspace_bytes
    assert fn(batch, heads, 1, 64, 16, 0) == ERR_SHAPE
    assert fn(batch - 1 if heads == 1 else batch, heads if heads == 1 else heads - 1, 1, 64, 16, 0) >= 0
    assert lib.qgemm_paged_attention(1, 1, GOOD, GOOD, GOOD, GOOD, GOOD, None, None, GOOD, GOOD, batch,
                                     heads, 1, 64, 64, 64, 4, 16, 1024, 1024, 64, 1, 1, 16, 0, 0.125,
                                     None) == ERR_SHAPE


def test_workspace_grows_with_the_shared_path_only(lib):
    fn = lib.qgemm_paged_attention_workspace_bytes
    assert fn(4, 8, 2, 128, 768, 0) == 0 and fn(4, 8, 2, 128, 1 << 20, 768) == 0
    assert fn(4, 8, 2, 128, 769, 0) > 0
