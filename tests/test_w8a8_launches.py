"""Every size that the int8 products take leads to a launch that the device takes: less than
2^32 threads in one dimension of its grid.  Host-only."""

import os
import random

import pytest

import bit_quantized_gemm_qgemm_amd as qg

# waves of a workgroup with each tile
WAVES = {(16, 16, 8): 8, (16, 32, 4): 4, (16, 64, 4): 4, (32, 32, 4): 4, (32, 64, 4): 8, (32, 128, 1): 4,
         (64, 64, 2): 4, (64, 128, 1): 4, (96, 256, 1): 4, (128, 128, 1): 4, (128, 256, 1): 4, (256, 256, 1): 8}


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(qg.LIB_PATH):
        from bit_quantized_gemm_qgemm_amd import build
        build.build()
    return qg.lib()


def threads(M, N, K, experts, gated=False):
    """Workgroups for every row block that the experts can have, times their threads."""
    tile = qg.qgemm_w8a8_tile(M, N, K, experts, gated)
    rows, cols, _ = tile
    packed = 2 * -(-N // 2 // 16) * 16 if gated else -(-N // 16) * 16
    blocks = min(M, experts) + M // rows if experts else -(-M // rows)
    return -(-blocks * -(-packed // cols) // 8) * 8 * 64 * WAVES[tile]


@pytest.mark.parametrize("M,N,K,experts,gated", [
    (65536, 32767, 0, 1024, False), (1024, (1 << 21) - 1, 0, 1024, False), (1024, (1 << 21) - 1, 16, 1024, False),
    (1024, (1 << 21) - 2, 128, 1024, True), (1444, 1486202, 1024, 1024, True), (200, 10718822, 0, 1024, False),
    (741, 2896756, 256, 1024, True), (147, 14549384, 0, 512, True), (64, (1 << 24) - 33, 0, 0, False),
    ((1 << 28) - 1, 7, 0, 0, False), ((1 << 28) - 1, 7, 16, 1024, False), ((1 << 28) - 1, 6, 0, 1024, True),
])
def test_at_the_limits(M, N, K, experts, gated):
    assert threads(M, N, K, experts, gated) < 1 << 32


def test_sizes_at_random():
    rng = random.Random(1)
    some = 0
    for _ in range(20000):
        K, experts = rng.choice([0, 0, 16, 128, 256, 1024, 4096]), rng.choice([0, 1, 2, 16, 128, 512, 1024])
        N = min(int(2 ** rng.uniform(1, 24)), ((1 << 31) - 1) // max(K, 128) - 32)
        M = min(int(2 ** rng.uniform(0, 28)), (1 << 28) - 1, ((1 << 31) - 1) // N)
        gated = N % 2 == 0 and rng.random() < 0.5
        assert threads(M, N, K, experts, gated) < 1 << 32, (M, N, K, experts, gated)
        some += M * N > 1 << 30
    assert some > 1000
