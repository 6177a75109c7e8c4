"""The kernel choice of the 8-bit products on the host: every size that fits a card's memory has a
kernel whose launch takes it."""
import random

import pytest

import weight_only_quantized_amd as w4

MEMORY = 288 << 30


@pytest.mark.parametrize("T,topk,E,K,N", [(1 << 20, 2, 64, 4096, 14336), (524289, 8, 64, 8192, 4096), (524289, 8, 128, 8192, 4096),
                                          (32850, 1, 2, 130944, 64), (1 << 22, 4, 256, 1024, 2048)])
def test_gathered_calls_past_32_bits_run_on_tiles(T, topk, E, K, N):
    """Tokens whose codes pass 2^32 bytes: the kernels that split K would need more threads than a
    launch has (32 x 64 results of at least 512 threads)."""
    assert T * K >= 1 << 32
    plan = w4.w4a16_test_w8a8_plan(T * topk, K, N, E)
    assert plan >= 100 and plan % 100 >= 3


def test_every_size_has_a_kernel():
    rng = random.Random(5)
    seen = set()
    for _ in range(20000):
        M = min((1 << 31) - 1, round(2 ** rng.uniform(0, 31)))
        K, N = 128 * round(2 ** rng.uniform(0, 9.99)), 64 * round(2 ** rng.uniform(0, 16))
        E = rng.choice([0, round(2 ** rng.uniform(0, 20))])
        used = 3 * M * K + 2 * M * N + max(E, 1) * K * N
        if used <= MEMORY:
            plan = w4.w4a16_test_w8a8_plan(M, K, N, E)
            assert plan >= 100, (M, K, N, E)
            seen.add(plan % 100)
    assert len(seen) >= 6


ROWS = (1, 2, 4, 16, 17, 77, 512, 1023, 1024, 1025, 1026, 2048, 4096, 1 << 17, 1 << 20)


@pytest.mark.parametrize("K", [128, 4096, 14336, 130944])
def test_one_workspace_serves_every_row_count(K):
    """The size for all calls of up to so many rows grows with the rows and covers each of them."""
    last = 0
    for M in ROWS:
        room = w4.w8a8_max_workspace_bytes(M, K)
        assert room >= last and all(room >= w4.w8a8_workspace_bytes(m, K) for m in ROWS if m <= M)
        assert any(room == w4.w8a8_workspace_bytes(m, K) for m in ROWS if m <= M)
        last = room
    for M, k in ((0, K), (-1, K), (1 << 31, K), (4, 100), (4, 1 << 17)):
        assert w4.w8a8_max_workspace_bytes(M, k) == 0


def test_calls_take_the_common_workspace():
    """What a call finds after the workspace's size is right: a bias off its alignment."""
    F, K, N = 1 << 40, 4096, 64
    room = w4.w8a8_max_workspace_bytes(4096, K)
    for M in (1, 16, 512, 1024, 1025, 4096):
        assert w4.lib().w8a8_gemm(F, 0, F, F, F + 1, F, 0, M, K, N, 1, F, room, None) == 4
