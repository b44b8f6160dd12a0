"""Which kernel a block-scaled product takes (host code, nothing is launched)."""

import random

import pytest

from int8_int4_dequant_amd import qw

ESHAPE, EM, EARG = -3, -4, -9
F32, BF16 = 0, 1


def path(op, m, n, k, y_type=BF16, experts=0):
    return qw.qw_block_debug_path(op, experts, m, n, k, y_type)


TILED = 33000  # reported tiles of 64 and more weight rows are above


@pytest.mark.parametrize("m,n,k", [(131072, 151936, 4096),    # logits of a long batch: 0.3 million tiles
                                   (1 << 20, 65536, 1024), (1 << 26, 200, 300)])
@pytest.mark.parametrize("y_type", [F32, BF16])
def test_large_products_are_tiled(m, n, k, y_type):
    assert path(0, m, n, k, y_type) > TILED


@pytest.mark.parametrize("m,n,k,experts", [(1 << 20, 16384, 4096, 128), (1 << 21, 28672, 8192, 8)])
@pytest.mark.parametrize("y_type", [F32, BF16])
def test_large_grouped_products_are_tiled(m, n, k, experts, y_type):
    assert path(2, m, n, k, y_type, experts) > TILED


def test_expert_mlp_ways():
    assert path(3, 32, 1408, 4096, BF16, 64) == 1
    assert path(3, 400 * 64, 1408, 2048, BF16, 64) == 3
    assert path(3, 65536, 1 << 19, 128, BF16, 512) == 3      # its blocks take tile after tile
    assert path(3, 400 * 64, 1400, 2048, BF16, 64) == 2      # no whole blocks of hidden values
    assert path(3, 400 * 64, 1408, 2048, F32, 64) == 2       # fp32 sums: on the bf16 cores
    # more rows never go back to a way for fewer
    ways = [path(3, rows, 1408, 2048, BF16, 64) for rows in range(1, 20000, 7)]
    assert ways == sorted(ways)


def test_small_products():
    assert path(0, 1, 4096, 4096) == 1 and path(0, 1, 100, 128, F32) == 1
    assert path(0, 1, 100, 128 * 97) == 16016    # more blocks of k than the stream kernel holds
    assert path(0, 300, 100, 0) < TILED and path(2, 300, 100, 0, F32, 3) < TILED  # nothing to sum
    assert path(1, 100, 128, 512) == 0           # one tile is not cut


def test_tiles_fit_a_launch():
    """A tiled kernel is one launch, of at most 2^22 thread blocks."""
    rng = random.Random(5)
    for _ in range(20000):
        k = rng.choice([1, 100, 128, 300, 4096, 1 << 22])
        kp = qw.qw_block_pitch(k)
        m = int(2 ** rng.uniform(4, 36)) // kp + 17
        n = int(2 ** rng.uniform(0, 36)) // max(m, kp) + 1
        experts = rng.choice([0, 0, 1, 8, 512])
        tile = path(2 if experts else 0, m, n, k, rng.choice([F32, BF16]), experts)
        if tile > TILED:
            bn, bm = divmod(tile, 1000)
            assert (min(m, (m + max(experts, 1) * (bm - 1)) // bm)) * -(-n // bn) <= 1 << 22, (m, n, k, experts)


def test_refusals():
    assert path(4, 8, 8, 8) == path(-1, 8, 8, 8) == path(0, 8, 8, 8, 2) == EARG
    assert path(2, 8, 8, 8, F32, 0) == path(2, 8, 8, 8, F32, 513) == path(3, 8, 8, 8, F32, 0) == EARG
    assert path(0, 8, -1, 8) == path(0, 8, 8, -1) == path(0, 8, 8, (1 << 22) + 1) == ESHAPE
    assert path(0, -1, 8, 8) == path(2, (1 << 30) + 1, 8, 8, F32, 2) == EM
    assert path(3, (1 << 30) + 1, 8, 8, F32, 2) == ESHAPE


@pytest.mark.parametrize("topk,experts,d,f", [(1, 1, 128, 128), (2, 8, 512, 384), (8, 64, 4096, 1408), (3, 60, 1003, 300)])
def test_work_for_the_largest_call_is_enough_for_smaller_ones(topk, experts, d, f):
    L = qw.lib()
    edges = [4 * experts, 16 * experts, 64 * experts, 4096, 1 << 18, (1 << 18) * 3, 1 << 20]
    ts = sorted({max(0, e // topk + i) for e in edges for i in (-1, 0, 1, 2, 200)} | set(range(20)))
    for query in (lambda t: L.qw_moe_sort_work_bytes(t, topk, experts),
                  lambda t: L.qw_moe_mlp_work_bytes(t, topk, experts, d, f),
                  lambda t: L.qw_block_matmul_work_bytes(t, d)):
        sizes = [query(t) for t in ts]
        assert min(sizes) >= 0 and sizes == sorted(sizes)
    for t in (4 * experts // topk, 64 * experts // topk + 1):
        for e, dd, ff in ((experts + 1, d, f), (experts, d + 1, f), (experts, d, f + 1)):
            assert L.qw_moe_mlp_work_bytes(t, topk, e, dd, ff) >= L.qw_moe_mlp_work_bytes(t, topk, experts, d, f)
