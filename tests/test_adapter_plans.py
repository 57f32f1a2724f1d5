"""The adapters' scratch plans: a buffer made for the largest batch serves every smaller one."""
import numpy as np
import pytest

import weight_only_quantized_moe_amd as hm


def _never_shrinks(rows, *shape):
    plans = [hm.moe_lora_scratch_bytes(int(m), *shape) for m in rows]
    for (m, a), (n, b) in zip(zip(rows, plans), zip(rows[1:], plans[1:])):
        assert b[0] >= a[0] and b[1] >= a[1], f"{shape}: {m} rows take {a}, {n} rows {b}"


@pytest.mark.parametrize("shape", [(16, 4096, 4096, 64), (8, 4096, 4096, 64), (1, 4096, 4096, 64), (300, 2048, 1536, 16),
                                   (2048, 64, 64, 8), (4, 6144, 4096, 128), (60, 8192, 8, 40), (3, 8, 8192, 24)])
def test_scratch_never_shrinks_row_by_row(shape):
    """Through every change of plan: how tiles are found, one launch or two, tile rows, splits."""
    _never_shrinks(range(0, 4200), *shape)


def test_scratch_never_shrinks_over_all_sizes():
    r = np.random.default_rng(5)
    for _ in range(300):
        G, rank = int(2 ** r.uniform(0, 11)), 8 * int(r.integers(1, 17))
        K, N = (8 * int(2 ** r.uniform(0, 12)) for _ in range(2))
        rows = np.unique(np.concatenate([(2 ** r.uniform(0, 22, 60)).astype(np.int64), np.arange(18),
                                         [127, 128, 129, 511, 512, 799, 800, 1024, 1025, 2048, 2049, 2999, 3000, 8192, 8193]]))
        _never_shrinks(rows, G, K, N, rank)


def test_permute_scratch_never_shrinks():
    for k, E in ((1, 1), (8, 256), (16, 1024), (6, 61)):
        n = [hm.moe_permute_scratch_bytes(M, k, E) for M in range(0, 20000, 37)]
        assert all(a <= b for a, b in zip(n, n[1:]))
