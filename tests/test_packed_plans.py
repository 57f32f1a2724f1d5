"""Scratch of the operators on 4-bit matrices: enough for fewer rows, and none for what a call does not use."""
import numpy as np
import pytest

import weight_only_quantized_moe_amd as hm


def test_scratch_never_shrinks_over_all_sizes():
    r = np.random.default_rng(6)
    for _ in range(200):
        K, N = 32 * int(2 ** r.uniform(0, 13)), int(2 ** r.uniform(0, 18))
        rows = np.unique(np.concatenate([(2 ** r.uniform(0, 22, 60)).astype(np.int64), np.arange(18),
                                         [31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1023, 1024, 1025, 4096]]))
        plans = [hm.moe_linear_scratch_bytes(int(m), K, N) for m in rows]
        for (m, a), (n, b) in zip(zip(rows, plans), zip(rows[1:], plans[1:])):
            assert b[0] >= a[0] and b[1] >= a[1], f"[{N}, {K}]: {m} rows take {a}, {n} rows {b}"


@pytest.mark.parametrize("K", [1 << 17, 1 << 20])
def test_no_room_for_sums_that_one_block_has_alone(K):
    """A gradient of so many columns is not split over the rows of W: what it needs is dy, and exponents."""
    back = hm.moe_linear_scratch_bytes(64, K, 96)[1]
    assert back <= 64 * 96 * 2 + 4 * (K + 64) + (1 << 16)
