"""Scales and rows far apart, and at the ends of their types' ranges, in the products with 4-bit matrices."""
import numpy as np
import pytest

from oracle import formats as F
from oracle import packed as P
from packed_testlib import FORMATS, IDS, check, offset_values, packed, rounded, upload

pytestmark = pytest.mark.gpu

BACK = pytest.mark.parametrize("back", [False, True], ids=["forward", "back"])


@pytest.fixture(scope="module")
def hm():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_moe_amd as m
    m.load_library()
    return m


def call(hm, xt, w, M, K, N, back, base=None):
    import torch
    y = torch.empty(M, K if back else N, dtype=xt.dtype, device="cuda")
    n = hm.moe_linear_scratch_bytes(M, K, N)[back]
    ws = torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device="cuda")
    (hm.moe_linear_backward if back else hm.moe_linear)(xt.cuda(), upload(w), y, base, ws)
    return y


def product(x, W, back):
    return (P.linear_backward if back else P.linear)(x, W)


def sums_of(x, w, W, back):
    S = offset_values(w, W)
    return np.abs(x) @ (S if back else S.T)


@BACK
@pytest.mark.parametrize("M", [20, 70, 1030])
@pytest.mark.parametrize("fmt", [FORMATS[0], FORMATS[1], FORMATS[4]], ids=["nvfp4", "mxfp4", "int4"])
def test_rows_near_the_ends_of_bf16(hm, fmt, M, back):
    """Rows whose results lie inside fp32, though sums without NVFP4's scale of the matrix would not. Forward,
    up to 1024 rows may be summed without exponents of their own: |x| below 2^128 / (2688 K) there."""
    rng = np.random.default_rng(M)
    K, N = 256, 160
    w = packed(rng, (N, K), *fmt, "bf16")
    W = P.values(w)
    n_in = N if back else K
    far = 121 if back or M > 1024 else 128 - 12 - 8 - 3     # 2688 < 2^12, K = 2^8, |x| < 8
    x = np.clip(rng.standard_normal((M, n_in)), -7.9, 7.9)
    x[3] = 0.0
    x[4] *= 2.0 ** far
    x[5] *= 2.0 ** -118
    x, xt = rounded(x, "bf16")
    scale = np.ones((M, 1))
    scale[4], scale[5] = 2.0 ** -far, 2.0 ** 118
    got = call(hm, xt, w, M, K, N, back).double().cpu().numpy() * scale
    check(got, product(x * scale, W, back), sums_of(x * scale, w, W, back), n_in + 8, "bf16")
    assert (got[3] == 0).all()
