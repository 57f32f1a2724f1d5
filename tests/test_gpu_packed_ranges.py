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


FAR = (0, 3, 10, 20, 23, 26, 31, 40, 60)      # powers of two below the largest


def far_scales(rng, w, shape, dtype):
    """Scales of a matrix [N, groups] each at one of FAR below the largest, two of which lie in every row and in
    every column of groups."""
    N, groups = shape
    down = rng.choice(FAR, shape)
    down[np.arange(N), rng.integers(0, groups, N)] = 0
    down[rng.integers(0, N, groups), np.arange(groups)] = 0
    if w["fmt"] == "mxfp4":
        w["s"] = (140 - down).astype(np.uint8)
        return F.e8m0_value(w["s"]).astype(np.float64), 2.0 ** 13
    top = 256.0
    v = top * 2.0 ** -down.astype(np.float64) * rng.uniform(0.5, 1.0, shape)
    w["s"], w["s_t"] = rounded(v, dtype)
    return w["s"], top


@BACK
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M", [16, 70, 1100])
@pytest.mark.parametrize("fmt", FORMATS[1:], ids=IDS[1:])
def test_scales_far_apart(hm, fmt, M, dtype, back):
    """Each weight alone, by rows of x (or dy) with one element of 1: whole where its scale is at least 2^-24
    (MXFP4: 2^-35) of the largest in its row, or its group over all rows in the gradient; below, the scale
    is within 2^-33 of the largest (MXFP4: the weight within 2^-36). In the gradient that is a row of W which dy
    takes alone, beside larger ones that it leaves out."""
    rng = np.random.default_rng([M, back])
    K, N, (f, group, zero) = 512, 300, fmt
    w = packed(rng, (N, K), f, group, zero, dtype)
    G = group or 32
    s, top = far_scales(rng, w, (N, K // G), dtype)
    W = P.values(w)
    n_in = N if back else K
    at = rng.integers(0, n_in, M)
    x = np.zeros((M, n_in))
    x[np.arange(M), at] = 1.0
    want = W[at] if back else W[:, at].T
    each = np.repeat(s, G, -1)
    each = each[at] if back else each[:, at].T
    got = call(hm, rounded(x, dtype)[1], w, M, K, N, back).double().cpu().numpy()
    if f == "mxfp4":
        off = np.where(each >= top * 2.0 ** -35, 0.0, top * 2.0 ** -36)
    else:
        off = np.where(each >= top * 2.0 ** -24, 0.0, 15 * top * 2.0 ** -33)
    half = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}[dtype]
    tiny = 2.0 ** -25 if dtype == "fp16" else 2.0 ** -134      # half the smallest step
    err = np.abs(got - want)
    assert (err <= off + half * (np.abs(want) + off) + tiny).all(), np.argwhere(err > off + half * np.abs(want) + tiny)[:4]
    whole = off == 0
    assert whole.any() and np.array_equal(got[whole], rounded(want, dtype)[0][whole])


@BACK
@pytest.mark.parametrize("M", [16, 70, 1100])
@pytest.mark.parametrize("fmt", FORMATS[1:], ids=IDS[1:])
def test_sums_of_scales_far_apart(hm, fmt, M, back):
    """The same bounds in whole sums, with each weight's part of them."""
    rng = np.random.default_rng([M, back, 1])
    K, N, (f, group, zero) = 512, 300, fmt
    w = packed(rng, (N, K), f, group, zero, "bf16")
    G = group or 32
    s, top = far_scales(rng, w, (N, K // G), "bf16")
    W = P.values(w)
    n_in = N if back else K
    x, xt = rounded(rng.standard_normal((M, n_in)), "bf16")
    lim = 2.0 ** -35 if f == "mxfp4" else 2.0 ** -24
    off = np.where(np.repeat(s, G, -1) >= top * lim, 0.0, top * (2.0 ** -36 if f == "mxfp4" else 15 * 2.0 ** -33))
    extra = np.abs(x) @ (off if back else off.T)
    got = call(hm, xt, w, M, K, N, back).double().cpu().numpy()
    ref, S = product(x, W, back), sums_of(x, w, W, back)
    noise = (n_in + 8) * 2.0 ** -24 * S + extra
    assert (np.abs(got - ref) <= 2.0 ** -8 * (np.abs(ref) + noise) * 1.01 + noise).all()


@BACK
@pytest.mark.parametrize("M", [3, 30, 70, 1100])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_every_e4m3_scale(hm, dtype, M, back):
    """Negative, zero and subnormal E4M3 scales: each weight alone, equal."""
    rng = np.random.default_rng([M, back, 2])
    K, N = 512, 300
    w = packed(rng, (N, K), "nvfp4")
    s = rng.integers(0, 256, w["s"].shape, dtype=np.uint8)
    w["s"] = np.where((s & 0x7F) == 0x7F, 0x80, s).astype(np.uint8)      # (0x7F and 0xFF are NaN)
    w["g"] = np.ones(1, np.float32)
    W = P.values(w)
    n_in = N if back else K
    at = rng.integers(0, n_in, M)
    x = np.zeros((M, n_in))
    x[np.arange(M), at] = 1.0
    want = W[at] if back else W[:, at].T
    assert (want < 0).any() and (want == 0).any()
    got = call(hm, rounded(x, dtype)[1], w, M, K, N, back).double().cpu().numpy()
    assert np.array_equal(got, want)


@BACK
@pytest.mark.parametrize("M", [2, 16, 40, 70, 1100])
def test_every_e8m0_scale(hm, M, back):
    """E8M0 bytes from 0 to 252, the last whose largest weights are finite in bf16: one byte a group of columns,
    so that every exponent is its own."""
    rng = np.random.default_rng([M, back, 3])
    K, N = 32 * 253, 40
    w = packed(rng, (N, K), "mxfp4")
    w["s"] = np.broadcast_to(np.arange(253, dtype=np.uint8), (N, 253)).copy()
    if not back:       # forward an exponent is a row's
        K, N = 64, 253
        w = packed(rng, (N, K), "mxfp4")
        w["s"] = np.broadcast_to(np.arange(253, dtype=np.uint8)[:, None], (N, 2)).copy()
    W = P.values(w)
    n_in = N if back else K
    at = rng.integers(0, n_in, M)
    x = np.zeros((M, n_in))
    x[np.arange(M), at] = 1.0
    want = W[at] if back else W[:, at].T
    got = call(hm, rounded(x, "bf16")[1], w, M, K, N, back).double().cpu().numpy()
    assert np.array_equal(got, want)


@pytest.mark.parametrize("M", [3, 33, 64, 70, 1100])
@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
def test_special_values_in_the_gradient(hm, fmt, M):
    """NaN and infinities in a row of dy: its own row only. A NaN scale: the columns of its group only."""
    import torch
    rng = np.random.default_rng(M)
    K, N = 256, 60
    w = packed(rng, (N, K), *fmt, "bf16")
    _, dyt = rounded(rng.standard_normal((M, N)), "bf16")
    clean = call(hm, dyt, w, M, K, N, True)
    assert torch.isfinite(clean).all()
    bad = dyt.clone()
    bad[1, 7], bad[2, 9] = float("nan"), float("-inf")
    dx = call(hm, bad, w, M, K, N, True)
    assert torch.isnan(dx[1]).all() and not torch.isfinite(dx[2]).any()
    keep = [m for m in range(M) if m not in (1, 2)]
    assert torch.equal(dx[keep], clean[keep])
    if fmt[0] == "int4":
        w["s_t"][5, 1] = float("nan")
    else:
        w["s"][5, 1] = 0x7F if fmt[0] == "nvfp4" else 255
    dx = call(hm, dyt, w, M, K, N, True)
    width = {"nvfp4": 16, "mxfp4": 32}.get(fmt[0], fmt[1])
    cols = torch.arange(K) // width == 1
    assert torch.isnan(dx[:, cols]).all() and torch.equal(dx[:, ~cols], clean[:, ~cols])
