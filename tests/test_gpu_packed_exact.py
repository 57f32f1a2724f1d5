"""What enters the products of moe_linear, its gradient and moe_tokens is not rounded: an addend that takes
the leading bits out of a result shows the ones below, which a result alone would round away."""
import numpy as np
import pytest

from oracle import packed as P
from packed_testlib import check, offset_values, packed, rounded, upload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hm():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_moe_amd as m
    m.load_library()
    return m


def identity(fmt, N, K):
    """A packed matrix whose row n is 1 in column n % K and 0 elsewhere (code 2 is 1.0)."""
    q = np.zeros((N, K // 2), np.uint8)
    n = np.arange(N)
    q[n, n % K // 2] = np.where(n % 2, 0x20, 0x02)
    w = {"fmt": fmt, "q": q, "z": None, "g": None, "group": 0}
    if fmt == "nvfp4":
        w["s"], w["g"] = np.full((N, K // 16), 0x38, np.uint8), np.ones(1, np.float32)
    else:
        w["s"] = np.full((N, K // 32), 127, np.uint8)
    assert (P.values(w)[n, n % K] == 1).all() and P.values(w).sum() == N
    return w


def one_expert(w):
    return dict(w, q=w["q"][None], s=w["s"][None])


def tokens(hm, x, w13, w2, base, S):
    """One expert of weight 1, or, with S, a shared expert beside one whose weights are zero."""
    import torch
    M, H = x.shape
    zero = lambda w: dict(w, q=np.zeros_like(w["q"]))  # noqa: E731
    shared = (upload(w13), upload(w2), None) if S else None
    a, b = (one_expert(zero(w) if S else w) for w in (w13, w2))
    y = torch.empty(M, H, dtype=x.dtype, device="cuda")
    I = w2["q"].shape[1] * 2
    ws = torch.full((hm.moe_tokens_scratch_bytes(M, 1, H, I, 1, I if S else 0),), 0xFF, dtype=torch.uint8, device="cuda")
    hm.moe_tokens(x.cuda(), torch.zeros(1, H, dtype=x.dtype, device="cuda"), upload(a), upload(b), 1, y,
                  None if base is None else base.cuda(), shared, scratch=ws)
    return y.cpu().double().numpy()


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("H,I", [(64, 32), (64, 96), (256, 256), (320, 288)])   # steps, pairs, partial pairs
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_h_keeps_its_24_bits(hm, fmt, H, I, shared):
    """y = base + h with base the fp16 nearest to -h: what is left is h below its eleventh bit. x has one
    element other than zero, so that gate and up are one exact product each; silu is off by (|gate| + 4) of
    fp32's half steps (exp's argument, exp, 1 +, reciprocal, product), the two products beside by one each."""
    rng = np.random.default_rng([H, I])
    w13 = packed(rng, (2 * I, H), fmt, spread=1)
    W13 = P.values(w13)
    M = 5
    x = np.zeros((M, H))
    cols = rng.choice(H, M, replace=False)
    x[np.arange(M), cols] = rng.integers(3, 9, M) * 2.0
    a, b = x @ W13[:I].T, x @ W13[I:].T
    h = (a / (1 + np.exp(-a)) * b)[:, np.arange(H) % I]
    base, bt = rounded(-h, "fp16")
    y = tokens(hm, rounded(x, "fp16")[1], w13, identity(fmt, H, I), bt, shared)
    want = h + base
    tol = np.abs(h) * ((np.abs(a)[:, np.arange(H) % I] + 7) * 2.0 ** -24) * 1.01 + np.abs(want) * 2.0 ** -11 + 2.0 ** -25
    # the test can tell 16 bits (off by up to 2^-17) from 24
    assert (tol < np.abs(h) * 2.0 ** -18)[np.abs(h) > 0.25].any()
    assert (np.abs(y - want) <= tol).all(), float((np.abs(y - want) / tol).max())


@pytest.mark.parametrize("H,I", [(64, 32), (256, 256)])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_an_infinite_h_is_infinite(hm, fmt, H, I):
    """gate and up of 2^100 and more: h is an infinity, and so is y wherever its weight is not zero."""
    rng = np.random.default_rng(I)
    w13 = packed(rng, (2 * I, H), fmt)
    w13["q"] = np.full_like(w13["q"], 0x22)       # positive weights
    w2 = packed(rng, (H, I), fmt)
    w2["q"] = np.where(rng.random(w2["q"].shape) < 0.5, 0x11, 0x19).astype(np.uint8)   # element 2j + 1: 0.5, 2j: +-0.5
    w2["q"][:, 1:] = 0x22
    x = np.zeros((3, H))
    x[1, 0] = 2.0 ** 110
    x[0, 1] = x[2, 2] = 1.0
    y = tokens(hm, rounded(x, "bf16")[1], w13, w2, None, False)
    W2 = P.values(w2)
    up = (W2 > 0).all(1)
    assert up.any() and not up.all()
    assert (y[1, up] == np.inf).all() and np.isnan(y[1, ~up]).all()
    assert np.isfinite(y[[0, 2]]).all()


def weights_alone(hm, M, K, N, back, group, zero, dtype):
    """base + W, row by row: rows of x (or of dy) with one element of 1, base the nearest to -W. What is left
    of a weight of up to 16 bits below its first 8 or 11 is a number of the type: equal."""
    import torch
    rng = np.random.default_rng([M, K, N, back, group, zero])
    w = packed(rng, (N, K), "int4", group, zero, dtype, spread=0)
    w["s"], w["s_t"] = rounded(rng.uniform(1.0, 8.0, (N, K // group)), dtype)
    W = P.values(w)
    n_in, n_out = (N, K) if back else (K, N)
    at = rng.integers(0, n_in, M)
    x = np.zeros((M, n_in))
    x[np.arange(M), at] = 1.0
    mine = W[at] if back else W[:, at].T
    base, bt = rounded(-mine, dtype)
    left = mine + base
    assert (rounded(left, dtype)[0] == left).all() and (left != 0).mean() > 0.1
    y = torch.empty(M, n_out, dtype=bt.dtype, device="cuda")
    n = hm.moe_linear_scratch_bytes(M, K, N)[back]
    ws = torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device="cuda")
    (hm.moe_linear_backward if back else hm.moe_linear)(rounded(x, dtype)[1].cuda(), upload(w), y, bt.cuda(), ws)
    assert np.array_equal(y.cpu().double().numpy(), left)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("group,zero", [(32, True), (64, True), (128, True), (32, False), (128, False)])
@pytest.mark.parametrize("M", [1, 16, 30, 64])
def test_int4_weights_are_whole_in_few_rows(hm, M, group, zero, dtype):
    for back in (False, True):
        weights_alone(hm, M, 384, 150, back, group, zero, dtype)


# the tiled product: one slab's shares of the reduction axis, and whole tiles
@pytest.mark.parametrize("group,zero", [(32, True), (64, True), (128, True), (32, False), (128, False)])
@pytest.mark.parametrize("M,K,N", [(70, 384, 150), (1030, 384, 150), (1300, 128, 4001)])
def test_int4_weights_are_whole_in_many_fp16_rows(hm, M, K, N, group, zero):
    for back in (False, True):
        weights_alone(hm, M, K, N, back, group, zero, "fp16")


@pytest.mark.parametrize("group,zero", [(32, True), (64, True), (128, True), (32, False), (128, False)])
@pytest.mark.parametrize("M,K,N", [(70, 384, 150), (1030, 384, 150), (1300, 128, 4001), (66, 8192, 300), (70, 128, 5000)])
def test_int4_weights_are_whole_in_many_bf16_rows(hm, M, K, N, group, zero):
    """Zero points are a product of their own there: of the groups' sums of x, or of dy and (8 - z) s."""
    for back in (False, True):
        weights_alone(hm, M, K, N, back, group, zero, "bf16")


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,K,N", [(200, 640, 333), (1100, 2176, 520)])
def test_zero_points_at_both_ends(hm, M, K, N, group, back):
    """Codes and zero points of 0 and 15, where the two products cancel most."""
    import torch
    rng = np.random.default_rng([M, K, N, group])
    w = packed(rng, (N, K), "int4", group, True, "bf16", spread=1)
    w["q"] = rng.choice([0x00, 0xFF, 0xF0, 0x0F], w["q"].shape).astype(np.uint8)
    w["z"] = rng.choice([0, 15, 0xF0], w["z"].shape).astype(np.uint8)
    W = P.values(w)
    n_in, n_out = (N, K) if back else (K, N)
    x, xt = rounded(rng.standard_normal((M, n_in)) + 1.0, "bf16")
    y = torch.empty(M, n_out, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((hm.moe_linear_scratch_bytes(M, K, N)[back],), 0xFF, dtype=torch.uint8, device="cuda")
    (hm.moe_linear_backward if back else hm.moe_linear)(xt.cuda(), upload(w), y, None, ws)
    ref = (P.linear_backward if back else P.linear)(x, W)
    S = offset_values(w, W)
    check(y, ref, np.abs(x) @ (S if back else S.T), n_in + 8, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [40, 1100])
def test_one_group(hm, M, group, dtype):
    """A row of W that is one group, and one row of W."""
    for back in (False, True):
        weights_alone(hm, M, group, 40, back, group, True, dtype)
    weights_alone(hm, M, 256, 1, True, group, True, dtype)
