"""moe_linear and moe_linear_backward against float64: every format and type, one row to many, odd
widths, strides, addends, special values, other streams, captured replays, and beside the adapters."""
import numpy as np
import pytest

from oracle import packed as P
from packed_testlib import FORMATS, IDS, check, offset_values, packed, rounded, torch_dtype, upload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hm():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_moe_amd as m
    m.load_library()
    return m


def scratch(hm, M, K, N, back):
    import torch
    n = hm.moe_linear_scratch_bytes(M, K, N)[back]
    return torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device="cuda")   # NaN in every type


def run(hm, rng, fmt, M, K, N, back, dtype, base="matrix", strided=False, w=None):
    """One call against the oracle. base: None, "matrix", "own" (the output itself) or "bias"."""
    import torch
    f, g, z = fmt
    w = packed(rng, (N, K), f, g, z, dtype) if w is None else w
    W = P.values(w)
    n_in, n_out = (N, K) if back else (K, N)
    x, xt = rounded(rng.standard_normal((M, n_in)), dtype)
    b, bt = rounded(rng.standard_normal((1 if base == "bias" else M, n_out)), dtype)
    pad = 5 if strided else 0

    def place(t, rows, cols):
        """On the GPU, behind an odd offset and with gaps between rows when strided."""
        buf = torch.full((rows * (cols + pad) + 3,), 7.0, dtype=t.dtype, device="cuda")
        v = buf[3 if strided else 0:][: rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
        v.copy_(t)
        return buf, v

    _, xd = place(xt, M, n_in)
    ybuf, y = place(torch.zeros(M, n_out, dtype=xt.dtype), M, n_out)
    bd = None
    if base == "matrix":
        _, bd = place(bt, M, n_out)
    elif base == "own":
        y.copy_(bt)
        bd = y
    elif base == "bias":
        bd = bt.cuda().expand(M, n_out)
    before = ybuf.clone()
    call = hm.moe_linear_backward if back else hm.moe_linear
    call(xd, upload(w), y, bd, scratch(hm, M, K, N, back))
    torch.cuda.synchronize()
    ref = (P.linear_backward if back else P.linear)(x, W, None if base is None else b)
    in_sums = offset_values(w, W)
    sums = np.abs(x) @ (in_sums if back else in_sums.T) + (0.0 if base is None else np.abs(b))
    tiled = back or M > 64      # (some of these take the packed product, which rounds no weight)
    step = 2.0 ** -11 if tiled and f == "int4" else 2.0 ** -24   # weights rounded to fp16
    rms = None
    if tiled and f == "int4":
        rms = np.sqrt(((x ** 2) @ ((W ** 2) if back else (W ** 2).T)).mean()) * 2.0 ** -11.5
    check(y, ref, sums, n_in + 8, dtype, step, rms, (fmt, M, K, N, back, dtype))
    # nothing beside the output is touched
    ybuf_view = ybuf[3 if strided else 0:][: M * (n_out + pad)].view(M, n_out + pad)
    ybuf_view[:, :n_out] = before[3 if strided else 0:][: M * (n_out + pad)].view(M, n_out + pad)[:, :n_out]
    assert torch.equal(ybuf, before)


# rows: each number of row tiles the packed product takes, both sides of the gradient's last few rows (64)
# and of the tiled product's tiles; more forward rows are test_tiles'
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 32, 33, 64, 65, 128, 129, 300])
@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
def test_rows(hm, fmt, M):
    rng = np.random.default_rng([M, FORMATS.index(fmt)])
    run(hm, rng, fmt, M, 384, 100, False, "bf16" if M % 2 else "fp16")
    run(hm, rng, fmt, M, 384, 100, True, "fp16" if M % 2 else "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("K,N", [(32, 1), (64, 3), (96, 16), (128, 17), (160, 33), (416, 257), (1024, 1003),
                                 (2144, 130), (128, 2048), (8320, 48)])
@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
def test_widths(hm, fmt, K, N, dtype):
    """Columns that end inside a step of 128, in every count of blocks; rows that end inside a tile."""
    step = max(fmt[1], 32)
    K = -(-K // step) * step
    rng = np.random.default_rng([K, N, FORMATS.index(fmt)])
    for M in (1, 5, 40, 70):
        run(hm, rng, fmt, M, K, N, False, dtype, "matrix" if M > 1 else None)
    for M in (1, 70):
        run(hm, rng, fmt, M, K, N, True, dtype, "matrix" if M > 1 else None)


# each number of pairs of 256 columns that a wave keeps, with the last pair whole and partial, one and two
# tiles an item, and more columns than any of them takes
@pytest.mark.parametrize("K,N", [(256, 40), (288, 40), (2048, 70), (2336, 33), (3840, 20), (4000, 20), (4096, 8200),
                                 (5120, 24), (6144, 24), (7936, 24), (4128, 24), (2048, 8210)])
@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
def test_shares_of_the_reduction(hm, fmt, K, N):
    step = max(fmt[1], 32)
    K = -(-K // step) * step
    rng = np.random.default_rng([K, N])
    for M, dtype in ((1, "bf16"), (11, "fp16"), (33, "bf16")):
        run(hm, rng, fmt, M, K, N, False, dtype, "matrix")


# the tiled product's tiles and shares of the reduction axis, both sides of each choice, forward and back
@pytest.mark.parametrize("M,K,N", [(65, 512, 20000), (1030, 256, 300), (1100, 1056, 700), (2049, 96, 1500),
                                   (4100, 64, 4100), (2500, 288, 2100), (1025, 2048, 96)])
def test_tiles(hm, M, K, N):
    rng = np.random.default_rng([M, K, N])
    for fmt, back, dtype in ((FORMATS[0], False, "bf16"), (FORMATS[2], False, "fp16"), (FORMATS[1], True, "bf16"),
                             (FORMATS[3], True, "fp16")):
        run(hm, rng, fmt, M, K, N, back, dtype, "matrix")


@pytest.mark.parametrize("M", [1, 16, 17, 33, 64])
@pytest.mark.parametrize("K,N", [(32, 5), (160, 31), (1056, 1000), (6144, 130), (512, 4133)])
def test_gradient_of_few_rows(hm, M, K, N):
    """The gradient straight from the codes: shares of n, partial blocks of 32 rows and of 128 columns."""
    rng = np.random.default_rng([M, K, N])
    for fmt, dtype in ((FORMATS[0], "fp16"), (FORMATS[1], "bf16"), (FORMATS[2], "bf16")):
        run(hm, rng, fmt, M, K, N, True, dtype, "matrix")


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("base", [None, "matrix", "own", "bias"])
@pytest.mark.parametrize("M", [1, 3, 20, 50, 90])
def test_addends_and_strides(hm, M, base, back):
    rng = np.random.default_rng([M, back])
    for fmt in (FORMATS[0], FORMATS[4]):
        run(hm, rng, fmt, M, 320, 75, back, "bf16", base, True)


def test_wide_scales(hm):
    """Scales 2^+-30 apart (INT4, bf16) and E8M0 bytes of the whole range: the fp16 form of the
    many-row product keeps each column's own exponent."""
    rng = np.random.default_rng(5)
    for fmt in (FORMATS[1], FORMATS[3]):
        for M in (3, 80, 1030):
            w = packed(rng, (40, 256), *fmt, "bf16", spread=0)
            far = 2.0 ** rng.integers(-30, 31, (40, 1))
            if fmt[0] == "mxfp4":
                w["s"] = (w["s"] + np.log2(far)).astype(np.uint8)
            else:
                w["s"], w["s_t"] = rounded(w["s"] * far, "bf16")
            run(hm, rng, fmt, M, 256, 40, False, "bf16", None, w=w)


@pytest.mark.parametrize("M", [4, 80, 1030])
@pytest.mark.parametrize("fmt", [FORMATS[0], FORMATS[1], FORMATS[2]], ids=["nvfp4", "mxfp4", "int4"])
def test_whole_numbers_are_exact(hm, fmt, M):
    """Codes, scales and rows whose products and sums are whole numbers below 2^11: equal."""
    import torch
    rng = np.random.default_rng(M)
    K, N = 160, 50
    w = packed(rng, (N, K), *fmt, "fp16")
    if fmt[0] == "nvfp4":
        w["s"], w["g"] = np.full_like(w["s"], 0x40), np.ones(1, np.float32)     # 2
    elif fmt[0] == "mxfp4":
        w["s"] = np.full_like(w["s"], 128)
    else:
        w["s"], w["s_t"] = rounded(np.ones_like(w["s"]), "fp16")
    W = P.values(w)
    for back in (False, True):
        n_in, n_out = (N, K) if back else (K, N)
        x = np.where(rng.random((M, n_in)) < 0.2, rng.integers(-2, 3, (M, n_in)), 0).astype(np.float64)
        y = torch.empty(M, n_out, dtype=torch.float16, device="cuda")
        xd = torch.from_numpy(x).to(torch.float16).cuda()
        (hm.moe_linear_backward if back else hm.moe_linear)(xd, upload(w), y, None, scratch(hm, M, K, N, back))
        ref = x @ (W if back else W.T)
        assert np.abs(ref).max() < 2048
        assert np.array_equal(y.cpu().double().numpy(), ref)


@pytest.mark.parametrize("M", [3, 70, 1030])
def test_special_values_stay_in_their_row(hm, M):
    """NaN and infinities in a row of x: its own row only; NaN scales: their column only."""
    import torch
    rng = np.random.default_rng(M)
    K, N = 256, 60
    for fmt in (FORMATS[0], FORMATS[1], FORMATS[3]):
        w = packed(rng, (N, K), *fmt, "bf16")
        x, xt = rounded(rng.standard_normal((M, K)), "bf16")
        clean = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        hm.moe_linear(xt.cuda(), upload(w), clean, None, scratch(hm, M, K, N, 0))
        xt[1, 7] = float("nan")
        xt[2, 9] = float("inf")
        y = torch.empty_like(clean)
        hm.moe_linear(xt.cuda(), upload(w), y, None, scratch(hm, M, K, N, 0))
        assert torch.isnan(y[1]).all()
        assert not torch.isfinite(y[2]).any()
        keep = [m for m in range(M) if m not in (1, 2)]
        assert torch.equal(y[keep], clean[keep])
        if fmt[0] == "int4":
            w["s_t"][5, 0] = float("nan")
        else:
            w["s"][5, 0] = 0x7F if fmt[0] == "nvfp4" else 255
        xt = rounded(x, "bf16")[1]
        hm.moe_linear(xt.cuda(), upload(w), y, None, scratch(hm, M, K, N, 0))
        cols = [n for n in range(N) if n != 5]
        assert torch.isnan(y[:, 5]).all() and torch.equal(y[:, cols], clean[:, cols])
        # and in the gradient: the columns of that group
        if M > 64:
            dy = torch.randn(M, N, device="cuda").bfloat16()
            dx = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
            hm.moe_linear_backward(dy, upload(w), dx, None, scratch(hm, M, K, N, 1))
            width = {"nvfp4": 16, "mxfp4": 32}.get(fmt[0], fmt[1])
            assert torch.isnan(dx[:, :width]).all() and torch.isfinite(dx[:, width:]).all()


@pytest.mark.parametrize("M", [70, 1030])
def test_extreme_rows(hm, M):
    """Zero rows, rows near the ends of bf16's range, one row beside them."""
    import torch
    rng = np.random.default_rng(1)
    K, N = 256, 40
    w = packed(rng, (N, K), *FORMATS[3], "bf16")
    W = P.values(w)
    x = rng.standard_normal((M, K))
    x[3] = 0.0
    x[4] *= 2.0 ** 118
    x[5] *= 2.0 ** -120
    x, xt = rounded(x, "bf16")
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    hm.moe_linear(xt.cuda(), upload(w), y, None, scratch(hm, M, K, N, 0))
    got = y.double().cpu().numpy()
    assert (got[3] == 0).all()
    scale = np.ones((M, 1))
    scale[4], scale[5] = 2.0 ** -118, 2.0 ** 120
    check(got * scale, P.linear(x * scale, W), np.abs(x * scale) @ offset_values(w, W).T, K + 8, "bf16", 2.0 ** -11)


@pytest.mark.parametrize("M", [4, 40, 100, 1030])
def test_subnormal_rows(hm, M):
    """fp16 rows of whole multiples of 2^-24, which fp16 holds below its normal numbers: all of them
    count. Products are whole numbers of 2^-14 below 2^11 of them: equal."""
    import torch
    rng = np.random.default_rng(M)
    K, N = 256, 40
    w = packed(rng, (N, K), "int4", 32, False, "fp16")
    w["s"], w["s_t"] = rounded(np.full_like(w["s"], 1024.0), "fp16")
    W = P.values(w)
    for back in (False, True):
        n_in, n_out = (N, K) if back else (K, N)
        x = np.where(rng.random((M, n_in)) < 0.2, rng.integers(-3, 4, (M, n_in)), 0) * 2.0 ** -24
        y = torch.empty(M, n_out, dtype=torch.float16, device="cuda")
        xd = torch.from_numpy(x).to(torch.float16).cuda()
        (hm.moe_linear_backward if back else hm.moe_linear)(xd, upload(w), y, None, scratch(hm, M, K, N, back))
        ref = x @ (W if back else W.T)
        assert np.abs(ref).max() < 2048 * 2.0 ** -14
        assert np.array_equal(y.cpu().double().numpy(), ref)


@pytest.mark.parametrize("M", [2, 48, 100, 1030])
@pytest.mark.parametrize("back", [False, True])
def test_captured_and_on_another_stream(hm, M, back):
    """A captured call, replayed with new rows between eager calls on the same scratch."""
    import torch
    rng = np.random.default_rng(M)
    K, N = 512, 200
    w = upload(packed(rng, (N, K), *FORMATS[4], "bf16"))
    n_in, n_out = (N, K) if back else (K, N)
    call = hm.moe_linear_backward if back else hm.moe_linear
    ws = scratch(hm, M, K, N, back)
    x = torch.randn(M, n_in, device="cuda").bfloat16()
    y, eager = (torch.empty(M, n_out, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(x, w, y, None, ws)
    torch.cuda.current_stream().wait_stream(side)
    call(x, w, eager, None, ws)
    torch.cuda.synchronize()
    assert torch.equal(y, eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(x, w, y, None, ws)
    for _ in range(4):
        x.copy_(torch.randn(M, n_in, device="cuda"))
        call(x, w, eager, None, ws)
        y.zero_()
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager)


@pytest.mark.parametrize("M", [200, 1030])
def test_two_calls_at_once(hm, M):
    """Two streams, each with its own scratch."""
    import torch
    rng = np.random.default_rng(3)
    K, N = 1024, 512
    w = upload(packed(rng, (N, K), *FORMATS[0], "bf16"))
    xs = [torch.randn(M, K, device="cuda").bfloat16() for _ in range(2)]
    want = [torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ws = [scratch(hm, M, K, N, 0) for _ in range(2)]
    for x, y, s in zip(xs, want, ws):
        hm.moe_linear(x, w, y, None, s)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [torch.empty_like(y) for y in want]
    for _ in range(5):
        for x, y, s, st in zip(xs, got, ws, streams):
            with torch.cuda.stream(st):
                hm.moe_linear(x, w, y, None, s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_gradient_against_differences(hm):
    """<dy, y(x + e) - y(x - e)> = 2 <dx, e> for steps that the types hold exactly."""
    import torch
    rng = np.random.default_rng(11)
    for fmt in (FORMATS[0], FORMATS[1], FORMATS[4]):
        for M in (4, 70):
            K, N = 256, 96
            w = packed(rng, (N, K), *fmt, "fp16")
            W = P.values(w)
            x = rng.integers(-3, 4, (M, K)).astype(np.float64)
            e = rng.integers(-1, 2, (M, K)).astype(np.float64)
            dy = rng.integers(-2, 3, (M, N)).astype(np.float64)

            def y_of(v):
                y = torch.empty(M, N, dtype=torch.float16, device="cuda")
                hm.moe_linear(torch.from_numpy(v).half().cuda(), upload(w), y, None, scratch(hm, M, K, N, 0))
                return y.double().cpu().numpy()
            dx = torch.empty(M, K, dtype=torch.float16, device="cuda")
            hm.moe_linear_backward(torch.from_numpy(dy).half().cuda(), upload(w), dx, None, scratch(hm, M, K, N, 1))
            lhs = (dy * (y_of(x + e) - y_of(x - e))).sum(1)
            rhs = 2 * (dx.double().cpu().numpy() * e).sum(1)
            # half steps of fp16 of each y and dx, and of each weight in their sums
            ys = np.abs(x + e) @ np.abs(W.T) + np.abs(x - e) @ np.abs(W.T)
            tol = (np.abs(dy) * ys).sum(1) * 2 * 2.0 ** -11 \
                + 2 * (np.abs(e) * (np.abs(dy) @ np.abs(W))).sum(1) * 2 * 2.0 ** -11
            assert (np.abs(lhs - rhs) <= tol).all()


@pytest.mark.parametrize("M", [1, 12, 150])
def test_with_adapters(hm, M):
    """A frozen projection with adapters beside it, forward and backward, as one program runs them:
    y = lora(x, base = linear(x)), dx = lora_backward(dy, dbase = linear_backward(dy))."""
    import torch
    rng = np.random.default_rng(M)
    K, N, G, r = 256, 192, 3, 16
    w = packed(rng, (N, K), *FORMATS[1], "bf16")
    W = P.values(w)
    x, xt = rounded(rng.standard_normal((M, K)), "bf16")
    dy, dyt = rounded(rng.standard_normal((M, N)), "bf16")
    A, At = rounded(rng.standard_normal((G, r, K)) * K ** -0.5, "bf16")
    B, Bt = rounded(rng.standard_normal((G, N, r)) * r ** -0.5, "bf16")
    scale = rng.uniform(0.5, 2, G).astype(np.float32)
    ids = rng.integers(-1, G, M).astype(np.int32)
    dev = [t.cuda() for t in (xt, dyt, At, Bt)]
    xd, dyd, Ad, Bd = dev
    sd, idd = torch.from_numpy(scale).cuda(), torch.from_numpy(ids).cuda()
    pw = upload(w)
    f, b = hm.moe_lora_scratch_bytes(M, G, K, N, r)
    lf, lb = hm.moe_linear_scratch_bytes(M, K, N)
    ws = torch.empty(max(f, b, lf, lb, 256), dtype=torch.uint8, device="cuda")
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    z = torch.empty(M, r, device="cuda")
    dx = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    dA, dB = torch.empty(G, r, K, device="cuda"), torch.empty(G, N, r, device="cuda")

    def step():
        hm.moe_linear(xd, pw, y, None, ws)
        hm.moe_lora(xd, idd, Ad, Bd, sd, y, y, z, ws)
        hm.moe_linear_backward(dyd, pw, dx, None, ws)
        hm.moe_lora_backward(dyd, xd, z, idd, Ad, Bd, sd, dx, dx, dA, dB, ws)

    step()
    on = (ids >= 0)[:, None]
    g = np.maximum(ids, 0)
    zr = np.where(on, np.einsum("mrk,mk->mr", A[g], x), 0.0)
    add = np.where(on, scale[g][:, None] * np.einsum("mnr,mr->mn", B[g], zr), 0.0)
    dz = np.where(on, scale[g][:, None] * np.einsum("mnr,mn->mr", B[g], dy), 0.0)
    dadd = np.einsum("mrk,mr->mk", A[g], dz)
    yl, dl = P.linear(x, W), P.linear_backward(dy, W)
    for got, part, extra in ((y, yl, add), (dx, dl, dadd)):
        err = np.abs(got.double().cpu().numpy() - (part + extra))
        # two roundings to bf16, and fp32 sums of at most 300 terms of values up to a few
        assert (err <= 2.0 ** -8 * (np.abs(part) + np.abs(part + extra)) * 1.01 + 300 * 2.0 ** -24 * 40).all()
    eager = [t.clone() for t in (y, dx, dA, dB)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in (y, dx, dA, dB):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip((y, dx, dA, dB), eager))


def test_large_offsets(hm):
    """A matrix whose codes pass 2^31 bytes, a few of its last rows checked."""
    import torch
    K, N = 16384, 270000            # 2.2 GB of codes
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    q = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    s = torch.randint(116, 121, (N, K // 32), dtype=torch.uint8, device="cuda", generator=gen)
    x, xt = rounded(np.random.default_rng(0).standard_normal((2, K)), "bf16")
    y = torch.empty(2, N, dtype=torch.bfloat16, device="cuda")
    hm.moe_linear(xt.cuda(), hm.PackedMatrix(hm.WEIGHT_MXFP4, q, s), y)
    rows = [0, 1, 131072, 262143, 262144, N - 2, N - 1]
    W = P.values({"fmt": "mxfp4", "q": q[rows].cpu().numpy(), "s": s[rows].cpu().numpy()})
    check(y[:, rows], P.linear(x, W), np.abs(x) @ np.abs(W).T, K + 8, "bf16")


def test_many_slabs(hm):
    """An output wider than one slab of the tiled product's scratch, both directions."""
    rng = np.random.default_rng(2)
    run(hm, rng, FORMATS[0], 66, 32, 530000, False, "bf16", "bias")
    run(hm, rng, FORMATS[3], 66, 8192, 4224, True, "bf16", "matrix")


def test_no_rows(hm):
    import torch
    w = upload(packed(np.random.default_rng(0), (16, 64), "mxfp4"))
    x, y = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 16, dtype=torch.bfloat16, device="cuda")
    hm.moe_linear(x, w, y)
    hm.moe_linear_backward(y, w, x)
