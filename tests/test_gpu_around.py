"""The operators around the experts on the GPU, against the float64 oracle: row movements,
routing gradient and adapters, forward and backward, at the sizes, masks and layouts where
they can go wrong; their runs together; graphs and streams.

Tolerances are bounds, element by element: a sum of n products in fp32 is off by at most
(n + 1) * 2^-24 times the sum of the products' magnitudes (any order), and a rounding to a
type by at most half a step, eps / 2 relative (TINY covers results below the normal range)."""
import numpy as np
import pytest

import synth
from hmoe_testlib import (check_output, make_layer, scratch_for, tiny_packed, to_dev, to_dev_bits,
                          torch_mod)
from oracle import around as R
from oracle import formats as F
from oracle import layer as OL

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
TINY = 1e-30
HALF = {"bfloat16": 2.0 ** -8, "float16": 2.0 ** -11, "float32": U32}
# half of fp16's smallest step, for results below its normal range
FLOOR = {"bfloat16": TINY, "float16": 2.0 ** -25, "float32": TINY}


@pytest.fixture(scope="module")
def hm():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_moe_amd as m
    m.load_library()
    return m


def f64(t):
    return t.detach().double().cpu().numpy()


def close(got, ref, bound, what):
    got, ref = f64(got), np.asarray(ref, np.float64)
    assert got.shape == ref.shape
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, worst "
                           f"{np.nanmax(np.abs(got - ref) - bound):.3e} beyond the bound, first at "
                           f"{np.argwhere(bad)[0]}")


def rand(torch, seed, *shape, dtype="float32", std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(getattr(torch, dtype)).cuda()


def padded(torch, t, pad, shift):
    """The same matrix inside a wider one: row stride + pad, first column at `shift`."""
    wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    v = wide[:, shift:shift + t.shape[1]]
    v.copy_(t)
    return v


def ids_of(M, k, E, kind, seed=0):
    r = np.random.default_rng([seed, M, k, E])
    if kind == "one":                       # every token to the same experts
        ids = np.tile(r.permutation(E)[:k], (M, 1))
    elif kind == "none":                    # nothing held here
        ids = np.full((M, k), E)
    else:
        ids = np.argsort(r.random((M, E)), axis=1)[:, :k]
        if kind == "share":                 # ids of other processes, below and above
            ids = ids * 3 - E
            ids.reshape(-1)[:: 7] = 2 ** 31 - 1
            ids.reshape(-1)[3:: 11] = -(2 ** 31)
    return ids.astype(np.int32)


def run_permute(hm, torch, x, ids, E, rows=None):
    M, k = ids.shape
    rows = torch.full((M * k, x.shape[1]), 77.0, dtype=x.dtype, device="cuda") if rows is None else rows
    i32 = dict(dtype=torch.int32, device="cuda")
    srt, sr, off = torch.full((M * k,), 5, **i32), torch.full((M, k), 5, **i32), torch.full((E + 1,), 5, **i32)
    n = hm.moe_permute_scratch_bytes(M, k, E)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    hm.moe_permute(x, to_dev(ids), E, rows, srt, sr, off, ws)
    torch.cuda.synchronize()
    return rows, srt, sr, off


# 256 x 8 slots is the last single launch, 257 x 8 the first sort; 1024 x 8 the last sort in one
# block; 5000 x 8 with 1024 experts has its block count bounded by the count table
PERMUTE = [(0, 2, 4, 8, "bfloat16", "any"), (1, 1, 1, 1, "float32", "any"), (1, 8, 128, 2048, "bfloat16", "any"),
           (3, 16, 40, 13, "float16", "any"), (8, 8, 256, 6144, "bfloat16", "share"),
           (128, 8, 256, 96, "float16", "share"), (129, 8, 256, 96, "bfloat16", "share"),
           (129, 8, 256, 33, "bfloat16", "none"), (31, 2, 8, 2047, "float32", "one"),
           (256, 8, 64, 64, "bfloat16", "any"), (257, 8, 64, 65, "float32", "any"),
           (1500, 3, 1024, 8, "bfloat16", "share"), (5000, 8, 1024, 4, "float16", "any"),
           (4096, 8, 8, 4, "bfloat16", "one"), (2000, 2, 2, 40, "float32", "one"),
           (1300, 16, 17, 24, "bfloat16", "any"),
           (1024, 8, 256, 24, "bfloat16", "share"), (1025, 8, 641, 24, "float16", "share"), (900, 9, 640, 17, "float32", "any")]


@pytest.mark.parametrize("M,k,E,H,dtype,kind", PERMUTE)
def test_permute(hm, M, k, E, H, dtype, kind):
    torch = torch_mod()
    x, ids = rand(torch, M, M, H, dtype=dtype), ids_of(M, k, E, kind)
    rows, srt, sr, off = run_permute(hm, torch, x, ids, E)
    ix = R.permute_index(ids, E)
    np.testing.assert_array_equal(off.cpu().numpy(), ix["off"])
    np.testing.assert_array_equal(srt.cpu().numpy(), ix["sorted"])
    np.testing.assert_array_equal(sr.cpu().numpy(), ix["slot_row"])
    # rows past the last held one stay as they were
    np.testing.assert_array_equal(f64(rows), R.permute(f64(x), ix, np.full((M * k, H), 77.0)))


@pytest.mark.parametrize("M", [9, 300])
@pytest.mark.parametrize("H,pad,shift", [(40, 8, 0), (40, 3, 1), (41, 7, 5)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_row_movements_strided(hm, M, H, pad, shift, dtype):
    """Rows inside wider matrices, at odd offsets: what lies between them stays."""
    torch = torch_mod()
    k, E = 4, 9
    x, ids = rand(torch, 1, M, H, dtype=dtype), ids_of(M, k, E, "share")
    wide = torch.full((M * k, H + pad), 3.0, dtype=x.dtype, device="cuda")
    rows, _, sr, off = run_permute(hm, torch, padded(torch, x, pad, shift), ids, E, wide[:, shift:shift + H])
    ix = R.permute_index(ids, E)
    want = np.full((M * k, H + pad), 3.0)
    want[:, shift:shift + H] = R.permute(f64(x), ix, want[:, shift:shift + H])
    np.testing.assert_array_equal(f64(wide), want)
    src, w, dy = rand(torch, 2, M * k, H, dtype=dtype), rand(torch, 3, M, k), rand(torch, 4, M, H, dtype=dtype)
    tight = [torch.empty(M, H, dtype=x.dtype, device="cuda"), torch.zeros(M * k, H, dtype=x.dtype, device="cuda")]
    dw = [torch.empty(M, k, device="cuda") for _ in range(2)]
    hm.moe_unpermute(src, sr, w, tight[0])
    hm.moe_unpermute_backward(dy, src, sr, w, tight[1], dw[0])
    out = torch.full((M, H + pad), 3.0, dtype=x.dtype, device="cuda")
    dr = torch.full((M * k, H + pad), 0.0, dtype=x.dtype, device="cuda")
    hm.moe_unpermute(padded(torch, src, pad, shift), sr, w, out[:, shift:shift + H])
    hm.moe_unpermute_backward(padded(torch, dy, pad, shift), padded(torch, src, pad, shift), sr, w,
                              dr[:, shift:shift + H], dw[1])
    torch.cuda.synchronize()
    assert torch.equal(out[:, shift:shift + H], tight[0]) and torch.equal(dr[:, shift:shift + H], tight[1])
    assert torch.equal(dw[0], dw[1])
    keep = [c for c in range(H + pad) if not shift <= c < shift + H]
    assert bool((out[:, keep] == 3.0).all()) and bool((dr[:, keep] == 0.0).all())


ROWS = [(1, 1, 1, "float32"), (1, 8, 2048, "bfloat16"), (8, 8, 6144, "bfloat16"), (5, 16, 13, "float16"),
        (33, 9, 1000, "bfloat16"), (64, 6, 2049, "float32"), (257, 3, 130, "float16"), (300, 8, 520, "bfloat16")]


@pytest.mark.parametrize("M,k,H,dtype", ROWS)
@pytest.mark.parametrize("kind", ["any", "share"])
def test_unpermute_and_gradients(hm, M, k, H, dtype, kind):
    torch = torch_mod()
    E = max(k, 11)
    sr = R.permute_index(ids_of(M, k, E, kind), E)["slot_row"].copy()
    if kind == "share" and M > 4:
        sr[1] = -1                                        # a token none of whose slots is held
        sr[2, 0], sr[3, 0] = M * k, 2 ** 31 - 1           # out of range: as dropped
    live = np.unique(sr[(sr >= 0) & (sr < M * k)])
    rows = rand(torch, 1, M * k, H, dtype=dtype)
    dead = np.setdiff1d(np.arange(M * k), live)
    if dead.size:                                         # rows that nobody names are never read
        rows[torch.from_numpy(dead).cuda()] = float("nan")
    w, dy = rand(torch, 2, M, k), rand(torch, 3, M, H, dtype=dtype)
    srd = to_dev(sr)
    y, dx = (torch.full((M, H), 9.0, dtype=rows.dtype, device="cuda") for _ in range(2))
    dr = torch.full((M * k, H), 9.0, dtype=rows.dtype, device="cuda")
    dw = torch.full((M, k), 9.0, device="cuda")
    hm.moe_unpermute(rows, srd, w, y)
    hm.moe_permute_backward(rows, srd, dx)
    hm.moe_unpermute_backward(dy, rows, srd, w, dr, dw)
    torch.cuda.synchronize()
    v, wn, dyn = f64(rows), f64(w), f64(dy)
    half, floor = HALF[dtype], FLOOR[dtype]
    sums = np.abs(np.nan_to_num(v))
    for got, weight, what in ((y, wn, "y"), (dx, None, "dx")):
        ref = R.unpermute(v, sr, weight)
        mag = R.unpermute(sums, sr, None if weight is None else np.abs(weight))
        close(got, ref, (k + 1) * U32 * mag * (1 + half) + half * np.abs(ref) + floor, what)
    ref_r, ref_w = R.unpermute_backward(dyn, v, sr, wn, np.full((M * k, H), 9.0))
    _, mag_w = R.unpermute_backward(np.abs(dyn), sums, sr, wn, np.zeros((M * k, H)))
    # one product in fp32, then the rounding to the rows' type
    close(dr, ref_r, (half + 2 * U32) * np.abs(ref_r) + floor, "drows")
    close(dw, ref_w, (H + 1) * U32 * mag_w + TINY, "dw")


@pytest.mark.parametrize("M,E,k", [(0, 8, 2), (1, 1, 1), (1, 128, 8), (7, 61, 6), (8, 256, 8), (130, 1024, 16),
                                   (1000, 257, 3), (33, 16, 16)])
def test_route_backward(hm, M, E, k):
    torch = torch_mod()
    lg = rand(torch, M + E, M, E, std=3.0)
    ids = torch.empty(M, k, dtype=torch.int32, device="cuda")
    w = torch.empty(M, k, device="cuda")
    if M:
        hm.moe_route(lg, k, ids, w)
    dw = rand(torch, 5, M, k)
    dl = torch.full((M, E), 9.0, device="cuda")
    hm.moe_route_backward(ids, w, dw, dl)
    torch.cuda.synchronize()
    i, wn, dn = ids.cpu().numpy(), f64(w), f64(dw)
    mag = np.zeros((M, E))
    np.put_along_axis(mag, i.astype(np.int64), wn * (np.abs(dn) + (wn * np.abs(dn)).sum(1, keepdims=True)), 1) if M else None
    close(dl, R.route_backward(i, wn, dn, E), (k + 4) * U32 * mag + TINY, "dlogits")


def test_route_backward_odd_ids(hm):
    """The same id twice adds up, ids outside [0, E) add nothing, NaN stays in its token."""
    torch = torch_mod()
    ids = np.array([[3, 3, 1], [-1, 2, 9], [0, 1, 2]], np.int32)
    w = np.array([[.5, .25, .25], [.2, .3, .5], [.1, .2, .7]], np.float32)
    dw = np.array([[1, 2, 4], [1, 2, 4], [np.nan, 0, 0]], np.float32)
    dl = torch.empty(3, 5, device="cuda")
    hm.moe_route_backward(to_dev(ids), to_dev(w), to_dev(dw), dl)
    got = f64(dl)
    ref = R.route_backward(ids, w, dw, 5)
    np.testing.assert_allclose(got[:2], ref[:2], rtol=0, atol=1e-5)
    assert np.isnan(got[2, :3]).all() and (got[2, 3:] == 0).all() and np.isfinite(got[:2]).all()


# ---- adapters ------------------------------------------------------------------------------

def lora_ids(M, G, kind, seed=0):
    r = np.random.default_rng([seed, M, G])
    if kind == "one":
        ids = np.full(M, G - 1)
    elif kind == "none":
        ids = np.full(M, -1)
    elif kind == "runs":                                   # requests of many tokens each
        ids = np.sort(r.integers(0, G, M))
    else:
        ids = r.integers(0, G, M)
        if kind == "mixed":
            ids[r.random(M) < 0.3] = -1
            ids[:: 17] = G + 5
            ids[1:: 23] = -(2 ** 31)
    return ids.astype(np.int32)


class LoraCase:
    def __init__(self, torch, M, G, K, N, r, kind, seed=0):
        bf = "bfloat16"
        self.M, self.G, self.K, self.N, self.r = M, G, K, N, r
        self.ids_np = lora_ids(M, G, kind, seed)
        self.ids = to_dev(self.ids_np)
        self.x, self.dy = rand(torch, 1 + seed, M, K, dtype=bf), rand(torch, 2, M, N, dtype=bf)
        self.base, self.dbase = rand(torch, 3, M, N, dtype=bf), rand(torch, 4, M, K, dtype=bf)
        self.A, self.B = rand(torch, 5, G, r, K, dtype=bf, std=K ** -0.5), rand(torch, 6, G, N, r, dtype=bf)
        self.scale = rand(torch, 7, G)
        self.held = (self.ids_np >= 0) & (self.ids_np < G)

    def scratch(self, hm, torch):
        f, b = hm.moe_lora_scratch_bytes(self.M, self.G, self.K, self.N, self.r)
        # filled with NaN: nothing of it may reach a result
        return [torch.full((max(n, 256) // 4,), float("nan"), device="cuda") for n in (f, b)]

    def forward(self, hm, torch, base="given"):
        y = torch.full((self.M, self.N), 7.0, dtype=torch.bfloat16, device="cuda")
        z = torch.full((self.M, self.r), 7.0, device="cuda")
        hm.moe_lora(self.x, self.ids, self.A, self.B, self.scale, self.base if base == "given" else base, y, z,
                    self.scratch(hm, torch)[0])
        torch.cuda.synchronize()
        return y, z

    def backward(self, hm, torch, z, dbase="given"):
        dx = torch.full((self.M, self.K), 7.0, dtype=torch.bfloat16, device="cuda")
        dA = torch.full((self.G, self.r, self.K), 7.0, device="cuda")
        dB = torch.full((self.G, self.N, self.r), 7.0, device="cuda")
        hm.moe_lora_backward(self.dy, self.x, z, self.ids, self.A, self.B, self.scale,
                             self.dbase if dbase == "given" else dbase, dx, dA, dB, self.scratch(hm, torch)[1])
        torch.cuda.synchronize()
        return dx, dA, dB

    def check_forward(self, y, z, base=None):
        x, a, b, s = (np.nan_to_num(f64(t)) for t in (self.x, self.A, self.B, self.scale))
        base = f64(self.base) if base is None else base
        ry, rz = R.lora(x, self.ids_np, a, b, s, base)
        my, mz = R.lora(np.abs(x), self.ids_np, np.abs(a), np.abs(b), np.abs(s), np.abs(base))
        ez = (self.K + 1) * U32 * mz
        close(z, rz, ez + TINY, "z")
        # z's own error through B; its two bf16 parts leave 2^-16; 2 r products and the base
        # added up in fp32; y rounded once
        ey = R.lora(np.zeros_like(x), self.ids_np, a, b, s, 0 * base)[0]
        for g in range(self.G):
            t = self.ids_np == g
            ey[t] = abs(s[g]) * (ez[t] + 2.0 ** -16 * np.abs(rz[t]) + 2 * U32 * np.abs(rz[t])) @ np.abs(b[g]).T
        ey += (2 * self.r + 4) * U32 * my
        close(y, ry, ey * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ry) + TINY, "y")

    def check_backward(self, z, dx, dA, dB, dbase=None):
        x, dy, zz = (np.nan_to_num(f64(t)) for t in (self.x, self.dy, z))
        a, b, s = f64(self.A), f64(self.B), f64(self.scale)
        dbase = f64(self.dbase) if dbase is None else dbase
        args = (dy, x, zz, self.ids_np, a, b, s, dbase)
        rx, rA, rB = R.lora_backward(*args)
        ab = [np.abs(v) if v is not self.ids_np else v for v in args]
        mx, mA, mB = R.lora_backward(*ab)
        counts = np.array([(self.ids_np == g).sum() for g in range(self.G)])[:, None, None]
        # dz: N + 2 products and roundings, relative to its magnitude sum; dx as y above
        rel = (self.N + 3) * U32
        ex = (rel + 2.0 ** -16 + (2 * self.r + 4) * U32) * mx
        close(dx, rx, ex * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(rx) + TINY, "dx")
        # weight gradients: three bf16 parts leave 2^-24 of dz (z), then three sums of `counts`
        close(dA, rA, (rel + (3 * counts + 12) * U32) * mA + TINY, "dA")
        close(dB, rB, (3 * counts + 14) * U32 * mB + TINY, "dB")


# ranks on both sides of 16, 32, 64 (packed parts, MFMA depths); rows on both sides of 16, 32,
# 64 (tile rows), of 24 and 48 rows an adapter (tile heights), of 128 and 2048 (how blocks find
# their tiles) and of 1024 (one launch); adapters on both sides of 255 (counts a block holds);
# K and N below, at and past 64 (steps, column groups); weight gradients with and without waves
# that share rows
LORA = [(1, 1, 8, 8, 8, "one"), (1, 16, 2048, 1536, 16, "any"), (2, 3, 72, 40, 24, "mixed"), (15, 1, 64, 64, 16, "one"),
        (16, 2, 128, 72, 32, "any"), (17, 1, 200, 136, 40, "one"), (33, 4, 264, 520, 64, "mixed"),
        (64, 48, 6144, 4096, 16, "mixed"), (65, 1, 320, 192, 8, "one"), (100, 4, 136, 64, 72, "runs"),
        (130, 2, 256, 264, 96, "mixed"), (200, 3, 512, 328, 128, "runs"), (150, 2048, 64, 64, 8, "any"),
        (1024, 5, 96, 88, 16, "mixed"), (1025, 5, 96, 88, 16, "mixed"), (1100, 2048, 24, 16, 8, "mixed"),
        (1500, 1, 200, 72, 64, "one"), (3000, 7, 72, 200, 48, "runs"), (2500, 40, 136, 24, 104, "mixed"),
        (5000, 3, 64, 64, 24, "any"), (70, 2, 8, 16, 120, "none"), (1200, 2, 16, 8, 8, "none"),
        (128, 5, 72, 64, 16, "mixed"), (129, 5, 72, 64, 16, "mixed"), (500, 255, 40, 88, 16, "mixed"),
        (500, 256, 40, 88, 16, "mixed"), (900, 254, 2056, 72, 128, "any"), (2048, 9, 96, 88, 64, "mixed"),
        (2049, 9, 96, 88, 64, "mixed"), (2048, 255, 24, 40, 40, "any"), (700, 1, 4104, 264, 64, "one"),
        (1024, 60, 2048, 1536, 32, "mixed"), (90, 20, 4096, 4104, 64, "any"), (300, 70, 520, 2056, 128, "mixed"),
        (120, 2, 8200, 136, 32, "mixed"), (2000, 1, 4096, 64, 24, "one"),
        (9000, 300, 24, 16, 8, "mixed"), (20000, 1500, 16, 8, 16, "any"),
        (7000, 3, 136, 24, 128, "mixed"), (7000, 400, 72, 16, 96, "mixed"),
        (4500, 1, 72, 64, 16, "one"), (4500, 20, 72, 64, 32, "one"), (4200, 2, 2056, 1544, 64, "runs")]


@pytest.mark.parametrize("M,G,K,N,r,kind", LORA)
def test_lora_forward_and_gradients(hm, M, G, K, N, r, kind):
    torch = torch_mod()
    c = LoraCase(torch, M, G, K, N, r, kind)
    # what rows without an adapter hold must not reach anything
    if (~c.held).any():
        off = torch.from_numpy(np.flatnonzero(~c.held)).cuda()
        c.x[off] = float("nan")
        c.dy[off] = float("inf")
    y, z = c.forward(hm, torch)
    c.check_forward(y, z)
    off = torch.from_numpy(np.flatnonzero(~c.held)).cuda()
    assert torch.equal(y[off], c.base[off])
    z[off] = float("nan")
    dx, dA, dB = c.backward(hm, torch, z)
    c.check_backward(z, dx, dA, dB)
    assert torch.equal(dx[off], c.dbase[off])
    again = c.forward(hm, torch)
    assert torch.equal(again[0], y)
    assert all(torch.equal(p, q) for p, q in zip(c.backward(hm, torch, z), (dx, dA, dB)))


@pytest.mark.parametrize("M", [20, 1300])
def test_lora_base_forms_and_strides(hm, M):
    """No base, base in place, no z, and rows inside wider matrices give the same bits."""
    torch = torch_mod()
    c = LoraCase(torch, M, 3, 72, 136, 24, "mixed")
    y, z = c.forward(hm, torch)
    y0, z0 = c.forward(hm, torch, base=None)
    c.check_forward(y0, z0, base=np.zeros((M, c.N)))
    ws = c.scratch(hm, torch)
    inplace = c.base.clone()
    hm.moe_lora(c.x, c.ids, c.A, c.B, c.scale, inplace, inplace, None, ws[0])
    assert torch.equal(inplace, y)
    wide = torch.full((M, c.N + 5), 3.0, dtype=torch.bfloat16, device="cuda")
    hm.moe_lora(padded(torch, c.x, 3, 1), c.ids, c.A, c.B, c.scale, padded(torch, c.base, 7, 3),
                wide[:, 1:1 + c.N], None, ws[0])
    assert torch.equal(wide[:, 1:1 + c.N], y) and bool((wide[:, 1 + c.N:] == 3.0).all()) and bool((wide[:, 0] == 3.0).all())
    dx, dA, dB = c.backward(hm, torch, z)
    dx0, dA0, dB0 = c.backward(hm, torch, z, dbase=None)
    c.check_backward(z, dx0, dA0, dB0, dbase=np.zeros((M, c.K)))
    inplace, dA1, dB1 = c.dbase.clone(), torch.empty_like(dA), torch.empty_like(dB)
    hm.moe_lora_backward(padded(torch, c.dy, 1, 1), padded(torch, c.x, 9, 2), z, c.ids, c.A, c.B, c.scale,
                         inplace, inplace, dA1, dB1, ws[1])
    torch.cuda.synchronize()
    assert torch.equal(inplace, dx) and torch.equal(dA1, dA) and torch.equal(dB1, dB)


def test_lora_no_rows(hm):
    """M = 0: the forward does nothing, the gradients are zeros."""
    torch = torch_mod()
    c = LoraCase(torch, 0, 3, 64, 32, 8, "any")
    c.forward(hm, torch)
    _, dA, dB = c.backward(hm, torch, torch.empty(0, 8, device="cuda"))
    assert not dA.any() and not dB.any()


def test_lora_infinite_rows_stay_in_their_rows(hm):
    torch = torch_mod()
    c = LoraCase(torch, 40, 2, 64, 72, 16, "any")
    y, z = c.forward(hm, torch)
    c.x[5, 3], c.x[21, 60] = float("inf"), float("nan")
    y1, z1 = c.forward(hm, torch)
    rest = [m for m in range(40) if m not in (5, 21)]
    assert torch.equal(y1[rest], y[rest]) and torch.equal(z1[rest], z[rest])
    assert bool(torch.isinf(z1[5]).all()) and bool(torch.isnan(z1[21]).all())
    assert not torch.isfinite(y1[[5, 21]].float()).any()


# ---- runs together -------------------------------------------------------------------------

def test_chain_matches_the_layer(hm):
    """moe_route, moe_permute, the experts' products on moe_dequant's weights and
    moe_unpermute compute what hybrid_moe_forward computes (its output bar)."""
    torch = torch_mod()
    packed, w = tiny_packed("nvfp4", "prefix")
    E, H, I, k, M = packed["E"], packed["H"], packed["I"], packed["top_k"], 200
    layer, wts = make_layer(packed, M), hm.DeviceWeights(packed)
    xb, lg = synth.activations_bf16(w, M), to_dev(synth.router_logits(w, M))
    x = to_dev_bits(xb)
    y = torch.empty_like(x)
    hm.hybrid_moe_forward(layer, wts, x, lg, y, scratch_for(layer))
    ids = torch.empty(M, k, dtype=torch.int32, device="cuda")
    tw = torch.empty(M, k, device="cuda")
    hm.moe_route(lg, k, ids, tw)
    rows, srt, sr, off = run_permute(hm, torch, x.view(torch.bfloat16), ids.cpu().numpy(), E)
    out = torch.empty(M * k, H, device="cuda")
    ends = off.cpu().tolist()
    for e in range(E):
        W13, W2 = torch.empty(2 * I, H, device="cuda"), torch.empty(H, I, device="cuda")
        hm.moe_dequant(layer, wts, e, hm.TENSOR_W13, W13)
        hm.moe_dequant(layer, wts, e, hm.TENSOR_W2, W2)
        a, b = ends[e], ends[e + 1]
        gu = rows[a:b].float() @ W13.t()
        out[a:b] = (torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]) @ W2.t()
    chain = torch.empty(M, H, device="cuda")
    hm.moe_unpermute(out, sr, tw, chain)
    torch.cuda.synchronize()
    check_output(y.cpu().numpy().view(np.uint16), f64(chain), "layer against the chain")


@pytest.mark.parametrize("M", [5, 40])
def test_adapters_beside_the_layer(hm, M):
    """hybrid_moe_forward then moe_lora in place on one stream: layer plus adapters."""
    torch = torch_mod()
    packed, w = tiny_packed("nvfp4", "prefix")
    H = packed["H"]
    layer, wts = make_layer(packed, M), hm.DeviceWeights(packed)
    xb, lg = synth.activations_bf16(w, M), synth.router_logits(w, M)
    c = LoraCase(torch, M, 4, H, H, 16, "mixed")
    c.x = to_dev_bits(xb).view(torch.bfloat16)
    y = torch.empty(M, H, dtype=torch.int16, device="cuda")
    hm.hybrid_moe_forward(layer, wts, to_dev_bits(xb), to_dev(lg), y, scratch_for(layer))
    alone = y.clone()
    hm.moe_lora(c.x.view(torch.int16), c.ids, c.A, c.B, c.scale, y, y, None, c.scratch(hm, torch)[0])
    torch.cuda.synchronize()
    c.base = alone.view(torch.bfloat16)
    _, z = c.forward(hm, torch)
    c.check_forward(y.view(torch.bfloat16), z)
    ref = OL.forward(packed, xb, lg)["y"]
    # against the oracle's layer with the oracle's adapters on top, at the layer's bar
    ref = R.lora(F.bf16_value(xb), c.ids_np, f64(c.A), f64(c.B), f64(c.scale), ref)[0]
    check_output(y.cpu().numpy().view(np.uint16), ref, f"M={M}")


def test_adapters_per_expert_on_permuted_rows(hm):
    """One group per (adapter, expert) on rows in expert order, then back into tokens."""
    torch = torch_mod()
    M, k, E, n_ad, K, N, r = 90, 4, 6, 3, 64, 128, 8
    ids = ids_of(M, k, E, "any")
    ad = np.random.default_rng(1).integers(-1, n_ad, M)
    c = LoraCase(torch, M * k, n_ad * E, K, N, r, "any")
    x = rand(torch, 9, M, K, dtype="bfloat16")
    rows, srt, sr, off = run_permute(hm, torch, x, ids, E)
    slot = srt.cpu().numpy()
    expert = ids.reshape(-1)[slot]
    c.ids_np = np.where(ad[slot // k] < 0, -1, ad[slot // k] * E + expert).astype(np.int32)
    c.ids, c.x = to_dev(c.ids_np), rows
    y, z = c.forward(hm, torch)
    c.check_forward(y, z)
    w = rand(torch, 10, M, k)
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    hm.moe_unpermute(y, sr, w, out)
    ref, mag = (R.unpermute(v, sr.cpu().numpy(), u) for v, u in ((f64(y), f64(w)), (np.abs(f64(y)), np.abs(f64(w)))))
    close(out, ref, (k + 1) * U32 * mag * 2 + 2.0 ** -8 * np.abs(ref) + TINY, "combined")


def test_training_step_gradients(hm):
    """Forward and backward of route -> permute -> experts -> unpermute against float64
    autograd of the whole layer: logits, tokens and expert weights."""
    torch = torch_mod()
    M, k, E, H = 70, 3, 8, 48
    lg, x, dy = rand(torch, 1, M, E), rand(torch, 2, M, H), rand(torch, 3, M, H)
    W = rand(torch, 4, E, H, H, std=H ** -0.5)
    ids, tw = torch.empty(M, k, dtype=torch.int32, device="cuda"), torch.empty(M, k, device="cuda")
    hm.moe_route(lg, k, ids, tw)
    rows, srt, sr, off = run_permute(hm, torch, x, ids.cpu().numpy(), E)
    ends = off.cpu().tolist()
    out, drows, drin = (torch.empty(M * k, H, device="cuda") for _ in range(3))
    parts = [(e, slice(ends[e], ends[e + 1])) for e in range(E)]
    for e, p in parts:
        out[p] = rows[p] @ W[e].t()
    y, dx, dw, dl = torch.empty_like(x), torch.empty_like(x), torch.empty_like(tw), torch.empty_like(lg)
    hm.moe_unpermute(out, sr, tw, y)
    hm.moe_unpermute_backward(dy, out, sr, tw, drows, dw)
    dW = torch.empty_like(W)
    for e, p in parts:
        drin[p] = drows[p] @ W[e]
        dW[e] = drows[p].t() @ rows[p]
    hm.moe_permute_backward(drin, sr, dx)
    hm.moe_route_backward(ids, tw, dw, dl)
    torch.cuda.synchronize()
    l6, x6, W6 = (t.double().cpu().requires_grad_() for t in (lg, x, W))
    top = ids.cpu().long()
    w6 = torch.softmax(l6.gather(1, top), 1)
    y6 = sum(w6[:, j:j + 1] * torch.bmm(W6[top[:, j]], x6[:, :, None])[:, :, 0] for j in range(k))
    y6.backward(dy.double().cpu())
    # every value is a sum of at most 3 stages of H, k or M fp32 terms of its own magnitude;
    # 3 * 200 * 2^-24 of the largest value bounds each
    for got, ref, what in ((y, y6, "y"), (dx, x6.grad, "dx"), (dW, W6.grad, "dW"), (dl, l6.grad, "dlogits")):
        ref = ref.detach().numpy()
        close(got, ref, 600 * U32 * np.abs(ref).max(), what)


# ---- graphs and streams --------------------------------------------------------------------

def _sequence(hm, torch, M, seed):
    """All operators once on one set of buffers; returns (inputs, outputs, call)."""
    k, E, H = 4, 16, 136
    c = LoraCase(torch, M, 3, H, 72, 16, "mixed", seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    t = {"lg": rand(torch, seed, M, E), "aid": c.ids, "x": c.x, "dyr": rand(torch, seed + 1, M, H, dtype="bfloat16"),
         "ids": torch.zeros(M, k, **i32), "w": torch.zeros(M, k, device="cuda"),
         "rows": torch.zeros(M * k, H, dtype=torch.bfloat16, device="cuda"), "srt": torch.zeros(M * k, **i32),
         "sr": torch.zeros(M, k, **i32), "off": torch.zeros(E + 1, **i32), "u": torch.zeros_like(c.x),
         "dx0": torch.zeros_like(c.x), "dr": torch.zeros(M * k, H, dtype=torch.bfloat16, device="cuda"),
         "dw": torch.zeros(M, k, device="cuda"), "dl": torch.zeros(M, E, device="cuda"),
         "y": torch.zeros(M, 72, dtype=torch.bfloat16, device="cuda"), "z": torch.zeros(M, 16, device="cuda"),
         "dx": torch.zeros_like(c.x), "dA": torch.zeros(3, 16, H, device="cuda"), "dB": torch.zeros(3, 72, 16, device="cuda")}
    ws = c.scratch(hm, torch)
    pw = torch.empty(max(hm.moe_permute_scratch_bytes(M, k, E), 256), dtype=torch.uint8, device="cuda")

    def call(stream=None):
        kw = {"stream": stream}
        hm.moe_route(t["lg"], k, t["ids"], t["w"], **kw)
        hm.moe_permute(t["x"], t["ids"], E, t["rows"], t["srt"], t["sr"], t["off"], pw, **kw)
        hm.moe_unpermute(t["rows"], t["sr"], t["w"], t["u"], **kw)
        hm.moe_unpermute_backward(t["dyr"], t["rows"], t["sr"], t["w"], t["dr"], t["dw"], **kw)
        hm.moe_permute_backward(t["dr"], t["sr"], t["dx0"], **kw)
        hm.moe_route_backward(t["ids"], t["w"], t["dw"], t["dl"], **kw)
        hm.moe_lora(t["x"], c.ids, c.A, c.B, c.scale, c.base, t["y"], t["z"], ws[0], **kw)
        hm.moe_lora_backward(c.dy, t["x"], t["z"], c.ids, c.A, c.B, c.scale, t["dx0"], t["dx"], t["dA"], t["dB"],
                             ws[1], **kw)

    outs = [n for n in t if n not in ("lg", "aid", "x", "dyr")]
    return t, outs, call


@pytest.mark.parametrize("M", [6, 200, 700, 1400, 2500])
def test_graph_replays(hm, M):
    """A captured run of every operator, replayed on new inputs with eager work between."""
    torch = torch_mod()
    t, outs, call = _sequence(hm, torch, M, 11)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for i in range(4):
        t["lg"].copy_(rand(torch, 100 + i, *t["lg"].shape))
        t["x"].copy_(rand(torch, 200 + i, *t["x"].shape, dtype="bfloat16"))
        t["aid"].copy_(to_dev(lora_ids(M, 3, ("mixed", "one", "none", "runs")[i], i)))
        call()
        torch.cuda.synchronize()
        eager = {n: t[n].clone() for n in outs}
        for n in outs:
            t[n].zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for n in outs:
            assert torch.equal(t[n], eager[n]), f"replay {i}: {n}"


def test_graphs_share_scratch(hm):
    """Captured calls of different sizes on one scratch buffer, replayed in turn on one stream:
    nothing of one call's scratch reaches the next."""
    torch = torch_mod()
    cases = [LoraCase(torch, M, G, 136, 200, r, "mixed", s)
             for s, (M, G, r) in enumerate([(2500, 5, 24), (7, 3, 16), (300, 9, 64), (1100, 300, 8)])]
    ws = torch.empty(max(t.numel() for c in cases for t in c.scratch(hm, torch)), device="cuda")
    runs = []
    for c in cases:
        y, z = torch.empty_like(c.base), torch.empty(c.M, c.r, device="cuda")
        dx, dA, dB = torch.empty_like(c.dbase), torch.empty_like(c.A, dtype=torch.float32), torch.empty_like(c.B, dtype=torch.float32)

        def call(c=c, y=y, z=z, dx=dx, dA=dA, dB=dB):
            hm.moe_lora(c.x, c.ids, c.A, c.B, c.scale, c.base, y, z, ws)
            hm.moe_lora_backward(c.dy, c.x, z, c.ids, c.A, c.B, c.scale, c.dbase, dx, dA, dB, ws)

        call()
        torch.cuda.synchronize()
        outs = (y, z, dx, dA, dB)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        runs.append((g, call, outs, [t.clone() for t in outs]))
    for i in range(3):
        for g, call, outs, _ in runs:
            for t in outs:
                t.zero_()
            ws.fill_(float("nan"))
            g.replay() if i != 1 else call()
        torch.cuda.synchronize()
        for _, _, outs, want in runs:
            assert all(torch.equal(t, w) for t, w in zip(outs, want)), i


@pytest.mark.parametrize("M", [30, 1400])
def test_two_streams_at_once(hm, M):
    """Calls on two streams with buffers of their own do not disturb each other."""
    torch = torch_mod()
    runs = [_sequence(hm, torch, M, s) for s in (21, 22)]
    want = []
    for t, outs, call in runs:
        call()
        torch.cuda.synchronize()
        want.append({n: t[n].clone() for n in outs})
        for n in outs:
            t[n].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(3):
        for s, (t, outs, call) in zip(streams, runs):
            call(s.cuda_stream)
    torch.cuda.synchronize()
    for (t, outs, _), w in zip(runs, want):
        for n in outs:
            assert torch.equal(t[n], w[n]), n


def test_far_rows_pass_32_bits(hm):
    """Row offsets past 2^31 elements: a wide row stride."""
    torch = torch_mod()
    M, k, E, H = 40, 4, 8, 64
    stride = 1 << 24                                       # 160 rows x 2^24 = 2.7e9 elements
    ids = ids_of(M, k, E, "any")
    x = rand(torch, 1, M, H, dtype="bfloat16")
    wide = torch.empty(M * k * stride, dtype=torch.bfloat16, device="cuda").view(M * k, stride)[:, :H]
    rows, _, sr, _ = run_permute(hm, torch, x, ids, E, wide)
    ix = R.permute_index(ids, E)
    np.testing.assert_array_equal(f64(rows), R.permute(f64(x), ix, np.zeros((M * k, H))))
    w, dy = rand(torch, 2, M, k), rand(torch, 3, M, H, dtype="bfloat16")
    got = [torch.empty(M, H, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    hm.moe_unpermute(rows, sr, w, got[0])
    hm.moe_unpermute(rows.contiguous(), sr, w, got[1])
    assert torch.equal(got[0], got[1])
    dw = [torch.empty(M, k, device="cuda") for _ in range(2)]
    dr = torch.empty(M * k, H, dtype=torch.bfloat16, device="cuda")
    hm.moe_unpermute_backward(dy, rows.contiguous(), sr, w, dr, dw[0])
    hm.moe_unpermute_backward(dy, rows, sr, w, rows_out := wide.clone().contiguous(), dw[1])
    torch.cuda.synchronize()
    assert torch.equal(dw[0], dw[1]) and torch.equal(rows_out, dr)
    c = LoraCase(torch, M * k, 3, H, 72, 16, "mixed")
    c.x = rows.contiguous()
    y, z = c.forward(hm, torch)
    c.x = rows
    y1, z1 = c.forward(hm, torch)
    assert torch.equal(y, y1) and torch.equal(z, z1)
