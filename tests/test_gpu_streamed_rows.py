"""The row movements past 64 MiB of rows, where rows are read and written around the caches: every
type, few and many slots, odd widths, rows inside wider matrices at odd offsets, dropped slots.

The references are float64 sums on the device; the bounds are those of a sum of n fp32 products,
(n + 1) * 2^-24 of their magnitudes, and of one rounding to the rows' type."""
import numpy as np
import pytest

from hmoe_testlib import to_dev, torch_mod
from oracle import around as R

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
HALF = {"bfloat16": 2.0 ** -8, "float16": 2.0 ** -11, "float32": U32}
FLOOR = {"bfloat16": 1e-30, "float16": 2.0 ** -25, "float32": 1e-30}
STREAMED = 64 << 20


@pytest.fixture(scope="module")
def hm():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_moe_amd as m
    m.load_library()
    return m


def _inside(torch, rows, H, dtype, pad, shift, fill):
    """[rows, H] inside [rows, H + pad]; returns (view, whole)."""
    whole = torch.full((rows, H + pad), fill, dtype=dtype, device="cuda")
    return whole[:, shift:shift + H], whole


def _untouched(whole, H, shift, fill):
    return bool((whole[:, :shift] == fill).all()) and bool((whole[:, shift + H:] == fill).all())


def _close(got, ref, bound, what):
    off = (got.double() - ref).abs() > bound
    off |= got.double().isnan()
    assert not off.any(), f"{what}: {int(off.sum())} of {off.numel()} off, first at {off.nonzero()[0].tolist()}"


@pytest.mark.parametrize("M,k,H,dtype,pad,shift", [
    (1100, 8, 2049, "float32", 0, 0), (1100, 8, 2049, "float32", 7, 3), (560, 16, 2051, "float32", 2, 1),
    (2100, 8, 2051, "bfloat16", 0, 0), (2000, 9, 2051, "bfloat16", 9, 5), (5700, 3, 2055, "bfloat16", 1, 0),
    (1100, 16, 2051, "float16", 3, 1), (2100, 8, 2050, "float16", 0, 0), (17000, 1, 2053, "float16", 5, 2),
    (40000, 4, 257, "bfloat16", 0, 0)])
def test_streamed_rows(hm, M, k, H, dtype, pad, shift):
    torch = torch_mod()
    dt = getattr(torch, dtype)
    n, E = M * k, 24
    assert n * H * torch.empty(0, dtype=dt).element_size() > STREAMED
    g = torch.Generator(device="cuda")
    g.manual_seed(M + k)
    normal = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731

    def filled(rows):
        v, whole = _inside(torch, rows, H, dt, pad, shift, 3.0)
        v.copy_(normal(rows, H))
        return v, whole

    ids = (np.random.default_rng([M, k]).integers(0, E + 6, (M, k)) - 3).astype(np.int32)    # some dropped
    ix = R.permute_index(ids, E)
    held = int(ix["off"][-1])
    x, _ = filled(M)
    rows, whole = _inside(torch, n, H, dt, pad, shift, 3.0)
    i32 = dict(dtype=torch.int32, device="cuda")
    srt, sr, off = torch.zeros(n, **i32), torch.zeros(M, k, **i32), torch.zeros(E + 1, **i32)
    ws = torch.empty(max(hm.moe_permute_scratch_bytes(M, k, E), 256), dtype=torch.uint8, device="cuda")
    hm.moe_permute(x, to_dev(ids), E, rows, srt, sr, off, ws)
    np.testing.assert_array_equal(off.cpu().numpy(), ix["off"])
    np.testing.assert_array_equal(srt.cpu().numpy(), ix["sorted"])
    np.testing.assert_array_equal(sr.cpu().numpy(), ix["slot_row"])
    assert torch.equal(rows[:held], x[srt[:held].long() // k])
    assert bool((rows[held:] == 3.0).all()) and _untouched(whole, H, shift, 3.0)

    src, _ = filled(n)
    src[held:] = float("nan")                                 # rows that no slot names
    dy, _ = filled(M)
    w = normal(M, k)
    y, dx = (_inside(torch, M, H, dt, pad, shift, 3.0) for _ in range(2))
    dr = _inside(torch, n, H, dt, pad, shift, 3.0)
    dw = torch.full((M, k), 9.0, device="cuda")
    hm.moe_unpermute(src, sr, w, y[0])
    hm.moe_permute_backward(src, sr, dx[0])
    hm.moe_unpermute_backward(dy, src, sr, w, dr[0], dw)
    zeros = lambda *s: torch.zeros(*s, dtype=torch.float64, device="cuda")  # noqa: E731
    ry, my, rx, mx = (zeros(M, H) for _ in range(4))
    rw, mw = zeros(M, k), zeros(M, k)
    half, floor = HALF[dtype], FLOOR[dtype]
    for j in range(k):
        t = (sr[:, j] >= 0).nonzero()[:, 0]
        r = sr[t, j].long()
        v, d, wj = src[r].double(), dy[t].double(), w[t, j].double()[:, None]
        ry[t] += wj * v
        my[t] += (wj * v).abs()
        rx[t] += v
        mx[t] += v.abs()
        rw[t, j] = (v * d).sum(1)
        mw[t, j] = (v * d).abs().sum(1)
        want = wj * d
        _close(dr[0][r], want, (half + 2 * U32) * want.abs() + floor, "drows")
    _close(y[0], ry, (k + 1) * U32 * my * (1 + half) + half * ry.abs() + floor, "y")
    _close(dx[0], rx, (k + 1) * U32 * mx * (1 + half) + half * rx.abs() + floor, "dx")
    _close(dw, rw, (H + 1) * U32 * mw + 1e-30, "dw")
    assert bool((dr[0][held:] == 3.0).all())
    for _, whole in (y, dx, dr):
        assert _untouched(whole, H, shift, 3.0)
