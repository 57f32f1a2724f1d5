"""The operators on 4-bit matrices without a GPU: refusals of the C ABI and the binding, scratch
planners, and the oracle's gradient against differences. Nothing here launches a kernel."""
import ctypes
import os
import re

import numpy as np
import pytest

import weight_only_quantized_moe_amd as hm
from oracle import packed as P
from packed_testlib import FORMATS, IDS, packed

OK, INVALID, UNSUPPORTED, ALIGN, CAPACITY, SCRATCH, HIP = range(7)
A = 1 << 40          # never dereferenced: every call below fails before any launch


def _linear(back, M=4, K=128, N=48, dtype=0, x=A, xs=None, fmt=2, group=64, q=3 * A, s=3 * A, z=None, g=None,
            base=None, bs=0, y=2 * A, ys=None, ws=A, nb=1 << 40, w=True):
    n_in, n_out = (N, K) if back else (K, N)
    m = hm.Packed(fmt, group, q, s, z, g)
    f = hm.load_library().moe_linear_backward if back else hm.load_library().moe_linear
    return f(x, n_in if xs is None else xs, ctypes.byref(m) if w else None, M, K, N, dtype, base, bs, y,
             n_out if ys is None else ys, ws, nb, None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw,status", [
    ({"M": 0}, OK), ({"M": -1}, INVALID), ({"K": 0}, INVALID), ({"N": 0}, INVALID), ({"w": False}, INVALID),
    ({"dtype": 2}, INVALID), ({"dtype": -1}, INVALID), ({"fmt": 3}, INVALID), ({"fmt": -1}, INVALID),
    ({"group": 16}, INVALID), ({"group": 0}, INVALID), ({"K": 96}, UNSUPPORTED), ({"K": 40, "fmt": 1}, UNSUPPORTED),
    ({"K": 160, "group": 128}, UNSUPPORTED), ({"M": (1 << 22) + 1}, UNSUPPORTED),
    ({"K": (1 << 20) + 64}, UNSUPPORTED), ({"N": (1 << 20) + 1}, UNSUPPORTED),
    ({"xs": 20}, INVALID), ({"ys": 20}, INVALID), ({"xs": -128}, INVALID), ({"xs": 1 << 41}, UNSUPPORTED),
    ({"base": 5 * A, "bs": 20}, INVALID), ({"base": 2 * A, "bs": 0}, INVALID), ({"base": 2 * A, "bs": 512}, INVALID),
    ({"base": 5 * A + 1, "bs": 128}, ALIGN),
    ({"x": None}, ALIGN), ({"x": A + 1}, ALIGN), ({"y": None}, ALIGN), ({"y": A + 1}, ALIGN),
    ({"q": None}, ALIGN), ({"q": A + 8}, ALIGN), ({"s": None}, ALIGN), ({"s": A + 2}, ALIGN), ({"z": A + 1}, ALIGN),
    ({"fmt": 0, "g": None}, ALIGN), ({"fmt": 0, "g": A + 2}, ALIGN),
    ({"y": A, "x": A}, INVALID), ({"y": 3 * A}, INVALID),
    ({"M": 5000, "nb": 0}, SCRATCH), ({"M": 5000, "ws": None}, ALIGN), ({"M": 5000, "ws": A + 16}, ALIGN),
])
def test_linear_refusals(back, kw, status):
    assert _linear(back, **kw) == status
    assert status == OK or hm.moe_last_error()


def test_few_rows_need_no_scratch():
    f, b = hm.moe_linear_scratch_bytes(1, 2048, 1536)
    assert f == 0 and b >= 0


def test_scratch_never_shrinks():
    for K, N in ((32, 1), (2048, 1536), (6144, 100001), (1 << 20, 8)):
        last = (0, 0)
        for M in (0, 1, 16, 17, 64, 65, 128, 1000, 4096, 1 << 22):
            now = hm.moe_linear_scratch_bytes(M, K, N)
            assert now[0] >= last[0] and now[1] >= last[1]
            last = now
    with pytest.raises(hm.HmoeError):
        hm.moe_linear_scratch_bytes(1, 33, 4)
    with pytest.raises(hm.HmoeError):
        hm.moe_linear_scratch_bytes(-1, 32, 4)


def _tokens(M=4, E=8, H=128, I=64, k=2, S=64, dtype=0, fmt=2, group=64, router=3 * A, gate=None, x=A, xs=None,
            base=None, bs=0, y=2 * A, ys=None, ids=None, w=None, ws=A, nb=1 << 40, layer=True, **mats):
    def m(name):
        return hm.Packed(*mats.get(name, (fmt, group, 4 * A, 4 * A, None, 4 * A)))
    d = hm.TokensDesc(E, H, I, k, S, dtype, router, gate, m("w13"), m("w2"), m("s13"), m("s2"))
    return hm.load_library().moe_tokens(ctypes.byref(d) if layer else None, x, H if xs is None else xs, M, base, bs,
                                        y, H if ys is None else ys, ids, w, ws, nb, None)


@pytest.mark.parametrize("kw,status", [
    ({"M": 0}, OK), ({"M": -1}, INVALID), ({"M": 17}, CAPACITY), ({"layer": False}, INVALID),
    ({"E": 0}, INVALID), ({"E": 1025}, INVALID), ({"k": 0}, INVALID), ({"k": 9}, INVALID), ({"E": 64, "k": 17}, INVALID),
    ({"H": 0}, INVALID), ({"I": 0}, INVALID), ({"S": -32}, INVALID), ({"H": 96}, UNSUPPORTED), ({"I": 32}, UNSUPPORTED),
    ({"S": 16}, UNSUPPORTED), ({"S": 96}, UNSUPPORTED), ({"H": (1 << 20) + 64}, UNSUPPORTED),
    ({"dtype": 2}, INVALID), ({"fmt": 5}, INVALID), ({"group": 8}, INVALID),
    ({"w2": (2, 32, 4 * A, 4 * A, None, None)}, INVALID), ({"s13": (1, 0, 4 * A, 4 * A, None, None)}, INVALID),
    ({"s2": (2, 64, None, 4 * A, None, None)}, ALIGN), ({"w13": (2, 64, 4 * A, 4 * A + 4, None, None)}, ALIGN),
    ({"router": None}, ALIGN), ({"router": A + 2}, ALIGN), ({"gate": A + 2}, ALIGN),
    ({"x": None}, ALIGN), ({"y": A + 1}, ALIGN), ({"xs": 100}, INVALID), ({"ys": 100}, INVALID),
    ({"base": 5 * A, "bs": 64}, INVALID), ({"base": 2 * A, "bs": 0}, INVALID),
    ({"ids": A + 4}, ALIGN), ({"w": A + 4}, ALIGN), ({"nb": 64}, SCRATCH), ({"ws": None}, ALIGN),
    ({"y": A}, INVALID), ({"y": 4 * A}, INVALID), ({"ids": 2 * A}, INVALID), ({"ids": 5 * A, "w": 5 * A}, INVALID),
])
def test_tokens_refusals(kw, status):
    assert _tokens(**kw) == status
    assert status == OK or hm.moe_last_error()


def test_without_a_shared_expert_its_matrices_are_not_looked_at():
    none = (9, 9, None, None, None, None)
    assert _tokens(S=0, s13=none, s2=none, M=0) == OK
    assert _tokens(S=0, s13=none, s2=none, nb=0) == SCRATCH


def test_tokens_scratch():
    sizes = [hm.moe_tokens_scratch_bytes(M, 128, 2048, 768, 8, 768) for M in range(17)]
    assert sizes == sorted(sizes)
    with pytest.raises(hm.HmoeError) as e:
        hm.moe_tokens_scratch_bytes(17, 128, 2048, 768, 8)
    assert e.value.status == CAPACITY


def test_binding_refusals():
    import torch
    u8, bf = torch.uint8, torch.bfloat16
    q, s4, s = torch.zeros(16, 32, dtype=u8), torch.zeros(16, 2, dtype=bf), torch.zeros(16, 2, dtype=u8)
    ok = hm.PackedMatrix(hm.WEIGHT_MXFP4, q, s)
    int4 = hm.PackedMatrix(hm.WEIGHT_INT4, q, s4, group=32)
    for bad in (lambda: hm.PackedMatrix(7, q, s), lambda: hm.PackedMatrix(hm.WEIGHT_MXFP4, q, s4),
                lambda: hm.PackedMatrix(hm.WEIGHT_MXFP4, q[:, :16], s), lambda: hm.PackedMatrix(hm.WEIGHT_MXFP4, q.int(), s),
                lambda: hm.PackedMatrix(hm.WEIGHT_MXFP4, q, s[:, :1]), lambda: hm.PackedMatrix(hm.WEIGHT_MXFP4, q[0], s),
                lambda: hm.PackedMatrix(hm.WEIGHT_INT4, q, s4, group=16), lambda: hm.PackedMatrix(hm.WEIGHT_INT4, q, s, group=32),
                lambda: hm.PackedMatrix(hm.WEIGHT_INT4, q, s4, z=s4, group=32),
                lambda: hm.PackedMatrix(hm.WEIGHT_NVFP4, q, torch.zeros(16, 4, dtype=u8)),
                lambda: hm.PackedMatrix(hm.WEIGHT_NVFP4, q, torch.zeros(16, 4, dtype=u8), g=torch.zeros(2)),
                lambda: hm.PackedMatrix(hm.WEIGHT_MXFP4, q[:, :8].contiguous(), s[:, :1].contiguous())):
        with pytest.raises(ValueError):
            bad()
    x, y = torch.zeros(3, 64, dtype=bf), torch.zeros(3, 16, dtype=bf)
    for args in ((x.float(), ok, y.float()), (x.half(), int4, y.half()), (x[:, :32], ok, y), (x, ok, y[:, :8]),
                 (x, ok, y.half()), (x, ok, y, y[:2]), (x.t(), ok, y)):
        with pytest.raises(ValueError):
            hm.moe_linear(*args)
    with pytest.raises(ValueError):
        hm.moe_linear_backward(y, ok, x[:, :32])
    with pytest.raises(ValueError, match="GPU"):
        hm.moe_linear(x, ok, y)                          # not on a GPU
    w13 = hm.PackedMatrix(hm.WEIGHT_MXFP4, torch.zeros(4, 64, 32, dtype=u8), torch.zeros(4, 64, 2, dtype=u8))
    w2 = hm.PackedMatrix(hm.WEIGHT_MXFP4, torch.zeros(4, 64, 16, dtype=u8), torch.zeros(4, 64, 1, dtype=u8))
    router = torch.zeros(4, 64, dtype=bf)
    with pytest.raises(ValueError):
        hm.moe_linear(x, w13, x)
    for args in ((x, router, w2, w13, 2, x), (x, router[:3], w13, w2, 2, x), (x, router.half(), w13, w2, 2, x),
                 (x, router, w13, ok, 2, x), (x, router, w13, w2, 2, y), (x, router, w13, w2, 2, x, None, (w13, w2, None))):
        with pytest.raises(ValueError):
            hm.moe_tokens(*args)
    with pytest.raises(ValueError, match="GPU"):
        hm.moe_tokens(x, router, w13, w2, 2, torch.zeros_like(x))


@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
def test_oracle_gradient(fmt):
    rng = np.random.default_rng(0)
    w = packed(rng, (24, 128), *fmt)
    W = P.values(w)
    assert W.shape == (24, 128) and np.isfinite(W).all() and 0.2 < W.std() * 128 ** 0.5 < 40
    x, dy = rng.standard_normal((3, 128)), rng.standard_normal((3, 24))
    dx = P.linear_backward(dy, W)
    for i in range(5):
        e = rng.standard_normal(x.shape)
        lhs = (dy * (P.linear(x + e, W) - P.linear(x - e, W))).sum()
        assert abs(lhs - 2 * (dx * e).sum()) <= 1e-9 * np.abs(dx).sum()


def test_oracle_codes():
    """Low nibble first; the code, its zero point and its scale by hand."""
    w = {"fmt": "int4", "q": np.array([[0x1F] + [0x88] * 15], np.uint8), "s": np.array([[0.5]]),
         "z": np.array([[0xF3]], np.uint8), "g": None, "group": 32}
    v = P.values(w)[0]
    assert v[0] == (15 - 3) * 0.5 and v[1] == (1 - 3) * 0.5 and (v[2:] == 2.5).all()
    mx = {"fmt": "mxfp4", "q": np.array([[0x72] + [0] * 15], np.uint8), "s": np.array([[130]], np.uint8), "z": None,
          "g": None}
    assert P.values(mx)[0, 0] == 8.0 and P.values(mx)[0, 1] == 48.0


@pytest.mark.parametrize("name", ["linear.hip", "tokens.hip", "packed.h"])
def test_atomics_count_and_mask_only(name):
    """Sums have a fixed order: read-modify-write atomics touch tickets and masks, no sums."""
    with open(os.path.join(os.path.dirname(hm.__file__), "csrc", name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    for call in re.findall(r"\b\w*atomic(?:\w*_fetch_\w+|[A-Z]\w*)\s*\([^;]*", text):
        assert re.match(r"atomicOr\(&s\.mask\[id\]|__hip_atomic_fetch_add\((p|a)\.done \+ ", call), call
