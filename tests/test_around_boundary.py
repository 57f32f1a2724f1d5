"""The operators around the experts without a GPU: what their entry points refuse
(status codes and messages through the C ABI, shape and type errors of the Python
binding), their scratch planners, and the oracle's gradients against differences.
Nothing here launches a kernel."""
import ctypes

import numpy as np
import pytest

import weight_only_quantized_moe_amd as hm
from oracle import around as R

OK, INVALID, UNSUPPORTED, ALIGN, CAPACITY, SCRATCH, HIP = range(7)
A = 1 << 40          # never dereferenced: every call below fails before any launch


def _permute(M=4, k=2, E=8, H=16, dtype=0, x=A, xs=16, ids=A, rows=2 * A, rs=16, srt=A, sr=A, off=A,
             ws=None, nb=0):
    return hm.load_library().moe_permute(x, xs, ids, M, k, E, H, dtype, rows, rs, srt, sr, off, ws, nb,
                                         None)


@pytest.mark.parametrize("kw,status", [
    ({"M": -1}, INVALID), ({"k": 0}, INVALID), ({"k": 17}, INVALID), ({"E": 0}, INVALID),
    ({"E": 1025}, INVALID), ({"H": 0}, INVALID), ({"dtype": 3}, INVALID), ({"dtype": -1}, INVALID),
    ({"xs": 15}, INVALID), ({"rs": 15}, INVALID), ({"xs": -16}, INVALID),
    ({"M": (1 << 24) // 2 + 1}, UNSUPPORTED),
    ({"M": 1 << 22, "H": 8192, "xs": 8192, "rs": 8192}, UNSUPPORTED),
    ({"xs": 1 << 41}, UNSUPPORTED),
    ({"x": None}, ALIGN), ({"x": A + 1}, ALIGN), ({"dtype": 2, "x": A + 2}, ALIGN), ({"rows": None}, ALIGN),
    ({"ids": A + 4}, ALIGN), ({"srt": A + 8}, ALIGN), ({"sr": None}, ALIGN), ({"off": A + 4}, ALIGN),
    ({"M": 8192}, SCRATCH), ({"M": 8192, "ws": A + 16, "nb": 1 << 30}, ALIGN),
    ({"M": 8192, "ws": None, "nb": 1 << 30}, ALIGN),
])
def test_permute_refusals(kw, status):
    assert _permute(**kw) == status
    assert hm.moe_last_error()


def test_row_gradients_refusals():
    lib = hm.load_library()

    def back(M=4, k=2, H=16, dt=0, d=A, ds=16, sr=A, dx=2 * A, xs=16):
        return lib.moe_permute_backward(d, ds, sr, M, k, H, dt, dx, xs, None)

    def un(M=4, k=2, H=16, dt=0, r=A, rs=16, sr=A, w=A, y=2 * A, ys=16):
        return lib.moe_unpermute(r, rs, sr, w, M, k, H, dt, y, ys, None)

    def unb(M=4, k=2, H=16, dt=0, dy=A, r=A, sr=A, w=A, dr=2 * A, dw=A, s=16):
        return lib.moe_unpermute_backward(dy, s, r, s, sr, w, M, k, H, dt, dr, s, dw, None)

    for f in (back, un, unb):
        assert f(M=0) == OK
        assert f(M=-1) == INVALID and f(k=17) == INVALID and f(H=0) == INVALID and f(dt=7) == INVALID
        assert f(sr=A + 4) == ALIGN and f(M=1 << 24) == UNSUPPORTED
    assert back(ds=8) == INVALID and back(dx=None) == ALIGN and back(d=A + 1) == ALIGN
    assert un(w=None) == ALIGN and un(ys=8) == INVALID and un(r=None) == ALIGN
    assert unb(dw=A + 4) == ALIGN and unb(s=15) == INVALID and unb(dr=None) == ALIGN


def test_route_backward_refusals():
    def f(M=4, E=8, k=2, ids=A, w=A, dw=A, dl=A):
        return hm.load_library().moe_route_backward(ids, w, dw, M, E, k, dl, None)
    assert f(M=0) == OK
    for kw in ({"M": -1}, {"E": 0}, {"E": 1025}, {"k": 0}, {"k": 9}, {"E": 64, "k": 17}):
        assert f(**kw) == INVALID, kw
    for kw in ({"ids": None}, {"w": A + 4}, {"dw": None}, {"dl": A + 8}):
        assert f(**kw) == ALIGN, kw


def _lora(M=2000, G=3, K=64, N=32, r=8, x=A, xs=None, ids=A, a=A, b=A, sc=A, base=A, bs=None, y=2 * A,
          ys=None, z=None, ws=A, nb=1 << 40):
    return hm.load_library().moe_lora(x, K if xs is None else xs, ids, a, b, sc, M, G, K, N, r, base,
                                      N if bs is None else bs, y, N if ys is None else ys, z, ws, nb, None)


def _lora_bwd(M=4, G=3, K=64, N=32, r=8, dy=A, ys=None, x=A, xs=None, z=A, ids=A, a=A, b=A, sc=A, base=A,
              bs=None, dx=2 * A, dxs=None, dA=A, dB=A, ws=A, nb=1 << 40):
    return hm.load_library().moe_lora_backward(
        dy, N if ys is None else ys, x, K if xs is None else xs, z, ids, a, b, sc, M, G, K, N, r, base,
        K if bs is None else bs, dx, K if dxs is None else dxs, dA, dB, ws, nb, None)


@pytest.mark.parametrize("f", [_lora, _lora_bwd])
@pytest.mark.parametrize("kw,status", [
    ({"M": -1}, INVALID), ({"G": 0}, INVALID), ({"K": 0}, INVALID), ({"N": -8}, INVALID), ({"r": 0}, INVALID),
    ({"K": 60}, UNSUPPORTED), ({"N": 36}, UNSUPPORTED), ({"r": 12}, UNSUPPORTED), ({"r": 136}, UNSUPPORTED),
    ({"G": 2049}, UNSUPPORTED), ({"M": (1 << 22) + 1}, UNSUPPORTED), ({"K": (1 << 20) + 8}, UNSUPPORTED),
    ({"xs": 63}, INVALID), ({"bs": 31}, INVALID), ({"ys": 31}, INVALID),
    ({"x": None}, ALIGN), ({"x": A + 1}, ALIGN), ({"ids": None}, ALIGN), ({"a": A + 8}, ALIGN),
    ({"b": None}, ALIGN), ({"sc": A + 4}, ALIGN), ({"z": A + 4}, ALIGN), ({"base": A + 1}, ALIGN),
    ({"ws": None}, ALIGN), ({"ws": A + 64}, ALIGN), ({"nb": 0}, SCRATCH),
])
def test_lora_refusals(f, kw, status):
    assert f(**kw) == status
    assert hm.moe_last_error()


def test_lora_own_refusals():
    assert _lora(M=0) == OK
    assert _lora(y=None) == ALIGN
    assert _lora(base=2 * A, bs=64) == INVALID            # in place with another stride
    assert _lora_bwd(base=2 * A, bs=128) == INVALID
    assert _lora_bwd(z=None) == ALIGN and _lora_bwd(dA=None) == ALIGN and _lora_bwd(dB=A + 4) == ALIGN
    assert _lora_bwd(dx=None) == ALIGN and _lora_bwd(dxs=8) == INVALID and _lora_bwd(dy=None) == ALIGN


def test_outputs_over_inputs_are_refused():
    lib = hm.load_library()
    assert _permute(rows=A) == INVALID
    assert lib.moe_permute_backward(A, 16, A, 4, 2, 16, 0, A, 16, None) == INVALID
    assert lib.moe_unpermute(A, 16, A, A, 4, 2, 16, 0, A, 16, None) == INVALID
    for dy, r in ((2 * A, A), (A, 2 * A)):
        assert lib.moe_unpermute_backward(dy, 16, r, 16, A, A, 4, 2, 16, 0, 2 * A, 16, A, None) == INVALID
    assert _lora(y=A, base=None) == INVALID
    assert _lora_bwd(dx=A, dy=3 * A, base=None) == INVALID and _lora_bwd(dx=A, x=3 * A, base=None) == INVALID
    assert "input" in lib.moe_last_error().decode()


def test_lora_scratch_over_all_sizes():
    """Every accepted size has a finite plan, whose bytes hold what the two launches exchange."""
    r = np.random.default_rng(3)
    for _ in range(4000):
        M, K, N = (int(2 ** r.uniform(0, e)) for e in (22, 17, 17))
        G, rank = int(2 ** r.uniform(0, 11)), 8 * int(r.integers(1, 17))
        f, b = hm.moe_lora_scratch_bytes(M, G, 8 * K, 8 * N, rank)
        assert f % 256 == 0 and f < 1 << 42 and b < 1 << 45
        assert b >= 2 * M * rank * 6 + G * rank * 8 * N * 2   # gradients' fragments, B turned
        if M > 1024:
            assert f >= M * rank * 4 + M * 4                  # z's parts, the sorted rows


def test_scratch_planners():
    assert hm.moe_permute_scratch_bytes(1024, 8, 256) == 0         # one block sorts alone
    assert hm.moe_permute_scratch_bytes(4096, 8, 256) > 0
    assert hm.moe_permute_scratch_bytes(0, 1, 1) == 0
    f, b = hm.moe_lora_scratch_bytes(4096, 8, 6144, 4096, 64)
    assert f > 4096 * 4 and b > 8 * 64 * 4096 * 2
    assert hm.moe_lora_scratch_bytes(256, 48, 2048, 4096, 64)[0] == 0     # one launch for few rows
    assert _lora(nb=hm.moe_lora_scratch_bytes(2000, 3, 64, 32, 8)[0] - 1) == SCRATCH
    assert _lora_bwd(nb=hm.moe_lora_scratch_bytes(4, 3, 64, 32, 8)[1] - 1) == SCRATCH
    for args in ((-1, 1, 8, 8, 8), (1, 1, 8, 8, 0)):
        with pytest.raises(hm.HmoeError):
            hm.moe_lora_scratch_bytes(*args)
    hm.moe_lora_scratch_bytes(0, 1, 8, 8, 8)
    with pytest.raises(hm.HmoeError):
        hm.moe_permute_scratch_bytes(1, 0, 8)


def test_binding_checks_tensors():
    """The binding refuses wrong shapes, types, layouts and tensors that are not on a GPU."""
    torch = pytest.importorskip("torch")
    M, k, E, H = 4, 2, 8, 16
    i32 = torch.int32

    def permute(x=None, ids=None, rows=None, srt=None, sr=None, off=None):
        d = lambda v, o: o if v is None else v  # noqa: E731
        hm.moe_permute(d(x, torch.zeros(M, H)), d(ids, torch.zeros(M, k, dtype=i32)), E,
                       d(rows, torch.zeros(M * k, H)), d(srt, torch.zeros(M * k, dtype=i32)),
                       d(sr, torch.zeros(M, k, dtype=i32)), d(off, torch.zeros(E + 1, dtype=i32)))

    with pytest.raises(ValueError, match="one GPU"):
        permute()
    for kw in ({"x": torch.zeros(M, H, dtype=torch.float64)}, {"x": torch.zeros(M + 1, H)},
               {"x": torch.zeros(H, M).t()}, {"rows": torch.zeros(M * k, H + 1)},
               {"rows": torch.zeros(M * k, H, dtype=torch.bfloat16)}, {"ids": torch.zeros(M, k)},
               {"ids": torch.zeros(k, M, dtype=i32).t()}, {"srt": torch.zeros(M * k + 1, dtype=i32)},
               {"off": torch.zeros(E, dtype=i32)}, {"sr": torch.zeros(M * k, dtype=i32)}):
        with pytest.raises(ValueError):
            permute(**kw)
    G, r, K, N = 3, 8, 64, 32
    bf = torch.bfloat16

    def lora(x=None, ids=None, a=None, b=None, sc=None, base=None, y=None, z=None):
        d = lambda v, o: o if v is None else v  # noqa: E731
        hm.moe_lora(d(x, torch.zeros(M, K, dtype=bf)), d(ids, torch.zeros(M, dtype=i32)),
                    d(a, torch.zeros(G, r, K, dtype=bf)), d(b, torch.zeros(G, N, r, dtype=bf)),
                    d(sc, torch.zeros(G)), base, d(y, torch.zeros(M, N, dtype=bf)), z)

    with pytest.raises(ValueError, match="one GPU"):
        lora()
    for kw in ({"x": torch.zeros(M, K)}, {"a": torch.zeros(G, r, K)}, {"b": torch.zeros(G + 1, N, r, dtype=bf)},
               {"b": torch.zeros(G, r, N, dtype=bf).transpose(1, 2)}, {"ids": torch.zeros(M, dtype=torch.int64)},
               {"sc": torch.zeros(G, dtype=bf)}, {"y": torch.zeros(M, N + 8, dtype=bf)},
               {"base": torch.zeros(M, N)}, {"z": torch.zeros(M, r, dtype=bf)}):
        with pytest.raises(ValueError):
            lora(**kw)


def test_binding_checks_gradients():
    torch = pytest.importorskip("torch")
    M, k, E, H, G, r, K, N = 4, 2, 8, 16, 3, 8, 64, 32
    bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    z = torch.zeros

    def lora(**kw):
        t = dict(dy=z(M, N, dtype=bf), x=z(M, K, dtype=bf), z=z(M, r), ids=z(M, dtype=i32), A=z(G, r, K, dtype=bf),
                 B=z(G, N, r, dtype=bf), scale=z(G), dbase=None, dx=z(M, K, dtype=bf), dA=z(G, r, K), dB=z(G, N, r))
        hm.moe_lora_backward(**{**t, **kw})

    def unpermute(**kw):
        t = dict(dy=z(M, H), rows=z(M * k, H), slot_row=z(M, k, dtype=i32), topk_w=z(M, k), drows=z(M * k, H), dw=z(M, k))
        hm.moe_unpermute_backward(**{**t, **kw})

    def route(**kw):
        t = dict(topk_ids=z(M, k, dtype=i32), topk_w=z(M, k), dw=z(M, k), dlogits=z(M, E))
        hm.moe_route_backward(**{**t, **kw})

    for f in (lora, unpermute, route):
        with pytest.raises(ValueError, match="one GPU"):
            f()
    for f, kw in ((lora, {"z": None}), (lora, {"dA": z(G, r, K, dtype=bf)}), (lora, {"dB": z(G, r, N)}),
                  (lora, {"dbase": z(M, N, dtype=bf)}), (lora, {"dx": z(M, K)}), (lora, {"dy": z(K, M, dtype=bf).t()}),
                  (unpermute, {"dw": z(M, k, dtype=bf)}), (unpermute, {"drows": z(M, H)}),
                  (unpermute, {"dy": z(M, H, dtype=bf)}), (unpermute, {"slot_row": z(M, k, dtype=f32)}),
                  (route, {"dlogits": z(M, E, dtype=bf)}), (route, {"dw": z(M, k + 1)}),
                  (route, {"topk_ids": z(k, M, dtype=i32).t()})):
        with pytest.raises(ValueError):
            f(**kw)


# ---- the oracle's gradients against central differences of its forward forms ------------

def _differences(f, v, step=1e-5):
    """d f / d v by central differences, entry by entry (f: scalar, float64)."""
    g = np.zeros(v.shape)
    for i in np.ndindex(*v.shape):
        up, down = v.copy(), v.copy()
        up[i] += step
        down[i] -= step
        g[i] = (f(up) - f(down)) / (2 * step)
    return g


# every function below is at most quadratic in the entry that is moved (softmax aside, whose
# third derivative is below 1), so the difference is exact up to rounding: values of about 10
# at 2^-53 over a step of 1e-5 leave 1e-9; softmax's truncation is below 1e-10
_CLOSE = dict(rtol=1e-7, atol=1e-7)


def test_oracle_permutation_gradients():
    r = np.random.default_rng(3)
    M, k, E, H = 5, 3, 4, 6
    ids = np.stack([r.permutation(E + 2)[:k] - 1 for _ in range(M)]).astype(np.int32)   # some dropped
    ix = R.permute_index(ids, E)
    x, w, cot = r.standard_normal((M, H)), r.random((M, k)), r.standard_normal((M * k, H))
    n = ix["off"][-1]
    assert 0 < n < M * k
    zero = np.zeros((M * k, H))
    got = R.unpermute(cot, ix["slot_row"], None)
    np.testing.assert_allclose(got, _differences(lambda v: float((R.permute(v, ix, zero)[:n] * cot[:n]).sum()), x), **_CLOSE)
    rows, dy = r.standard_normal((M * k, H)), r.standard_normal((M, H))
    dr, dw = R.unpermute_backward(dy, rows, ix["slot_row"], w, zero)
    f = lambda a, b: float((R.unpermute(a, ix["slot_row"], b) * dy).sum())  # noqa: E731
    np.testing.assert_allclose(dr, _differences(lambda v: f(v, w), rows), **_CLOSE)
    np.testing.assert_allclose(dw, _differences(lambda v: f(rows, v), w), **_CLOSE)


def test_oracle_route_gradient():
    r = np.random.default_rng(4)
    M, E, k = 4, 7, 3
    lg, dw = r.standard_normal((M, E)), r.standard_normal((M, k))
    ids = np.argsort(-lg, axis=1, kind="stable")[:, :k].astype(np.int32)

    def weights(v):
        s = np.take_along_axis(v, ids, 1)
        e = np.exp(s - s.max(1, keepdims=True))
        return e / e.sum(1, keepdims=True)
    got = R.route_backward(ids, weights(lg), dw, E)
    np.testing.assert_allclose(got, _differences(lambda v: float((weights(v) * dw).sum()), lg), **_CLOSE)


def test_oracle_lora_gradients():
    r = np.random.default_rng(5)
    M, G, K, N, q = 6, 3, 5, 4, 2
    ids = np.array([0, 2, -1, 2, 0, 7], np.int32)                  # adapter 1 has no rows
    x, base, dy = r.standard_normal((M, K)), r.standard_normal((M, N)), r.standard_normal((M, N))
    a, b, sc = r.standard_normal((G, q, K)), r.standard_normal((G, N, q)), r.random(G)
    y, z = R.lora(x, ids, a, b, sc, base)
    np.testing.assert_array_equal(y[[2, 5]], base[[2, 5]])
    dx, dA, dB = R.lora_backward(dy, x, z, ids, a, b, sc, np.zeros((M, K)))
    f = lambda x, a, b: float((R.lora(x, ids, a, b, sc, base)[0] * dy).sum())  # noqa: E731
    np.testing.assert_allclose(dx, _differences(lambda v: f(v, a, b), x), **_CLOSE)
    np.testing.assert_allclose(dA, _differences(lambda v: f(x, v, b), a), **_CLOSE)
    np.testing.assert_allclose(dB, _differences(lambda v: f(x, a, v), b), **_CLOSE)
    assert not dA[1].any() and not dB[1].any()
