"""Adapters on whole numbers, where every product and partial sum is exact in fp32: the outputs
have to be equal, at sizes that reach every form of the kernels."""
import numpy as np
import pytest

from hmoe_testlib import to_dev, torch_mod

pytestmark = pytest.mark.gpu

BITS = 20   # of the small operand: more than two bf16 parts hold (16, 17 with the signs)


@pytest.fixture(scope="module")
def hm():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_moe_amd as m
    m.load_library()
    return m


def _bits(M, C, seed):
    """[M, C] zeros and ones in the first BITS columns, and the numbers their lowest 8 make."""
    b = np.random.default_rng([seed, M]).integers(0, 2, (M, BITS))
    b[:, BITS - 1] = 1                                    # all numbers need the full width
    x = np.zeros((M, C), np.float32)
    x[:, :BITS] = b
    return x, b[:, :8] @ (1 << np.arange(8)), b @ (1 << np.arange(BITS))


def _reader(G, r, C):
    """[G, r, C]: an even rank reads the whole number, the odd one after it all but its lowest 8
    bits."""
    a = np.zeros((G, r, C), np.float32)
    a[:, :, :BITS] = 2.0 ** np.arange(BITS)
    a[:, 1::2, :8] = 0
    return a


def _taker(G, C, r):
    """[G, C, r]: column c takes the difference of one pair of ranks: the lowest 8 bits."""
    b = np.zeros((G, C, r), np.float32)
    c = np.arange(C)
    b[:, c, 2 * (c % (r // 2))] = 1
    b[:, c, 2 * (c % (r // 2)) + 1] = -1
    return b


# rows: 3 and 100 find their tiles by comparing, 300 and 1500 by counting, 2500 and more by a sort;
# up to 1024 one launch where the rank is at most 64; tiles of 64 rows from 3000 rows on. Ranks: on
# both sides of 16 and of each 32
@pytest.mark.parametrize("M,G", [(3, 2), (100, 3), (300, 5), (1500, 60), (1500, 2), (2500, 100), (3200, 3)])
@pytest.mark.parametrize("r", [8, 16, 24, 32, 40, 64, 72, 96, 104, 128])
def test_small_operand_keeps_its_bits(hm, M, G, r):
    """y = base + s B z and dx = dbase + s A^T dz with z and dz of 20 bits, of which the result
    holds the lowest 8 only: rounding z or dz to fewer bits would change it."""
    torch = torch_mod()
    C, bf = 264, torch.bfloat16
    x, low, whole = _bits(M, C, r)
    ids = np.random.default_rng([M, r]).integers(-1, G, M).astype(np.int32)
    scale = (2.0 ** (np.arange(G) % 5 - 2)).astype(np.float32)
    own = np.where(ids >= 0, scale[ids], 0.0)
    want = np.repeat((own * low)[:, None], C, 1)          # 8 bits times a power of two: exact in bf16
    f, b = hm.moe_lora_scratch_bytes(M, G, C, C, r)
    ws = torch.empty(max(f, b, 256), dtype=torch.uint8, device="cuda")
    reader, taker = (to_dev(v).to(bf) for v in (_reader(G, r, C), _taker(G, C, r)))
    xd, idd, sd = to_dev(x).to(bf), to_dev(ids), to_dev(scale)
    y, z = torch.empty(M, C, dtype=bf, device="cuda"), torch.empty(M, r, device="cuda")
    hm.moe_lora(xd, idd, reader, taker, sd, None, y, z, ws)
    np.testing.assert_array_equal(y.double().cpu().numpy(), want)
    np.testing.assert_array_equal(z.double().cpu().numpy()[:, 0], np.where(ids >= 0, whole, 0))
    # the gradient's chain has the same shape with B^T first and A^T second
    dx = torch.empty(M, C, dtype=bf, device="cuda")
    dA, dB = torch.empty(G, r, C, device="cuda"), torch.empty(G, C, r, device="cuda")
    hm.moe_lora_backward(xd, xd.clone(), z, idd, taker.transpose(1, 2).contiguous(),
                         reader.transpose(1, 2).contiguous(), sd, None, dx, dA, dB, ws)
    np.testing.assert_array_equal(dx.double().cpu().numpy(), want)


@pytest.mark.parametrize("M,r", [(5, 8), (5, 64), (300, 128), (3000, 32)])
def test_small_operand_at_the_end_of_fp32(hm, M, r):
    """A finite z above bf16's largest value stays finite in all products."""
    torch = torch_mod()
    C, bf = 64, torch.bfloat16
    x = torch.zeros(M, C, dtype=bf, device="cuda")
    x[:, :2] = 1
    a = torch.zeros(1, r, C, device="cuda")
    a[:, 0, 0], a[:, 0, 1] = 2.0 ** 127 * (2 - 2.0 ** -7), 2.0 ** 119      # z = 2^128 - 2^119
    b = torch.zeros(1, C, r, device="cuda")
    b[:, :, 0] = 2.0 ** -120
    ids, one = torch.zeros(M, dtype=torch.int32, device="cuda"), torch.ones(1, device="cuda")
    f, n = hm.moe_lora_scratch_bytes(M, 1, C, C, r)
    ws = torch.empty(max(f, n, 256), dtype=torch.uint8, device="cuda")
    y, z = torch.empty(M, C, dtype=bf, device="cuda"), torch.empty(M, r, device="cuda")
    hm.moe_lora(x, ids, a.to(bf), b.to(bf), one, None, y, z, ws)
    assert bool((z[:, 0].double() == 2.0 ** 128 - 2.0 ** 119).all()) and not z[:, 1:].any()
    assert bool((y == 256.0).all())                      # 255.5, half way between 255 and 256
    dy = torch.zeros(M, C, dtype=bf, device="cuda")
    dy[0], dy[-1] = 2.0 ** -120, -2.0 ** -121
    dx, dA, dB = torch.empty_like(x), torch.empty_like(a), torch.empty_like(b)
    hm.moe_lora_backward(dy, x, z, ids, a.to(bf), b.to(bf), one, None, dx, dA, dB, ws)
    assert bool((dB[0, :, 0] == 127.75).all()) and not dB[0, :, 1:].any()


@pytest.mark.parametrize("r", [16, 64])
def test_scratch_of_the_largest_batch(hm, r):
    """One buffer, planned for 3200 rows, and every smaller number of rows on it."""
    torch = torch_mod()
    G, C, bf = 16, 4096, torch.bfloat16
    f, b = hm.moe_lora_scratch_bytes(3200, G, C, C, r)
    fws, bws = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in (f, b))
    reader, taker = (to_dev(v).to(bf) for v in (_reader(G, r, C), _taker(G, C, r)))
    one = torch.ones(G, device="cuda")
    for M in (1, 8, 15, 16, 100, 799, 800, 1024, 1025, 2048, 2049, 3199, 3200):
        x, low, _ = _bits(M, C, r)
        ids = np.random.default_rng(M).integers(0, G, M).astype(np.int32)
        xd, idd = to_dev(x).to(bf), to_dev(ids)
        y, dx, z = torch.empty_like(xd), torch.empty_like(xd), torch.empty(M, r, device="cuda")
        dA, dB = torch.empty(G, r, C, device="cuda"), torch.empty(G, C, r, device="cuda")
        fws.fill_(255), bws.fill_(255)
        hm.moe_lora(xd, idd, reader, taker, one, None, y, z, fws)
        hm.moe_lora_backward(xd, xd.clone(), z, idd, taker.transpose(1, 2).contiguous(),
                             reader.transpose(1, 2).contiguous(), one, None, dx, dA, dB, bws)
        for t in (y, dx):
            np.testing.assert_array_equal(t.double().cpu().numpy(), np.repeat(low[:, None], C, 1), str(M))


@pytest.mark.parametrize("M,r", [(40, 8), (40, 64), (700, 24), (3200, 16), (3200, 128)])
@pytest.mark.parametrize("bad", ["inf", "nan"])
def test_non_finite_values_stay_in_their_adapter(hm, M, r, bad):
    """One infinite x reaches its adapter's column of dA, one infinite dy its adapter's column of
    dB, its dA and its row of dx; every other value keeps its bits."""
    torch = torch_mod()
    G, K, N, bf = 3, 136, 200, torch.bfloat16
    g = torch.Generator().manual_seed(M + r)
    n = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    x, dy, A, B = n(M, K).to(bf), n(M, N).to(bf), n(G, r, K).to(bf), n(G, N, r).to(bf)
    z, scale = n(M, r), n(G)
    ids = torch.randint(-1, G, (M,), generator=g, dtype=torch.int32)
    ids[7] = 1
    at = 7
    if M > 40:
        at = int((ids == 1).nonzero()[-1])               # the adapter's last row, which fills its last step
    ids = ids.cuda()
    ws = torch.empty(hm.moe_lora_scratch_bytes(M, G, K, N, r)[1], dtype=torch.uint8, device="cuda")

    def run(x, dy):
        out = (torch.empty(M, K, dtype=bf, device="cuda"), torch.empty(G, r, K, device="cuda"),
               torch.empty(G, N, r, device="cuda"))
        hm.moe_lora_backward(dy, x, z, ids, A, B, scale, None, *out, ws)
        return out
    dx, dA, dB = run(x, dy)
    xb = x.clone()
    xb[at, 33] = float(bad)
    dx1, dA1, dB1 = run(xb, dy)
    assert torch.equal(dx1, dx) and torch.equal(dB1, dB)
    assert not dA1[1, :, 33].isfinite().any()
    dA1[1, :, 33] = dA[1, :, 33]
    assert torch.equal(dA1, dA)
    db = dy.clone()
    db[at, 77] = float(bad)
    dx2, dA2, dB2 = run(x, db)
    assert not dB2[1, 77].isfinite().any() and not dx2[at].isfinite().any() and not dA2[1].isfinite().any()
    dB2[1, 77], dx2[at], dA2[1] = dB[1, 77], dx[at], dA[1]
    assert torch.equal(dx2, dx) and torch.equal(dA2, dA) and torch.equal(dB2, dB)
