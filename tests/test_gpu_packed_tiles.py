"""The tiled product's large tiles over many blocks of the reduction axis, and outputs of several slabs; what
ran is looked up, so that a size that no longer reaches its tile does not pass for it."""
import numpy as np
import pytest

from oracle import packed as P
from packed_testlib import FORMATS, check, offset_values, packed, rounded, upload

pytestmark = pytest.mark.gpu

NV, MX, I32Z, I32, I64Z, I128 = FORMATS[:6]
MIDDLE, WIDE, LARGE = "4, 4, 2, 2, 4", "8, 4, 2, 2, 3", "8, 4, 2, 4, 4"


@pytest.fixture(scope="module")
def hm():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_moe_amd as m
    m.load_library()
    return m


def kernels_of(call):
    """Names of the kernels of a call, or none where the profiler sees none."""
    import torch
    from torch.profiler import ProfilerActivity, profile
    with profile(activities=[ProfilerActivity.CUDA]) as p:
        call()
        torch.cuda.synchronize()
    return [e.name for e in p.events() if "hmoe::" in e.name]


def run(hm, fmt, dtype, M, C, O, back, tile, slabs=1, rows=None):
    """C: the reduction axis, O: the output's columns."""
    import torch
    f, group, zero = fmt
    K, N = (O, C) if back else (C, O)
    rng = np.random.default_rng([M, C, O, back])
    w = packed(rng, (N, K), f, group, zero, dtype)
    W = P.values(w)
    x, xt = rounded(rng.standard_normal((M, C)), dtype)
    b, bt = rounded(rng.standard_normal((1, O)), dtype)
    y = torch.full((M, O), 7.0, dtype=bt.dtype, device="cuda")
    ws = torch.full((hm.moe_linear_scratch_bytes(M, K, N)[back],), 0xFF, dtype=torch.uint8, device="cuda")
    pw, xd, bd = upload(w), xt.cuda(), bt.cuda().expand(M, O)
    names = kernels_of(lambda: (hm.moe_linear_backward if back else hm.moe_linear)(xd, pw, y, bd, ws))
    products = [n for n in names if "product16_kernel" in n]
    if back and f == "int4" and zero and dtype == "bf16":
        products = products[1:]             # the zero points' own
    if names:
        assert len(products) == slabs and all(f", {tile}, " in n for n in products), names
    if rows is None:
        rows = np.unique(np.concatenate([np.arange(0, M, 7), [1, 15, 16, M - 2, M - 1]]))
    ref = (P.linear_backward if back else P.linear)(x[rows], W, b)
    S = offset_values(w, W)
    sums = np.abs(x[rows]) @ (S if back else S.T) + np.abs(b)
    check(y[torch.from_numpy(rows).cuda()], ref, sums, C + 8, dtype)
    # whole: another call gives the same bits, rows that were not looked at among them
    again = torch.empty_like(y)
    (hm.moe_linear_backward if back else hm.moe_linear)(xd, pw, again, bd, ws)
    assert torch.equal(y, again)


# odd and even counts of blocks of 32, from one to several rounds of the buffers in LDS; ragged rows and columns
@pytest.mark.parametrize("C", [32, 64, 96, 128, 160, 288, 320, 608, 640])
def test_256_by_256(hm, C):
    run(hm, NV, "bf16", 4090, C, 3001, False, LARGE)
    run(hm, MX, "fp16", 4090, C, 3008, True, LARGE)
    if C % 64 == 0:
        run(hm, I64Z, "bf16", 4090, C, 3001, False, LARGE)
        run(hm, I64Z, "fp16", 4090, C, 3001, False, LARGE)


@pytest.mark.parametrize("C", [32, 64, 96, 128, 160, 288, 320, 608, 640])
def test_256_by_128(hm, C):
    run(hm, MX, "bf16", 2000, C, 4001, False, WIDE)
    run(hm, NV, "fp16", 2000, C - 5, 4032, True, WIDE)
    run(hm, I64Z, "bf16", 2000, C + 3, 4032, True, WIDE)
    run(hm, I32, "fp16", 2000, C - 1, 4032, True, WIDE)


def test_large_layers(hm):
    """The sizes of a prefill chunk and of a fine-tuning step, some rows of each."""
    rows = np.array([0, 1, 255, 256, 2047, 3999, 4000])
    run(hm, NV, "bf16", 4001, 6144, 4096, False, LARGE, rows=rows)
    run(hm, I64Z, "bf16", 4001, 4096, 6144, True, WIDE, rows=rows)


@pytest.mark.parametrize("fmt,dtype", [(NV, "bf16"), (MX, "bf16"), (I64Z, "bf16"), (I32Z, "fp16"), (I32, "fp16")])
def test_forward_slabs(hm, fmt, dtype):
    """Two slabs of columns without shares of the reduction axis, and two with."""
    run(hm, fmt, dtype, 66, 64, 530000, False, LARGE, 2)
    run(hm, fmt, dtype, 420, 4096, 8400, False, MIDDLE, 2)


@pytest.mark.parametrize("fmt,dtype", [(NV, "bf16"), (MX, "fp16"), (I64Z, "bf16"), (I128, "fp16")])
def test_gradient_slabs(hm, fmt, dtype):
    run(hm, fmt, dtype, 140, 8400, 4224, True, MIDDLE, 2)
