"""Helpers of the tests of the 4-bit matrices: random packed matrices on the host and the GPU, and
the bounds their results have to keep."""
from __future__ import annotations

import numpy as np

FORMATS = [("nvfp4", 0, False), ("mxfp4", 0, False), ("int4", 32, True), ("int4", 32, False),
           ("int4", 64, True), ("int4", 128, False), ("int4", 128, True)]
IDS = [f + (str(g) if g else "") + ("z" if z else "") for f, g, z in FORMATS]
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}   # relative to the value
# fp32's, of one operation
STEP32 = 2.0 ** -24


def torch_dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16}[name]


def rounded(a, dtype):
    """fp64 values of `a` rounded to the 16-bit type, and the tensor on the GPU when there is one."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch_dtype(dtype))
    return t.double().numpy(), t


def packed(rng, shape, fmt, group=0, zero=False, dtype="bf16", spread=2):
    """A random packed matrix [..., N, K] of entries near K^-1/2; `spread`: scales lie within
    2^+-spread."""
    *lead, K = shape
    std = K ** -0.5
    w = {"fmt": fmt, "q": rng.integers(0, 256, (*lead, K // 2), dtype=np.uint8), "z": None, "g": None,
         "group": group}
    if fmt == "nvfp4":
        w["s"] = rng.integers(0x6F - 8 * spread, 0x6F + 8 * spread, (*lead, K // 16), dtype=np.uint8)
        n = lead[0] if len(lead) == 2 else 1
        w["g"] = (rng.uniform(0.8, 1.2, n) * std / 64).astype(np.float32)
    elif fmt == "mxfp4":
        e = 125 + int(np.round(np.log2(std)))
        w["s"] = rng.integers(e - spread, e + spread + 1, (*lead, K // 32), dtype=np.uint8)
    else:
        s = std * 0.25 * 2.0 ** rng.uniform(-spread, spread, (*lead, K // group))
        w["s"], w["s_t"] = rounded(s, dtype)
        if zero:
            w["z"] = rng.integers(0, 16, (*lead, K // group), dtype=np.uint8)
    return w


def upload(w, device="cuda"):
    import torch

    import weight_only_quantized_moe_amd as hm
    code = {"nvfp4": hm.WEIGHT_NVFP4, "mxfp4": hm.WEIGHT_MXFP4, "int4": hm.WEIGHT_INT4}[w["fmt"]]

    def dev(a):
        return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(device)
    s = w["s_t"].contiguous().to(device) if w["fmt"] == "int4" else dev(w["s"])
    return hm.PackedMatrix(code, dev(w["q"]), s, dev(w["z"]), dev(w["g"]), w["group"])


def offset_values(w, W):
    """What enters the sums for each |weight|: INT4 codes come as 16 + q against 16 + z."""
    if w["fmt"] != "int4":
        return np.abs(W)
    return 62.0 * np.repeat(np.abs(w["s"]), w["group"], -1)


def check(got, ref, sums, terms, dtype, weight_step=0.0, weight_rms=None, what=""):
    """|got - ref| within the rounding of the result, `terms` fp32 roundings of the sum of absolute
    values `sums`, and a rounding of each weight by weight_step of it; where weights are rounded,
    also by rms: their errors are independent, at most weight_rms each."""
    got = got.double().cpu().numpy() if hasattr(got, "cpu") else got
    assert got.shape == ref.shape
    half = HALF_STEP[dtype] if dtype else 0.0
    tiny = 2.0 ** -25 if dtype == "fp16" else 0.0     # half the smallest step of fp16
    err = np.abs(got - ref)
    bound = half * (np.abs(ref) + (terms * STEP32 + weight_step) * sums) * 1.01 + tiny \
        + (terms * STEP32 + weight_step) * sums
    bad = ~(err <= bound)
    assert not bad.any(), (what, int(bad.sum()), float((err / bound).max()), np.argwhere(bad)[:3].tolist())
    if weight_rms is not None and ref.size >= 1000:
        rms = np.sqrt((err ** 2).mean())
        # the result's rounding alone: half a step at most
        lim = np.sqrt(((half * ref) ** 2).mean() + weight_rms ** 2) * 1.1 + terms * STEP32 * np.sqrt((sums ** 2).mean())
        assert rms <= lim, (what, rms, lim)
