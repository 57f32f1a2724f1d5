"""moe_tokens past the widths whose tokens a wave keeps in registers, and with infinities in a token."""
import numpy as np
import pytest

from packed_testlib import FORMATS, packed, upload
from test_gpu_tokens import case, hm  # noqa: F401

pytestmark = pytest.mark.gpu


# the last widths of the one kernel and the first of the other, whole pairs of 256 columns and not
@pytest.mark.parametrize("H", [4096, 4128, 6144, 6400, 7168, 8192, 8224])
def test_wide_layers(hm, H):  # noqa: F811
    rng = np.random.default_rng(H)
    for fmt, M in ((FORMATS[0], 3), (FORMATS[1], 16), (FORMATS[2], 1), (FORMATS[5], 9)):
        step = max(fmt[1], 32)
        case(hm, rng, fmt, "bf16", M, 5, -(-H // step) * step, 128, 2, S=128)


@pytest.mark.parametrize("fmt", [FORMATS[0], FORMATS[1], FORMATS[4]], ids=["nvfp4", "mxfp4", "int4"])
def test_an_infinite_token_stays_alone(hm, fmt):  # noqa: F811
    import torch
    rng = np.random.default_rng(12)
    E, H, I, k, M, S = 10, 256, 256, 3, 12, 256
    w13, w2 = (upload(packed(rng, s, *fmt)) for s in ((E, 2 * I, H), (E, H, I)))
    shared = (*(upload(packed(rng, s, *fmt)) for s in ((2 * S, H), (H, S))), None)
    router = torch.randn(E, H, device="cuda").bfloat16()
    x = torch.randn(M, H, device="cuda").bfloat16()
    ws = torch.empty(hm.moe_tokens_scratch_bytes(M, E, H, I, k, S), dtype=torch.uint8, device="cuda")
    want, y = torch.empty_like(x), torch.empty_like(x)
    hm.moe_tokens(x, router, w13, w2, k, want, shared=shared, scratch=ws)
    x[2, 5], x[7, 0] = float("inf"), float("-inf")
    hm.moe_tokens(x, router, w13, w2, k, y, shared=shared, scratch=ws)
    assert not torch.isfinite(y[[2, 7]]).any()
    keep = [m for m in range(M) if m not in (2, 7)]
    assert torch.equal(y[keep], want[keep])
    # and the next call with finite tokens is as the first
    x[2, 5] = x[7, 0] = 1.0
    again = torch.empty_like(x)
    hm.moe_tokens(x, router, w13, w2, k, y, shared=shared, scratch=ws)
    hm.moe_tokens(x, router, w13, w2, k, again, shared=shared, scratch=torch.zeros_like(ws))
    assert torch.isfinite(y).all() and torch.equal(y, again)
