"""moe_tokens against float64: every format and type, one token to the most, odd widths, the shared
expert, many tokens on one expert, captured replays, and the layer's own forward beside it."""
import numpy as np
import pytest

import synth
from hmoe_testlib import run_forward, tiny_packed, to_dev_bits
from oracle import formats as F
from oracle import layer as OL
from oracle import packed as P
from packed_testlib import FORMATS, HALF_STEP, IDS, packed, rounded, upload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hm():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_moe_amd as m
    m.load_library()
    return m


def bounds(x, ref_ids, p, w13, w2, W13, W2, shared):
    """Per token and column: how far y's sum may be off before its rounding. fp32 sums of the first
    product (K + 8 roundings of what enters it) go through silu(a) b, whose slopes are at most 1.1 |b|
    and |silu(a)|; h is off by 2^-16 of its value besides (two bf16 parts, exp, reciprocal)."""
    def one(x, w, v, w_in, v_in):
        I, H = v.shape[1], w.shape[1]
        a, b = w[:I] @ x, w[I:] @ x
        ea, eb = ((w_in[:I] @ np.abs(x)) * (H + 8) * 2.0 ** -24, (w_in[I:] @ np.abs(x)) * (H + 8) * 2.0 ** -24)
        sl = a / (1 + np.exp(-a))
        eh = 1.1 * np.abs(b) * ea + np.abs(sl) * eb + np.abs(sl * b) * 2.0 ** -16
        h = np.abs(sl * b)
        return np.abs(v) @ eh + (v_in @ h) * (2 * I + 300) * 2.0 ** -24
    out = np.zeros((x.shape[0], W2.shape[1]))
    for t in range(x.shape[0]):
        for j, e in enumerate(ref_ids[t]):
            out[t] += 1.01 * p[t, j] * one(x[t], W13[e], W2[e], w13[e], w2[e])
        if shared is not None:
            out[t] += one(x[t], *shared)
    return out


def off(w, W, e=None):
    """What enters the sums of the product: INT4 codes come as 16 + q against 16 + z."""
    if w["fmt"] != "int4":
        return np.abs(W)
    return 62.0 * np.repeat(np.abs(w["s"]), w["group"], -1)


def case(hm, rng, fmt, dtype, M, E, H, I, k, S=0, gate=True, base="matrix", strided=False, logits_scale=1.0,
         same=False):
    import torch
    f, g, z = fmt
    x, xt = rounded(np.repeat(rng.standard_normal((1, H)), M, 0) if same else rng.standard_normal((M, H)), dtype)
    router, rt = rounded(rng.standard_normal((E, H)) * H ** -0.5 * logits_scale, dtype)
    w13, w2 = packed(rng, (E, 2 * I, H), f, g, z, dtype), packed(rng, (E, H, I), f, g, z, dtype)
    W13, W2 = P.values(w13), P.values(w2)
    b, bt = rounded(rng.standard_normal((1 if base == "bias" else M, H)), dtype)
    shared = ref_shared = sh = None
    if S:
        s13, s2 = packed(rng, (2 * S, H), f, g, z, dtype), packed(rng, (H, S), f, g, z, dtype)
        gv, gt = rounded(rng.standard_normal(H) * H ** -0.5, dtype)
        V13, V2 = P.values(s13), P.values(s2)
        shared = (upload(s13), upload(s2), gt.cuda() if gate else None)
        ref_shared = (V13, V2, gv if gate else None)
        sh = (V13, V2, off(s13, V13), off(s2, V2))
    ref = P.tokens(x, router, W13, W2, k, None if base is None else b, ref_shared)
    pad = 5 if strided else 0
    xd = torch.zeros(M, H + pad, dtype=xt.dtype, device="cuda")[:, :H]
    xd.copy_(xt)
    y = torch.full((M, H + pad), 7.0, dtype=xt.dtype, device="cuda")
    bd = None
    if base == "matrix":
        bd = bt.cuda()
    elif base == "bias":
        bd = bt.cuda().expand(M, H)
    elif base == "own":
        y[:, :H].copy_(bt)
        bd = y[:, :H]
    ids = torch.empty(M, k, dtype=torch.int32, device="cuda")
    tw = torch.empty(M, k, device="cuda")
    n = hm.moe_tokens_scratch_bytes(M, E, H, I, k, S)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    hm.moe_tokens(xd, rt.cuda(), upload(w13), upload(w2), k, y[:, :H], bd, shared, ids, tw, ws)
    torch.cuda.synchronize()
    assert np.array_equal(ids.cpu().numpy(), ref["ids"])
    # logits are off by (H + 8) fp32 roundings of their terms, weights by that much of themselves, twice
    dl = (np.abs(x) @ np.abs(router).T).max() * (H + 8) * 2.0 ** -24
    assert (np.abs(tw.double().cpu().numpy() - ref["w"]) <= ref["w"] * (2 * dl + 2.0 ** -23)).all()
    assert (y[:, H:] == 7.0).all()
    got = y[:, :H].double().cpu().numpy()
    half = HALF_STEP[dtype]
    inner = bounds(x, ref["ids"], ref["w"], off(w13, W13), off(w2, W2), W13, W2, sh)
    # a weight's relative error moves its expert's whole share
    for t in range(M):
        for j, e in enumerate(ref["ids"][t]):
            inner[t] += np.abs(P.mlp(x[t], W13[e], W2[e])) * ref["w"][t, j] * (2 * dl + 2.0 ** -22)
        if S:
            inner[t] += np.abs(P.mlp(x[t], V13, V2)) * (dl + 2.0 ** -20)
    bound = half * (np.abs(ref["y"]) + inner) * 1.01 + inner + 2.0 ** -25
    err = np.abs(got - ref["y"])
    assert (err <= bound).all(), ((err / bound).max(), int((err > bound).sum()))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
def test_formats(hm, fmt, dtype):
    rng = np.random.default_rng([FORMATS.index(fmt), dtype == "bf16"])
    case(hm, rng, fmt, dtype, 3, 9, 384, 256, 4, S=128)


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 15, 16])
def test_token_counts(hm, M):
    rng = np.random.default_rng(M)
    case(hm, rng, FORMATS[0], "bf16", M, 16, 256, 128, 3)
    case(hm, rng, FORMATS[4], "fp16", M, 16, 256, 128, 3, S=64, gate=False)


@pytest.mark.parametrize("H,I,S", [(32, 32, 0), (32, 32, 32), (64, 96, 32), (160, 416, 224), (1056, 32, 160),
                                   (96, 1024, 0)])
def test_odd_widths(hm, H, I, S):
    """Widths that end inside a step of 128, and an h of another width than the shared expert's."""
    rng = np.random.default_rng([H, I, S])
    for fmt in (FORMATS[0], FORMATS[1], FORMATS[2]):
        case(hm, rng, fmt, "bf16", 5, 7, H, I, 2, S=S)


# pairs of 256 columns that a wave keeps of H, whole and partial; pairs and partial pairs of I and S
@pytest.mark.parametrize("H,I,S", [(2048, 64, 0), (2080, 32, 0), (2560, 32, 32), (4096, 32, 0), (4224, 32, 0),
                                   (6144, 32, 0), (6272, 32, 0), (64, 256, 256), (64, 512, 0), (64, 288, 352),
                                   (96, 768, 256), (64, 384, 128), (64, 256, 96)])
def test_shares_of_the_reduction(hm, H, I, S):
    rng = np.random.default_rng([H, I, S, 1])
    for fmt in (FORMATS[0], FORMATS[1], FORMATS[2], FORMATS[5]):
        step = max(fmt[1], 32)
        up = [-(-v // step) * step for v in (H, I, S)]
        case(hm, rng, fmt, "bf16", 3, 5, up[0], up[1], 2, S=up[2])


def test_many_shares_of_the_output(hm):
    """All 16 shares of a column tile, and one."""
    rng = np.random.default_rng(3)
    case(hm, rng, FORMATS[1], "bf16", 16, 40, 64, 512, 8)
    case(hm, rng, FORMATS[1], "bf16", 1, 3, 64, 32, 1)


@pytest.mark.parametrize("E,k,M", [(1, 1, 1), (1, 1, 16), (16, 16, 16), (64, 8, 6), (65, 1, 4), (300, 16, 16),
                                   (1024, 16, 16)])
def test_expert_counts(hm, E, k, M):
    rng = np.random.default_rng([E, k])
    case(hm, rng, FORMATS[1], "bf16", M, E, 64, 32, k)


@pytest.mark.parametrize("base", [None, "matrix", "own", "bias"])
def test_addends_and_strides(hm, base):
    rng = np.random.default_rng(7)
    case(hm, rng, FORMATS[3], "bf16", 6, 8, 192, 64, 2, S=32, base=base, strided=True)


def test_all_tokens_on_the_same_experts(hm):
    rng = np.random.default_rng(8)
    case(hm, rng, FORMATS[0], "fp16", 16, 32, 128, 64, 4, same=True)


def test_sharp_routing(hm):
    """Logits so far apart that one expert has nearly all the weight."""
    rng = np.random.default_rng(9)
    case(hm, rng, FORMATS[4], "bf16", 4, 12, 128, 64, 3, S=64, logits_scale=16.0)


def test_equal_logits_go_to_the_lower_id(hm):
    import torch
    rng = np.random.default_rng(10)
    E, H, I, k, M = 20, 64, 32, 5, 3
    w13, w2 = (upload(packed(rng, s, *FORMATS[1])) for s in ((E, 2 * I, H), (E, H, I)))
    x = torch.randn(M, H, device="cuda").bfloat16()
    y = torch.empty_like(x)
    ids = torch.empty(M, k, dtype=torch.int32, device="cuda")
    tw = torch.empty(M, k, device="cuda")
    ws = torch.empty(hm.moe_tokens_scratch_bytes(M, E, H, I, k), dtype=torch.uint8, device="cuda")
    hm.moe_tokens(x, torch.zeros(E, H, dtype=torch.bfloat16, device="cuda"), w13, w2, k, y, topk_ids=ids,
                  topk_w=tw, scratch=ws)
    assert torch.equal(ids.cpu(), torch.arange(k, dtype=torch.int32).expand(M, k))
    assert torch.allclose(tw, torch.full_like(tw, 1 / k), rtol=1e-6)


def test_a_bad_token_stays_alone(hm):
    """NaN in one token: its own row only."""
    import torch
    rng = np.random.default_rng(12)
    E, H, I, k, M, S = 10, 128, 64, 3, 5, 64
    for fmt in (FORMATS[0], FORMATS[2]):
        w13, w2 = (upload(packed(rng, s, *fmt)) for s in ((E, 2 * I, H), (E, H, I)))
        shared = (*(upload(packed(rng, s, *fmt)) for s in ((2 * S, H), (H, S))), None)
        router = torch.randn(E, H, device="cuda").bfloat16()
        x = torch.randn(M, H, device="cuda").bfloat16()
        ws = torch.empty(hm.moe_tokens_scratch_bytes(M, E, H, I, k, S), dtype=torch.uint8, device="cuda")
        want, y = torch.empty_like(x), torch.empty_like(x)
        hm.moe_tokens(x, router, w13, w2, k, want, shared=shared, scratch=ws)
        x[2, 5] = float("nan")
        hm.moe_tokens(x, router, w13, w2, k, y, shared=shared, scratch=ws)
        assert torch.isnan(y[2]).all()
        keep = [0, 1, 3, 4]
        assert torch.equal(y[keep], want[keep])


@pytest.mark.parametrize("M", [1, 8])
def test_captured_replays(hm, M):
    """New tokens, so other experts, between replays, with eager calls on the same scratch."""
    import torch
    rng = np.random.default_rng(M)
    E, H, I, k, S = 24, 256, 128, 4, 128
    w13, w2 = (upload(packed(rng, s, *FORMATS[0])) for s in ((E, 2 * I, H), (E, H, I)))
    shared = (*(upload(packed(rng, s, *FORMATS[0])) for s in ((2 * S, H), (H, S))), torch.randn(H, device="cuda").bfloat16())
    router = torch.randn(E, H, device="cuda").bfloat16()
    x = torch.randn(M, H, device="cuda").bfloat16()
    y, eager = torch.empty_like(x), torch.empty_like(x)
    ws = torch.empty(hm.moe_tokens_scratch_bytes(M, E, H, I, k, S), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        hm.moe_tokens(x, router, w13, w2, k, y, x, shared, scratch=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hm.moe_tokens(x, router, w13, w2, k, y, x, shared, scratch=ws)
    for _ in range(5):
        x.copy_(torch.randn(M, H, device="cuda"))
        hm.moe_tokens(x, router, w13, w2, k, eager, x, shared, scratch=ws)
        ws.fill_(0xFF)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager)


def test_beside_the_layers_forward(hm):
    """The uniform NVFP4 layer of the framework on the same weights and tokens, its logits from the
    router: both are within the layer's own bar of the same values."""
    import torch
    pk, w = tiny_packed(bit_map=None)
    M = 6
    x_bits = synth.activations_bf16(w, M)
    x = F.bf16_value(x_bits).astype(np.float64)
    router, rt = rounded(np.random.default_rng(0).standard_normal((w.E, w.H)) * w.H ** -0.5, "bf16")
    logits = x @ router.T
    ref = OL.forward(pk, x_bits, logits.astype(np.float32))["y"]
    kept = pk["kept"]

    def dev(a):
        return torch.from_numpy(np.ascontiguousarray(a)).cuda()
    w13 = hm.PackedMatrix(hm.WEIGHT_NVFP4, dev(kept["w13_q"]), dev(kept["w13_s"]), g=dev(kept["w13_g"]))
    w2 = hm.PackedMatrix(hm.WEIGHT_NVFP4, dev(kept["w2_q"]), dev(kept["w2_s"]), g=dev(kept["w2_g"]))
    xd = to_dev_bits(x_bits)
    y = torch.empty_like(xd)
    ws = torch.empty(hm.moe_tokens_scratch_bytes(M, w.E, w.H, w.I, w.top_k), dtype=torch.uint8, device="cuda")
    hm.moe_tokens(xd, rt.cuda(), w13, w2, w.top_k, y, scratch=ws)
    from hmoe_testlib import check_output, make_layer
    check_output(y.cpu().numpy().view(np.uint16), ref, "moe_tokens")
    layer = make_layer(pk, M)
    own, _ = run_forward(layer, hm.DeviceWeights(pk), x_bits, logits.astype(np.float32))
    check_output(own, ref, "hybrid_moe_forward")
