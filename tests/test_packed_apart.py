"""Outputs of the operators on 4-bit matrices that start where any of their weights do are refused. Nothing
here launches a kernel."""
import pytest

import weight_only_quantized_moe_amd as hm
from test_packed_boundary import A, INVALID, _linear, _tokens

Q, S, Z, G = 2, 3, 4, 5      # places in a matrix's description
MATRICES = ("w13", "w2", "s13", "s2")


def _with(fmt, name, place, at):
    """Matrices of the format whose arrays lie apart, but for one that lies at `at`."""
    group = 64 if fmt == hm.WEIGHT_INT4 else 0
    mats = {}
    for i, m in enumerate(MATRICES):
        first = (20 + 4 * i) * A
        d = [fmt, group, first, first + A, first + 2 * A, first + 3 * A]
        if m == name:
            d[place] = at
        mats[m] = tuple(d)
    return mats


@pytest.mark.parametrize("out", ["y", "ids", "w"])
@pytest.mark.parametrize("name", MATRICES)
@pytest.mark.parametrize("fmt,places", [(hm.WEIGHT_NVFP4, (Q, S, G)), (hm.WEIGHT_MXFP4, (Q, S)), (hm.WEIGHT_INT4, (Q, S, Z))])
def test_tokens_outputs_over_weights(fmt, places, name, out):
    at = 7 * A
    for place in places:
        assert _tokens(**{out: at}, **_with(fmt, name, place, at)) == INVALID, (name, place)
        assert "starts where an input does" in hm.moe_last_error()


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw", [{"q": 2 * A}, {"s": 2 * A}, {"z": 2 * A}, {"fmt": 0, "g": 2 * A}])
def test_linear_outputs_over_weights(back, kw):
    assert _linear(back, **kw) == INVALID
