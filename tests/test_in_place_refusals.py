"""Every output of the operators around the experts that starts where an input does is refused:
index and weight arrays as well as matrices. Nothing here launches a kernel."""
import pytest

import weight_only_quantized_moe_amd as hm

INVALID = 1
P = [(i + 1) << 40 for i in range(16)]     # distinct, aligned, never dereferenced


def _permute(x=P[0], ids=P[1], rows=P[2], srt=P[3], sr=P[4], off=P[5]):
    return hm.load_library().moe_permute(x, 16, ids, 4, 2, 8, 16, 0, rows, 16, srt, sr, off, None, 0, None)


def _permute_backward(drows=P[0], sr=P[1], dx=P[2]):
    return hm.load_library().moe_permute_backward(drows, 16, sr, 4, 2, 16, 0, dx, 16, None)


def _unpermute(rows=P[0], sr=P[1], w=P[2], y=P[3]):
    return hm.load_library().moe_unpermute(rows, 16, sr, w, 4, 2, 16, 0, y, 16, None)


def _unpermute_backward(dy=P[0], rows=P[1], sr=P[2], w=P[3], drows=P[4], dw=P[5]):
    return hm.load_library().moe_unpermute_backward(dy, 16, rows, 16, sr, w, 4, 2, 16, 0, drows, 16, dw, None)


def _route_backward(ids=P[0], w=P[1], dw=P[2], dl=P[3]):
    return hm.load_library().moe_route_backward(ids, w, dw, 4, 8, 2, dl, None)


def _lora(x=P[0], ids=P[1], a=P[2], b=P[3], sc=P[4], base=P[5], y=P[6], z=P[7]):
    return hm.load_library().moe_lora(x, 64, ids, a, b, sc, 4, 3, 64, 64, 8, base, 64, y, 64, z, P[15], 1 << 40, None)


def _lora_backward(dy=P[0], x=P[1], z=P[2], ids=P[3], a=P[4], b=P[5], sc=P[6], dbase=P[7], dx=P[8], dA=P[9], dB=P[10]):
    return hm.load_library().moe_lora_backward(dy, 64, x, 64, z, ids, a, b, sc, 4, 3, 64, 64, 8, dbase, 64, dx, 64,
                                               dA, dB, P[15], 1 << 40, None)


@pytest.mark.parametrize("f,ins,outs,allowed", [
    (_permute, ("x", "ids"), ("rows", "srt", "sr", "off"), ()),
    (_permute_backward, ("drows", "sr"), ("dx",), ()),
    (_unpermute, ("rows", "sr", "w"), ("y",), ()),
    (_unpermute_backward, ("dy", "rows", "sr", "w"), ("drows", "dw"), ()),
    (_route_backward, ("ids", "w", "dw"), ("dl",), ()),
    (_lora, ("x", "ids", "a", "b", "sc", "base"), ("y", "z"), (("base", "y"),)),
    (_lora_backward, ("dy", "x", "z", "ids", "a", "b", "sc", "dbase"), ("dx", "dA", "dB"), (("dbase", "dx"),))])
def test_an_output_over_an_input_or_output(f, ins, outs, allowed):
    for i, o in enumerate(outs):
        for other in ins + outs[:i]:
            if (other, o) in allowed:
                continue
            at = P[12]
            assert f(**{other: at, o: at}) == INVALID, f"{f.__name__}: {o} over {other}"
            assert hm.moe_last_error()


def test_in_place_over_a_second_input():
    """base may be y and dbase dx, but no other input with them."""
    assert _lora(x=P[12], base=P[12], y=P[12]) == INVALID
    for other in ("dy", "x"):
        assert _lora_backward(**{other: P[12]}, dbase=P[12], dx=P[12]) == INVALID
