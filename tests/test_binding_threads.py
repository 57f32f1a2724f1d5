"""The binding's first use, when another thread is in the middle of its own: a right call never
fails for that. The other thread's steps are played at the places where it can come between."""
import pytest

import weight_only_quantized_moe_amd as hm


def _route_tensors(torch):
    ids, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    return ids, w, torch.zeros_like(w), torch.zeros(4, 8)


def _calls(torch):
    """Right calls on CPU tensors: they get as far as the device check."""
    x, ids = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32)
    bf = torch.bfloat16
    return [lambda: hm.moe_permute(x, ids, 8, torch.zeros(8, 16, dtype=bf), torch.zeros(8, dtype=torch.int32),
                                   torch.zeros_like(ids), torch.zeros(9, dtype=torch.int32)),
            lambda: hm.moe_lora(x, ids[:, 0].contiguous(), torch.zeros(3, 8, 16, dtype=bf),
                                torch.zeros(3, 24, 8, dtype=bf), torch.zeros(3), None, torch.zeros(4, 24, dtype=bf)),
            lambda: hm.moe_route_backward(*_route_tensors(torch))]


@pytest.fixture
def unused(monkeypatch):
    """The binding as it is before its first call."""
    for name in ("_torch", "_I32", "_F32", "_this_device", "_raw_stream"):
        monkeypatch.setattr(hm, name, None)
    monkeypatch.setattr(hm, "_CODES", {})
    return monkeypatch


@pytest.mark.parametrize("i", range(3))
def test_while_the_types_are_entered(unused, i):
    """The second thread's call comes when the first one has just entered the element types."""
    torch = pytest.importorskip("torch")
    seen = []

    class Codes(dict):
        def update(self, *a):
            super().update(*a)
            if not seen:
                seen.append(1)
                with pytest.raises(ValueError, match="one GPU"):
                    _calls(torch)[i]()

    unused.setattr(hm, "_CODES", Codes())
    hm._load_torch()
    assert seen


@pytest.mark.parametrize("i", range(2))
def test_while_a_type_is_looked_up(unused, i):
    """The first thread ends its set-up right after the second one found its type missing."""
    torch = pytest.importorskip("torch")

    class Codes(dict):
        def get(self, *a):
            code = super().get(*a)
            if hm._torch is None:
                hm._load_torch()
            return code

    unused.setattr(hm, "_CODES", Codes())
    with pytest.raises(ValueError, match="one GPU"):
        _calls(torch)[i]()
