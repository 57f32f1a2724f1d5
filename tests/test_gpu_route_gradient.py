"""moe_route_backward where its sums' form shows: values below the normal range, an id in many
slots."""
import numpy as np
import pytest

from hmoe_testlib import to_dev, torch_mod
from oracle import around as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hm():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_quantized_moe_amd as m
    m.load_library()
    return m


def _run(hm, ids, w, dw, E):
    torch = torch_mod()
    dl = torch.full((ids.shape[0], E), 9.0, device="cuda")
    hm.moe_route_backward(to_dev(ids), to_dev(w), to_dev(dw), dl)
    return dl.cpu().numpy()


@pytest.mark.parametrize("E", [8, 300, 1024])
def test_gradients_below_the_normal_range(hm, E):
    """A logit far below the largest has a weight, and so a gradient, of a few steps of 2^-149:
    w (dw - w dw) with dw = 1 is w to the last bit."""
    tiny = (np.arange(1, 8) * 2.0 ** -149).astype(np.float32)
    M, k = 6, 8
    ids = np.tile(np.arange(E - k, E, dtype=np.int32), (M, 1))
    w = np.tile(np.concatenate([[1.0], tiny]).astype(np.float32), (M, 1))
    dw = np.tile(np.array([0] + [1] * 7, np.float32), (M, 1))
    got = _run(hm, ids, w, dw, E)
    np.testing.assert_array_equal(got[:, E - 7:], np.tile(tiny, (M, 1)))


@pytest.mark.parametrize("M,E,k", [(1, 1, 1), (5, 3, 3), (33, 16, 16), (70, 300, 16), (9, 1024, 7)])
def test_the_same_id_in_many_slots(hm, M, E, k):
    """Whole numbers: the slots of an id add up exactly, whatever their places."""
    r = np.random.default_rng([M, E, k])
    ids = (r.integers(0, 3, (M, k)) * 257 % (E + 2)).astype(np.int32)     # few ids, some outside
    ids[0] = ids[0, 0]
    w, dw = r.integers(1, 4, (M, k)).astype(np.float32), r.integers(-8, 9, (M, k)).astype(np.float32)
    np.testing.assert_array_equal(_run(hm, ids, w, dw, E), R.route_backward(ids, w, dw, E))
