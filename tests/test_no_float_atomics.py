"""The operators around the experts promise sums of a fixed order: their kernels add atomically to
counters of ids in LDS only."""
import os
import re

import pytest

import weight_only_quantized_moe_amd as hm

CSRC = os.path.join(os.path.dirname(hm.__file__), "csrc")


@pytest.mark.parametrize("name", ["permute.hip", "lora.hip", "route.hip", "group_count.h"])
def test_atomics_count_ids_only(name):
    with open(os.path.join(CSRC, name)) as f:
        for call in re.findall(r"\w*[aA]tomic\w*\s*\([^;]*", f.read()):
            assert re.match(r"atomicAdd\(&s_cnt\[e\], (1|__popcll\(m\))\)", call) or "__ATOMIC_" in call, call
