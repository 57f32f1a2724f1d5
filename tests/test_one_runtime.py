"""A program may ask a planner before it imports torch: the library and torch still share one HIP
runtime (with two of them in a process the library's launches find no device)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("first", ["hm.moe_lora_scratch_bytes(1, 1, 8, 8, 8)", "hm.moe_status_string(0)",
                                   "hm.moe_layer_create(8, 256, 128, 2, 4)"])
def test_one_hip_runtime(first):
    pytest.importorskip("torch")
    code = (f"import weight_only_quantized_moe_amd as hm\nkeep = {first}\nimport torch\n"
            "print(len({os.path.realpath(l.split()[-1]) for l in open('/proc/self/maps') if 'libamdhip64' in l}))")
    r = subprocess.run([sys.executable, "-c", "import os\n" + code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split()[-1] == "1"
