"""Calls of the experts' entry points whose arguments are good, where there is no GPU: the host side
runs as far as the launch, and a status comes back."""
import os
import subprocess
import sys

import pytest

from hyper_connection_mix_gb300 import build as hbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = 5  # HCMIX_ERR_CUDA

# aligned addresses that nothing reads: no kernel is launched
PROGRAM = """
import sys
from hyper_connection_mix_gb300 import experts
L, P = experts.lib(), 0x10000
calls = {
    "product": lambda: L.hc_mix_expert_product(P, 64, 0, 4, 64, 32, P, 64, 64 * 64, 0, P, 8, P, None),
    "gated": lambda: L.hc_mix_expert_product_gated(P, 64, 0, 4, 64, 32, P, 64, 64 * 64, 0, P, 8, P, P, None),
    "weight_backward": lambda: L.hc_mix_expert_product_weight_backward(P, 32, P, 64, 0, 4, 64, 32, 0, P, 8, P, 0, None),
    "weight_backward_f32": lambda: L.hc_mix_expert_product_weight_backward(P, 32, P, 64, 0, 4, 64, 32, 1, P, 8, P, 2, None),
    "weight_backward_of_none": lambda: L.hc_mix_expert_product_weight_backward(None, 32, None, 64, 0, 0, 64, 32, 0, P, 8, P, 0, None),
    "gate_backward": lambda: L.hc_mix_expert_gate_backward(P, 32, P, 64, 2, 4, 32, P, None),
    "q4": lambda: L.hc_mix_expert_product_q4(P, 64, 1, 4, 64, 32, P, P, 32, 0, P, 8, P, None),
}
print("status", calls[sys.argv[1]]())
"""


@pytest.mark.parametrize("call", ["product", "gated", "weight_backward", "weight_backward_f32", "weight_backward_of_none",
                                  "gate_backward", "q4"])
def test_a_status_comes_back(call):
    hbuild.build()
    run = subprocess.run([sys.executable, "-c", PROGRAM, call], cwd=ROOT, capture_output=True, text=True,
                         env={**os.environ, "CUDA_VISIBLE_DEVICES": ""})
    assert run.returncode == 0, (run.returncode, run.stderr[-2000:])
    assert run.stdout.split() == ["status", str(CUDA)]
