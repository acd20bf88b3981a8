"""The Python binding where its C++ half is not there, or is of another torch."""

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import sys, warnings
sys.modules["gated_delta_rule_intra_gb300._native"] = None  # an import of it fails
import torch
import gated_delta_rule_intra_gb300 as kda

lib = kda.load_library()
assert kda.kda_abi_version() == kda.ABI_VERSION and kda.kda_status_str(0)
x, g = torch.zeros(1, 4, 2, 128, dtype=torch.bfloat16), torch.zeros(1, 4, 2, 128)
calls = (lambda: kda.kda_chunk_fwd(x, x, x, g, g[..., 0]),
         lambda: kda.kda_chunk_bwd(x, x, x, g, g[..., 0], x, torch.zeros(0, dtype=torch.uint8)),
         lambda: kda.kda_step(x[0], x[0], x[0], g[0], g[0, ..., 0], torch.zeros(4, 2, 128, 128)),
         lambda: kda.kda_layer_norm_fwd(x),
         lambda: kda.kda_layer_norm_bwd(x, x, None, g[..., 0], g[..., 0]))
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    for call in calls:
        try:
            call()
        except ValueError as e:
            assert "CUDA" in str(e)
        else:
            raise AssertionError("a CPU tensor was taken")
assert len(seen) == 1 and "build_native" in str(seen[0].message), seen
print("ok")
"""


def test_the_library_works_without_the_bindings_native_half():
    """Only the short way into the newer calls is in _native.so: the library loads without it, says
    so once when one of them is used, and checks arguments as ever."""
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
