"""The package on a torch built without CUDA: it imports, its host-only entry points work, and a call
that needs a GPU fails with an error of torch's or its own. No GPU needed."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)  # what such a torch lacks
import numpy as np
import nvfp4_kv_cache_gb300 as msa

freq, scale = msa.msa_rope_inv_freq(64, 1e4)
assert np.allclose(freq, 1e4 ** (-np.arange(32) / 32), rtol=1e-13) and scale == 1.0
assert msa.msa_dense_attn_workspace_size(4, 4, 1) > 0
try:
    msa.msa_rope_fp8(torch.zeros(1, 64, 128), None, msa.Rope(None), torch.zeros(1, 64, 128, dtype=torch.uint8))
except AssertionError:  # "Torch not compiled with CUDA enabled"
    print("refused")
"""


def test_a_torch_without_cuda():
    sys.path.insert(0, ROOT)
    import __graft_entry__

    __graft_entry__._load_builder().build()
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split() == ["refused"]
