"""The binding imports and sizes workspaces where torch has no GPU backend: a torch built for
CPUs only lacks the private names that its GPU backend adds to torch._C."""
import os
import subprocess
import sys

import pytest

pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
from gated_delta_rule_prefill_amd import gdn
print("sizes", gdn.gdn_paged_decode_workspace_bytes(8, 2, 64, torch.bfloat16, 3),
      gdn.gdn_latent_decode_workspace_bytes(8, 256, 64, 64, 64, 3),
      gdn.gdn_latent_prefill_workspace_bytes(8, 256, 64, 64, 64, 3, 50, 90))
q, cache = torch.zeros(1, 4, 64).bfloat16(), torch.zeros(2, 4, 16, 64).bfloat16()
ints = torch.zeros(1, dtype=torch.int32)
try:
    gdn.gdn_paged_decode(q, cache, cache, ints.view(1, 1), ints)
except ValueError as e:
    print("refused", e)
"""


def test_binding_works_without_a_gpu_backend():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr
    sizes, refused = r.stdout.splitlines()
    assert all(int(x) > 0 for x in sizes.split()[1:]) and "on the GPU" in refused
