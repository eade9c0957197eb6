"""Sizes at which the pages' calls change how they launch."""
import os
import subprocess
import sys

import pytest
import torch

from _lib_util import ensure_built

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Batches around the one from which the plan's shared memory (16 bytes a sequence, and some that is static) passes 48 KB,
# in a process of its own: the limit of a kernel, once raised, stays raised.
EXTEND = """
import torch
from compressed_cache_decode_gb300 import lrkv
for B in (3055, 3056, 3060, 3071, 3073, 4096):
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    table, lens, refs = torch.full((B, 2), -1, dtype=torch.int32, device="cuda"), i([0] * B), i([0] * (B + 3))
    _, _, _, ws = lrkv.pages_extend([], table, lens, refs, 16, i([1] * B))
    torch.cuda.synchronize()
    assert lrkv.lrkv_read_device_status(ws) == lrkv.LRKV_OK
    assert table[:, 0].tolist() == list(range(B)) and lens.tolist() == [1] * B, B
    assert refs.tolist() == [1] * B + [0] * 3, B
print("done")
"""


def test_extend_of_any_batch_in_a_fresh_process():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    ensure_built()
    run = subprocess.run([sys.executable, "-c", EXTEND], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert run.returncode == 0 and "done" in run.stdout, run.stderr[-2000:]
