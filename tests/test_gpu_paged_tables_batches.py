"""Tables of batches whose sums take about the shared memory that a kernel has without asking for more, each
in a process of its own: what an earlier call has asked for stays with the kernel."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

CODE = """
import sys
import numpy as np
sys.path[:0] = sys.argv[1:3]
from test_gpu_paged_tables import case, reference, run
for batch in map(int, sys.argv[3:]):
    c = case(seed=batch, batch=batch, P=16, mp=12, new=3, prefix=2)
    want, flags = reference(c)
    got, got_flags = run(c)
    assert all(np.array_equal(got[k], v) for k, v in want.items()) and got_flags == flags, batch
"""


@pytest.mark.parametrize("batches", [(2047, 3055, 3056), (3056,), (3071,), (4096, 3060, 4096, 3071)], ids=str)
def test_batches_in_a_fresh_process(batches):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_verify_paged_e4m3_gb300 import build
    build.build()
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", CODE, os.path.dirname(here), here, *map(str, batches)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
