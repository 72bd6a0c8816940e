"""The checked build and a wait that runs out in the norm's backward pass: rows declared to lie outside their operand are
not copied, so the block's wait for them ends after its limit (about 2 s). What it gave up is NaN, the rest stands, and the
next call is as ever. One test runs the others in a child process that loads the checked library."""
import os
import re
import subprocess
import sys

import pytest
import torch

from combine_topk_ids_dest_gb300 import EpError, EpNorm, _lib
from test_gpu_checked import _trim, in_checked_child
from test_gpu_norm import make

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(_lib.checked(), reason="already the checked build")
def test_waits_under_checked_build(cuda_device):
    env = dict(os.environ, EP_GB300_CHECKED="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "-m", "gpu", "tests/test_gpu_checked_waits.py"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-6000:] + r.stderr[-3000:]
    tail = r.stdout.strip().splitlines()[-1]
    assert re.search(r"\b4 passed, 1 skipped\b", tail), tail


@in_checked_child
@pytest.mark.parametrize("T,H,wide,stage", [(5, 192, 0, 1), (5, 192, 8, 1), (4871, 256, 0, 16), (1000, 4104, 8, 1)])
def test_rows_given_up_are_nan(cuda_device, T, H, wide, stage):
    """stage: rows of a stage, of which a block gives up the last one here; wide: dy's rows are this much further apart."""
    x, _, w, dy, dh = make(T, H, torch.bfloat16)
    buffer = torch.zeros(T, H + wide, dtype=torch.bfloat16, device="cuda")
    buffer[:, :H] = dy
    dy = buffer[:, :H]
    call = EpNorm(w)
    want, dweight = call.backward(dy, x, dh)
    dx = torch.full_like(want, 7.0)
    _trim("moe_rows", 2)
    try:
        with pytest.raises(EpError) as e:
            call.backward(dy, x, dh, dx=dx)
    finally:
        _trim("", 0)
    assert e.value.status == _lib.EP_ERR_DEVICE_CHECK
    assert "3 device accesses" in str(e.value) and "moe: input row" in str(e.value), str(e.value)
    last = (T - 1) // stage * stage
    assert torch.equal(dx[:last], want[:last]) and bool(dx[last:].isnan().all())
    again = call.backward(dy, x, dh)
    assert torch.equal(again[0], want) and torch.equal(again[1], dweight)
