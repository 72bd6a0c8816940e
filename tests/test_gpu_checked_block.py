"""The checked build and the norm's and feed-forward block's kernels: their stores of results from registers are tested against
the operands' extents (results that leave through tensor maps are bounded by the maps); an access outside is skipped and the
call returns EP_ERR_DEVICE_CHECK. One test runs the operators' GPU tests in a child process that loads the checked
library, and there those that declare an operand shorter than it is.
"""
import os
import re
import subprocess
import sys

import pytest
import torch

from combine_topk_ids_dest_gb300 import EpError, EpFfn, EpNorm, _lib
from test_gpu_checked import _trim, in_checked_child
from test_gpu_checked_moe import ROOT, _reported
from test_gpu_ffn import make as make_ffn
from test_gpu_norm import make as make_norm

pytestmark = pytest.mark.gpu

SUITE = ["tests/test_gpu_norm.py", "tests/test_gpu_ffn.py", "tests/test_gpu_norm_cases.py", "tests/test_gpu_ffn_cases.py",
         "tests/test_gpu_block.py", "tests/test_gpu_checked_block.py"]
LATER = "not 32_bits and not at_once and not in_a_row"  # large, or of calls that would wait for one another here


@pytest.mark.skipif(_lib.checked(), reason="already the checked build")
def test_block_suite_under_checked_build(cuda_device):
    env = dict(os.environ, EP_GB300_CHECKED="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "-m", "gpu", "-k", LATER, *SUITE], cwd=ROOT,
                       env=env, capture_output=True, text=True, timeout=1800)
    assert r.returncode == 0, r.stdout[-6000:] + r.stderr[-3000:]
    tail = r.stdout.strip().splitlines()[-1]
    passed = re.search(r"(\d+) passed", tail)
    assert passed and int(passed.group(1)) >= 500 and re.search(r"\b1 skipped\b", tail), tail


@in_checked_child
def test_trimmed_norm_results_are_reported_and_skipped(cuda_device):
    x, _, w, dy, _ = make_norm(5, 192, torch.bfloat16)
    call = EpNorm(w)
    want, (dx, dweight) = call(x).out, call.backward(dy, x)
    out = torch.full_like(want, 7.0)
    _reported("moe_out", 192 * 2, 192 // 8, "moe: output row", lambda: call(x, out=out))  # 8 columns a store
    assert torch.equal(out[:4], want[:4]) and bool((out[4] == 7.0).all())
    got = torch.full_like(dx, 7.0)
    # dx's last store and dweight's last value
    _reported("moe_out", 4, 2, "moe: output row", lambda: call.backward(dy, x, dx=got))
    assert torch.equal(got[:4], dx[:4]) and torch.equal(got[4, :184], dx[4, :184]) and bool((got[4, 184:] == 7.0).all())
    again = call.backward(dy, x)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dweight)


@in_checked_child
@pytest.mark.parametrize("T", [5, 1100, 4000])
def test_trimmed_ffn_results_are_reported_and_skipped(cuda_device, T):
    x, gate_up, down, dy = make_ffn(T, 520, 1032)
    ffn = EpFfn(gate_up, down)
    want = ffn(x)
    out = torch.full_like(want, 7.0)
    _trim("moe_out", 520 * 2)
    try:
        with pytest.raises(EpError) as e:
            ffn(x, out=out)
    finally:
        _trim("", 0)
    # four columns a store of a split's blocks, one of a pair's
    assert re.search(r"\b(130|520) device accesses", str(e.value)) and "moe: output row" in str(e.value), str(e.value)
    assert torch.equal(out[:-1], want[:-1]) and bool((out[-1] == 7.0).all())
    _, saved = ffn.forward(x)
    dx = ffn.backward(dy, x, saved)[0]
    _reported("moe_out", 520 * 2, 520, "moe: output row", lambda: ffn.backward(dy, x, saved, need_weights=False))
    assert torch.equal(ffn.backward(dy, x, saved)[0], dx)
