"""The checked build (libep_gb300_checked.so) and the MoE operators: their reads of ids and routing
weights and their stores of ids, weights and results are tested against the operands' extents; an access
outside is skipped and the call returns EP_ERR_DEVICE_CHECK. (Operands that come through copy engines, the
packed weights and the workspaces are not tested.)

test_moe_suite_under_checked_build runs the operators' GPU tests in a child process that loads the checked
library, and there the tests below it, which declare an operand shorter than it is and expect just the
accesses to its last row to be reported and skipped.
"""
import os
import re
import subprocess
import sys

import pytest
import torch

from combine_topk_ids_dest_gb300 import EpExperts, EpRouter, Int4Linear, Int4Weight, _lib
from combine_topk_ids_dest_gb300._lib import EpError
import moe_ref
from test_gpu_checked import _trim, in_checked_child
from test_gpu_moe_experts import _case

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SUITE = ["tests/test_gpu_moe_router.py", "tests/test_gpu_moe_experts.py", "tests/test_gpu_moe_sizes.py",
         "tests/test_gpu_moe_values.py", "tests/test_gpu_moe_example.py", "tests/test_gpu_checked_moe.py"]


@pytest.mark.skipif(_lib.checked(), reason="already the checked build")
def test_moe_suite_under_checked_build(cuda_device):
    env = dict(os.environ, EP_GB300_CHECKED="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "-m", "gpu", *SUITE], cwd=ROOT,
                       env=env, capture_output=True, text=True, timeout=1800)
    assert r.returncode == 0, r.stdout[-6000:] + r.stderr[-3000:]
    tail = r.stdout.strip().splitlines()[-1]
    # the only one the child skips is this one
    passed = re.search(r"(\d+) passed", tail)
    assert passed and int(passed.group(1)) >= 200 and re.search(r"\b1 skipped\b", tail), tail


def _reported(site, nbytes, accesses, name, call):
    _trim(site, nbytes)
    try:
        with pytest.raises(EpError) as e:
            call()
    finally:
        _trim("", 0)
    assert e.value.status == _lib.EP_ERR_DEVICE_CHECK
    assert f"{accesses} device accesses" in str(e.value) and name in str(e.value), str(e.value)


@in_checked_child
@pytest.mark.parametrize("group", [0, 32])
def test_trimmed_results_are_reported_and_skipped(cuda_device, group):
    x, ids, weights, w, _ = _case(5, 192, 160, 4, 2, group, seed=1)
    experts = EpExperts(*w, top_k=2)
    want = experts(x, ids, weights)
    out = torch.full_like(want, 7.0)
    _reported("moe_out", 192 * 2, 192, "moe: output row", lambda: experts(x, ids, weights, out=out))
    assert torch.equal(out[:4], want[:4]) and bool((out[4] == 7.0).all())
    assert torch.equal(experts(x, ids, weights), want)


@in_checked_child
def test_trimmed_linear_results_are_reported_and_skipped(cuda_device):
    gen = torch.Generator(device="cuda").manual_seed(4)
    linear = Int4Linear(Int4Weight(*moe_ref.make_int4(gen, 333, 512, group=128)))
    x = torch.randn(9, 512, generator=gen, device="cuda").bfloat16()
    want = linear(x)
    out = torch.full_like(want, 7.0)
    _reported("moe_out", 333 * 2, 333, "moe: output row", lambda: linear(x, out=out))
    assert torch.equal(out[:8], want[:8]) and bool((out[8] == 7.0).all())


@in_checked_child
@pytest.mark.parametrize("T", [5, 300, 10000])
@pytest.mark.parametrize("site,name", [("moe_ids", "moe: ids"), ("moe_weights", "moe: routing weights")])
def test_trimmed_choices_are_reported(cuda_device, T, site, name):
    gen = torch.Generator(device="cuda").manual_seed(5)
    router = EpRouter((torch.randn(32, 128, generator=gen, device="cuda") / 12).bfloat16(), 6)
    x = torch.randn(T, 128, generator=gen, device="cuda").bfloat16()
    _reported(site, 6 * 4, 6, name, lambda: router(x))
    router(x)
