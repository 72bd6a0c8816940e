"""A kernel that lets its successor start early and then takes longer than the limit of the waits inside a block: those
waits begin when it has ended."""
import ctypes
import os
import subprocess

import pytest
import torch

from combine_topk_ids_dest_gb300 import EpFfn, EpNorm, build
from test_gpu_ffn import make

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def slow(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("early") / "libearly.so")
    subprocess.run([build.nvcc(), *build.ARCH, "-shared", "-Xcompiler", "-fPIC", os.path.join(ROOT, "tests", "c", "early_trigger.cu"),
                    "-o", so], check=True, capture_output=True)
    L = ctypes.CDLL(so)
    L.early_trigger.argtypes = [ctypes.c_longlong, ctypes.c_void_p, ctypes.c_void_p]
    value = torch.zeros(1, device="cuda")

    def run():
        assert L.early_trigger(2600, value.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0

    return run, value


@pytest.mark.parametrize("T,H,I", [(3, 264, 520), (700, 2056, 1400)])  # clusters that share a tile's inputs, and pairs
def test_ffn(cuda_device, slow, T, H, I):
    x, gate_up, down, dy = make(T, H, I)
    call = EpFfn(gate_up, down)
    want, saved = call.forward(x)
    grads = call.backward(dy, x, saved)
    torch.cuda.synchronize()
    slow[0]()
    got = call(x)
    slow[0]()
    again = call.backward(dy, x, saved)
    torch.cuda.synchronize()
    assert torch.equal(call(x), want)  # a wait that ran out is this call's error
    assert torch.equal(got, want) and all(torch.equal(a, b) for a, b in zip(grads, again))


def test_norm(cuda_device, slow):
    x, _, _, dy = make(300, 264, 8)
    call = EpNorm(torch.ones(264, dtype=torch.bfloat16, device="cuda"))
    want, back = call(x).out, call.backward(dy, x)
    torch.cuda.synchronize()
    slow[0]()
    got = call.backward(dy, x)
    assert torch.equal(call(x).out, want) and all(torch.equal(a, b) for a, b in zip(back, got))
