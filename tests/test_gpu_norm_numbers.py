"""The norm's numbers at their ends: eps of any size next to rows of any size.

The bounds are block_ref's: scaling by a power of two loses nothing, so rows whose squares leave fp32 have the same error."""
import ctypes

import pytest
import torch

import block_ref
from combine_topk_ids_dest_gb300 import EpNorm
from test_gpu_norm import make

pytestmark = pytest.mark.gpu
FP32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dtype,size,eps", [
    (FP32, 1e-25, 1e-45), (FP32, 1e-21, 1e-44), (FP32, 1e-18, 1e-38), (FP32, 1e-22, 2e-38), (BF16, 1e-30, 1e-42), (BF16, 1e-24, 1e-45),
    (BF16, 1e-20, 1e-39), (FP32, 2e-13, 1e-24), (FP32, 3e18, 1e37), (BF16, 1e18, 1e36), (FP32, 1e19, 3e38), (FP32, 1.5e18, 3.4e38), (FP32, 1.0, 3e38),
    (BF16, 1e30, 1e38)])
@pytest.mark.parametrize("T,H", [(5, 8), (3, 256), (400, 1000), (5, 8200)])
def test_any_eps_next_to_rows_of_any_size(cuda_device, T, H, dtype, size, eps):
    x, _, w, dy, dh = make(T, H, FP32, seed=H)
    x[T // 2] = 0
    x, w, dy = (x / 8 * size).to(dtype), w.to(dtype), dy.to(dtype)
    eps = ctypes.c_float(eps).value  # as the call takes it
    call = EpNorm(w, eps=eps)
    _, y = block_ref.norm(x, None, w, eps)
    # fp32's own subnormals: half a step of 2^-149 of what is small, times the products behind it
    block_ref.check(call(x).out, y, block_ref.NORM * y.abs() + 2.0 ** -140, "out")
    dx, edx, dw, edw = block_ref.norm_back(dy, x, None, w, eps)
    gdx, gdw = call.backward(dy, x)
    block_ref.check(gdx, dx, edx + 2.0 ** -140, "dx")
    block_ref.check(gdw, dw, edw + 2.0 ** -140, "dweight")
