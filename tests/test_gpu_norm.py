"""The norm, its 8-bit rows and its gradients against 64-bit forms."""
import pytest
import torch

import block_ref
from combine_topk_ids_dest_gb300 import EpNorm

pytestmark = pytest.mark.gpu
EPS = 1e-6
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def make(T, H, dtype, seed=0, wide=False):
    gen = torch.Generator("cuda").manual_seed(seed)

    def rows(scale=1.0):
        x = torch.randn((T, H), generator=gen, device="cuda")
        x[:, ::max(1, H // 5)] *= 8.0
        return (x * scale).to(dtype)

    w = 1 + 0.2 * torch.randn(H, generator=gen, device="cuda")
    return rows(), rows(), w if wide else w.to(dtype), rows(0.1), rows(0.1)


# both sides of a warp's, a block's and a unit's columns, groups that are short, the widest row
WIDTHS = [8, 120, 128, 136, 256, 264, 1000, 2048, 2056, 4096, 7168, 8200, 16384]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("T", [1, 3, 37, 700])
def test_forward(cuda_device, T, H, dtype):
    x, residual, w, _, _ = make(T, H, dtype, seed=T + H, wide=T == 37)
    call = EpNorm(w, eps=EPS, dtype=dtype)
    s, y = block_ref.norm(x, residual, w, EPS)
    r = call(x, residual, quantized=True)
    block_ref.check(r.residual, s, block_ref.FP32 * s.abs(), "residual")
    block_ref.check(r.out, y, block_ref.NORM * y.abs(), "out")
    block_ref.check_quantized(r.q, r.scales, y)
    _, y = block_ref.norm(x, None, w, EPS)
    r = call(x)
    assert r.residual is None and r.q is None and r.scales is None
    block_ref.check(r.out, y, block_ref.NORM * y.abs(), "out without residual")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("T", [1, 3, 37, 700, 3001])
def test_backward(cuda_device, T, H, dtype):
    h, _, w, dy, dh = make(T, H, dtype, seed=T + H, wide=T == 37)
    call = EpNorm(w, eps=EPS, dtype=dtype)
    for other in (dh, None):
        dx, edx, dw, edw = block_ref.norm_back(dy, h, other, w, EPS)
        got, gotw = call.backward(dy, h, other)
        block_ref.check(got, dx, edx, "dx")
        assert gotw.dtype is torch.float32
        block_ref.check(gotw, dw, edw, "dweight")
