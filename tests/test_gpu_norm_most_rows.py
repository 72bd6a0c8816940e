"""The norm on as many rows as a call may have: all zeros but a few, whose results are known."""
import pytest
import torch

import block_ref
from combine_topk_ids_dest_gb300 import EpNorm

pytestmark = pytest.mark.gpu
H, EPS = 8, 1e-6


@pytest.mark.parametrize("T", [2**31 - 1, 2**31 - 16, 2**31 - 17])
def test_most_rows(cuda_device, T):
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")  # 34 GB; its gradients, as much again, go where they came from
    gen = torch.Generator("cuda").manual_seed(1)
    at = torch.tensor([0, 1, 2**20 + 3, 2**30, 2**31 - 40, T - 17, T - 2, T - 1], device="cuda")
    rows = torch.randn(len(at), H, generator=gen, device="cuda").bfloat16()
    x[at] = rows
    w = (1 + 0.2 * torch.randn(H, generator=gen, device="cuda")).bfloat16()
    call = EpNorm(w, eps=EPS)
    dx = torch.full((T, H), 7.0, dtype=torch.bfloat16, device="cuda")
    _, dweight = call.backward(x, x, dx=dx)
    want, err, dw, edw = block_ref.norm_back(rows, rows, None, w, EPS)
    block_ref.check(dx[at], want, err, "dx")
    block_ref.check(dweight, dw, edw, "dweight")
    dx[at] = 0
    assert int(torch.count_nonzero(dx)) == 0
    _, y = block_ref.norm(rows, None, w, EPS)
    out = call(x, out=x).out
    block_ref.check(out[at], y, block_ref.NORM * y.abs(), "out")
    out[at] = 0
    assert int(torch.count_nonzero(out)) == 0
    del x, dx, out
    torch.cuda.empty_cache()
