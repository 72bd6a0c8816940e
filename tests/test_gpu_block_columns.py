"""Operands and results of the norm and the feed-forward block that are columns of one buffer's rows."""
import pytest
import torch

from combine_topk_ids_dest_gb300 import EpFfn, EpNorm
from test_gpu_ffn import make as make_ffn
from test_gpu_norm import make as make_norm

pytestmark = pytest.mark.gpu


def _beside(t, cols):
    """A buffer whose rows have t first, `cols` more columns next and 8 last: (buffer, t there, the columns)."""
    n = t.shape[1]
    b = torch.full((t.shape[0] + 1, n + cols + 8), 7.0, dtype=t.dtype, device="cuda")
    b[:-1, :n] = t
    return b, b[:-1, :n], b[:-1, n:n + cols]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(3, 264), (900, 256), (500, 2056)])
def test_norm(cuda_device, T, H, dtype):
    x, residual, w, dy, dh = make_norm(T, H, dtype, seed=T)
    call = EpNorm(w)
    want, back = call(x, residual), call.backward(dy, x, dh)
    (bx, wx, out), (br, wr, residual_out), (bd, wdy, dx) = (_beside(t, H) for t in (x, residual, dy))
    call(wx, wr, out=out, residual_out=residual_out)
    got = call.backward(wdy, x, dh, dx=dx)
    assert torch.equal(out, want.out) and torch.equal(residual_out, want.residual)
    assert torch.equal(dx, back[0]) and torch.equal(got[1], back[1])
    for b, t in ((bx, x), (br, residual), (bd, dy)):
        assert torch.equal(b[:-1, :H], t) and bool((b[-1] == 7).all()) and bool((b[:, 2 * H:] == 7).all())


@pytest.mark.parametrize("T,H,I", [(1, 264, 136), (70, 1024, 520), (900, 520, 1032)])
def test_ffn(cuda_device, T, H, I):
    x, gate_up, down, _ = make_ffn(T, H, I)
    call = EpFfn(gate_up, down)
    want = call(x)
    b, wx, out = _beside(x, H)
    call(wx, out=out)
    assert torch.equal(out, want) and torch.equal(b[:-1, :H], x)
    assert bool((b[-1] == 7).all()) and bool((b[:, 2 * H:] == 7).all())
