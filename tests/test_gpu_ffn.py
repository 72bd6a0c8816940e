"""The feed-forward block and its gradients against 64-bit forms."""
import pytest
import torch

import block_ref
from combine_topk_ids_dest_gb300 import EpFfn
from combine_topk_ids_dest_gb300._lib import EpError

pytestmark = pytest.mark.gpu


def make(T, H, I, seed=0, spread=1.0):
    gen = torch.Generator("cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    x = randn(T, H)
    x[:, ::max(1, H // 5)] *= 8.0
    gate_up, down = randn(2 * I, H) * (spread / H ** 0.5), randn(H, I) / I ** 0.5
    return x.bfloat16(), gate_up.bfloat16(), down.bfloat16(), (randn(T, H) * 0.1).bfloat16()


# one token, both sides of where the few rows' kernel ends, tiles that end anywhere
ROWS = [1, 2, 17, 63, 64, 65, 66, 100, 127, 128, 129, 191, 256, 257, 515, 1000]
WIDTHS = [(8, 8), (72, 40), (136, 264), (512, 200), (1032, 520), (2056, 1400)]


@pytest.mark.parametrize("H,I", WIDTHS)
@pytest.mark.parametrize("T", ROWS)
def test_forward(cuda_device, T, H, I):
    x, gate_up, down, _ = make(T, H, I, seed=T)
    ffn = EpFfn(gate_up, down)
    want, err, _ = block_ref.ffn(x, gate_up, down)
    block_ref.check(ffn(x), want, err, "y")


@pytest.mark.parametrize("H,I", WIDTHS)
@pytest.mark.parametrize("T", [1, 2, 17, 64, 65, 129, 257, 515, 1000])
def test_training(cuda_device, T, H, I):
    x, gate_up, down, dy = make(T, H, I, seed=T + 1)
    ffn = EpFfn(gate_up, down)
    want, err, state = block_ref.ffn(x, gate_up, down)
    y, saved = ffn.forward(x)
    block_ref.check(y, want, err, "y")
    assert saved.shape == (T, 2 * I)
    block_ref.check(saved, torch.cat(state[3:5], 1), torch.cat(state[5:7], 1), "saved")
    grads = ffn.backward(dy, x, saved)
    for name, got, (g, e) in zip(("dx", "dgate_up", "ddown"), grads, block_ref.ffn_back(dy, state)):
        assert got.dtype is torch.bfloat16 and got.shape == g.shape
        block_ref.check(got, g, e, name)
