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


# sizes whose launches have rounds that are cut over the pairs: parts of 1 to 4 blocks a tile, several products at once
CUT = [(515, 4096, 14336), (300, 7168, 2048), (1999, 2056, 1400), (700, 1024, 9000), (4100, 1032, 2504)]


@pytest.mark.parametrize("T,H,I", CUT)
def test_cut_rounds(cuda_device, T, H, I):
    x, gate_up, down, dy = make(T, H, I, seed=T)
    ffn = EpFfn(gate_up, down)
    want, err, state = block_ref.ffn(x, gate_up, down)
    y = ffn(x)
    block_ref.check(y, want, err, "y")
    y2, saved = ffn.forward(x)
    assert torch.equal(y, y2)
    grads = ffn.backward(dy, x, saved)
    for name, got, (g, e) in zip(("dx", "dgate_up", "ddown"), grads, block_ref.ffn_back(dy, state)):
        block_ref.check(got, g, e, name)


@pytest.mark.parametrize("T,H,I", [(515, 4096, 14336), (300, 7168, 2048), (1999, 2056, 1400), (128, 7168, 2048), (1, 4096, 4096)])
def test_calls_in_a_row_do_not_meet(cuda_device, T, H, I):
    """Kernels of calls that follow one another overlap: every call's results are those of a call alone, bit for bit."""
    a, b = make(T, H, I, seed=1), make(T, H, I, seed=2)
    ffns = [EpFfn(t[1], t[2]) for t in (a, b)]
    alone = []
    for f, t in zip(ffns, (a, b)):
        y, saved = f.forward(t[0])
        torch.cuda.synchronize()
        grads = f.backward(t[3], t[0], saved)
        torch.cuda.synchronize()
        alone.append((y, saved, *grads))
    got = []
    for i in (0, 0, 1, 0, 1, 1, 0, 1):  # nothing waits between
        t = (a, b)[i]
        y = ffns[i](t[0])
        y2, saved = ffns[i].forward(t[0])
        got.append((i, y, y2, saved, *ffns[i].backward(t[3], t[0], saved)))
    for i, y, *rest in got:
        assert torch.equal(y, alone[i][0])
        for x, want in zip(rest, alone[i]):
            assert torch.equal(x, want)
