"""The feed-forward block's gate far from zero: silu and its slope keep their value down to fp32's smallest numbers."""
import pytest
import torch

from combine_topk_ids_dest_gb300 import EpFfn

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("T", [1, 3, 300])
@pytest.mark.parametrize("g", [-60.0, -86.5, -87.5, -88.0, -88.5, -89.0, -92.0, -95.0, -100.0, 20.0, 88.0])
def test_one_gate(cuda_device, T, g):
    """Products of a single term each, so every value is known: the gate g, up and the second weight large enough to see
    silu(g) beside one rounding."""
    H, I, up = 64, 72, 2.0 ** 90
    x, gate_up, down = (torch.zeros(*s, dtype=BF16, device="cuda") for s in ((T, H), (2 * I, H), (H, I)))
    x[:, 0], gate_up[5, 0], gate_up[I + 5, 0], down[3, 5] = 1, g, up, 1
    dy = torch.zeros(T, H, dtype=BF16, device="cuda")
    dy[:, 3] = 1
    call = EpFfn(gate_up, down)
    y, saved = call.forward(x)
    wide = torch.tensor(g, dtype=torch.float64)
    s = torch.sigmoid(wide).item()
    rest = torch.sigmoid(-wide).item()  # 1 - s
    silu, slope = g * s, s * (1 + g * rest)
    # exp(-|g|) to 2 + 1.173 |g| units of the last place, quotient and products 8 more; fp32's subnormals: half a step of
    # 2^-149 of the exponential, of sigma and of silu, times what follows
    rel, tiny = (10 + 1.173 * abs(g)) * 2.0 ** -23, 3 * 2.0 ** -150

    def near(got, want, factor, roundings, what, small=1.0):
        # small: what follows the rounding of a value that may be one of bf16's subnormals, whose half step is 2^-134
        err = abs(want) * (rel + roundings * 2.0 ** -8 * 1.01) + abs(factor) * tiny * (1 + abs(g)) + (1 + abs(small)) * 2.0 ** -134
        d = (got.double() - want).abs().max().item()
        assert d <= err, f"{what}: {d:.3g} of {want:.3g}, bound {err:.3g}"

    near(y[:, 3], silu * up, up, 2, "y")  # h is rounded, then y
    grads = [torch.zeros(*t.shape, dtype=torch.float32, device="cuda") for t in (gate_up, down)]
    dx, dgate_up, ddown = call.backward(dy, x, saved, dgate_up=grads[0], ddown=grads[1])
    near(dgate_up[5, 0], T * up * slope, T * up, 1, "dW1")
    near(dgate_up[I + 5, 0], T * silu, T, 1, "dW3", T)
    near(ddown[3, 5], T * silu * up, T * up, 1, "dW2")
    near(dx[:, 0], up * slope * g + silu * up, up * (1 + abs(g)), 2 * (abs(slope * g) + abs(silu)) / max(abs(slope * g + silu), 1e-300), "dx",
         up)
