"""Plain 64-bit forms of the MoE operators and bounds on what fp32 sums may differ from them.

``g(n)`` below bounds the relative error of a sum of n products in fp32, in
any order and with truncating additions: n * 2**-23 of the sum of the
products' magnitudes. All bounds follow the formulas term by term from it.
"""
import torch

U_BF16, U_FP16 = 2.0 ** -8, 2.0 ** -11  # unit roundoff: 8 and 11 bits of significand
TINY = 2.0 ** -25  # fp16 results below the normal range


def g(n):
    return n * 2.0 ** -23


def dequant(codes, scales, zeros=None):
    """(q - z) * s of 4-bit codes [..., rows, cols/2], in 64 bits."""
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).double()
    n = scales.shape[-1]
    q = q.unflatten(-1, (n, q.shape[-1] // n))
    z = 8.0 if zeros is None else zeros.double()[..., None]
    return ((q - z) * scales.double()[..., None]).flatten(-2)


def make_int4(gen, *shape, group=32, zeros=False, dtype=torch.bfloat16, device="cuda"):
    """Random codes [..., rows, cols/2], scales and zero points for a weight of `shape` [..., rows, cols]."""
    lead, cols = shape[:-1], shape[-1]
    codes = torch.randint(0, 256, (*lead, cols // 2), generator=gen, device=device, dtype=torch.int32).to(torch.uint8)
    s = (torch.rand(*lead, cols // group, generator=gen, device=device) + 0.5) * (0.3 / cols ** 0.5)
    z = None
    if zeros:
        z = torch.randint(0, 16, (*lead, cols // group), generator=gen, device=device, dtype=torch.int32).to(torch.uint8)
    return codes, s.to(dtype), z


def linear(x, w):
    """y = x w^T and the bound on an fp32 sum's error; w in 64 bits."""
    x = x.double()
    return x @ w.t(), g(w.shape[1]) * (x.abs() @ w.abs().t())


def experts(x, ids, weights, gate_up, down, first=0):
    """The experts' weighted sum and the bound on its error before y is rounded (64-bit weights).

    gate and up: fp32 sums. silu's slope is at most 1.1. h keeps 16 bits of mantissa."""
    T, H = x.shape
    x = x.double()
    y, err = torch.zeros(T, H, dtype=torch.float64, device=x.device), torch.zeros(T, H, dtype=torch.float64, device=x.device)
    I = down.shape[2]
    for t in range(T):
        for k in range(ids.shape[1]):
            e = int(ids[t, k]) - first
            if not 0 <= e < gate_up.shape[0]:
                continue
            a, ea = gate_up[e] @ x[t], g(H + 8) * (gate_up[e].abs() @ x[t].abs())
            gate, up = a[:I], a[I:]
            s = gate * torch.sigmoid(gate)
            h = s * up
            eh = 1.1 * ea[:I] * (up.abs() + ea[I:]) + s.abs() * ea[I:] + 2.0 ** -16 * h.abs()
            w = float(weights[t, k])
            y[t] += w * (down[e] @ h)
            err[t] += abs(w) * (down[e].abs() @ (eh + g(I + 64) * h.abs()))
    return y, err


def close(got, want, err, unit):
    """Elementwise |got - want| within one rounding of the result plus the sums' error."""
    d = (got.double() - want).abs()
    bound = unit * (want.abs() + err) + err + (TINY if unit == U_FP16 else 0.0)
    assert bool((d <= bound).all()), f"worst {float((d / bound.clamp(min=1e-300)).max()):.3g} times the bound"


def scores(x, weight, scoring):
    """(logits, scores, bound on the scores' absolute error) [T, E] in 64 bits, for random inputs.

    The MMAs add 16 products to a partial sum at a time, 64 more additions join parts. Each may lose the last
    place of a partial sum, which stays within 4 standard deviations of the products' random walk."""
    l = x.double() @ weight.double().t()
    el = (x.shape[1] / 16 + 64) * 2.0 ** -23 * 4 * (x.double().square() @ weight.double().square().t()).sqrt()
    if scoring == "sigmoid":
        s = torch.sigmoid(l)
        return l, s, 0.25 * el + 4 * 2.0 ** -24
    s = torch.softmax(l, 1)
    return l, s, s * (2 * el.amax(1, keepdim=True) + 2.0 ** -20) + 2.0 ** -40


def choice(s, bias, top_k, groups=1, top_groups=1):
    """Chosen ids in descending order, ties to the lowest index, -1 where nothing is left; and the values."""
    T, E = s.shape
    c = s if bias is None else s + bias.double()
    c = torch.where(torch.isnan(c), torch.full_like(c, -torch.inf), c)
    if groups > 1:
        per = c.view(T, groups, E // groups)
        best = torch.sort(per, dim=2, descending=True).values[:, :, :2].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :top_groups]
        keep = torch.zeros_like(best, dtype=torch.bool).scatter(1, kept, True)
        c = torch.where(keep[:, :, None], per, torch.full_like(per, -torch.inf)).reshape(T, E)
    top = torch.sort(c, dim=1, descending=True, stable=True)
    ids, v = top.indices[:, :top_k], top.values[:, :top_k]
    return torch.where(v == -torch.inf, torch.full_like(ids, -1), ids), top.values


def chosen_weights(s, ids, renormalize, scale):
    w = s.gather(1, ids.clamp(min=0)) * (ids >= 0)
    if renormalize:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, w)
    return w * scale
