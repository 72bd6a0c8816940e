"""Plain 64-bit forms of the norm and the feed-forward block, and bounds on what the kernels may differ from them.

A rounding is off by at most half a step: UNIT[t] of the value. What rounded operands of a product leave in a sum is
taken as a sum of independent errors, each within half a step of its term: it exceeds SIGMAS times the root of the sum
of their squares with a probability of 2 exp(-SIGMAS^2 / 2) = 5e-11 (Hoeffding's inequality).
"""
import torch

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}  # half the smallest step
U = UNIT[torch.bfloat16]
SIGMAS = 7.0
FP32 = 2.0 ** -24
# A row's sums: a thread adds at most 32 columns one after the other, then 10 levels of a tree; 12 more roundings of the
# residual's addition, the root and the products.
NORM = 64 * FP32


def check(got, want, err, what=""):
    """|got - want| within one rounding of the result's type and the error `err` before it."""
    unit = UNIT[got.dtype]
    d = (got.double() - want).abs()
    bound = unit * (want.abs() + err) + err + TINY[got.dtype]
    worst = (d / bound).nan_to_num(nan=float("inf")).max().item() if d.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} times the bound"


def norm(x, residual, w, eps):
    """(s, y) in 64 bits."""
    s = x.double() if residual is None else x.double() + residual.double()
    return s, s / (s.square().mean(1, keepdim=True) + eps).sqrt() * w.double()


def check_quantized(q, scales, y, group=128):
    """Codes and scales of 64-bit rows y whose fp32 form is within NORM of them."""
    T, H = y.shape
    n = -(-H // group)
    assert q.shape == (T, H) and scales.shape == (T, n)
    pad = torch.zeros(T, n * group, dtype=torch.float64, device=y.device)
    pad[:, :H] = y.abs()
    want = (pad.view(T, n, group).amax(2) / 448).clamp(min=2.0 ** -126)
    assert bool(((scales.double() - want).abs() <= (NORM + 2 * FP32) * want).all()), "scales"
    s = scales.double().repeat_interleave(group, 1)[:, :H]
    half = torch.maximum(y.abs() * 2.0 ** -4, s * 2.0 ** -10)  # of e4m3's step: normal, and below 2^-6
    off = (q.double() * s - y).abs()
    assert bool((off <= half * (1 + 4 * NORM) + 4 * NORM * y.abs()).all()), "codes"


def norm_back(dy, h, dh, w, eps):
    """(dx, its error, dweight, its error) in 64 bits."""
    dy, h, w = dy.double(), h.double(), w.double()
    r = 1 / (h.square().mean(1, keepdim=True) + eps).sqrt()
    n, g = h * r, dy * w
    dx = r * (g - n * (g * n).mean(1, keepdim=True))
    err = 2 * NORM * r * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    if dh is not None:
        dx = dx + dh.double()
        err = err + FP32 * dx.abs()
    # at least 152 blocks add their rows one after the other, 32 warps every 32nd of up to 1024 parts, then 32 sums
    depth = h.shape[0] / 128 + 32 + 32
    return dx, err, (dy * n).sum(0), (2 * NORM + depth * FP32) * (dy * n).abs().sum(0)


def _product(a, b, ea=None):
    """a b^T and the error that its sum, and errors within ea of a's elements, leave: the MMAs add 16 products at a time
    to a partial sum, which stays within 4 standard deviations of the products' random walk, 64 additions join parts;
    each may lose the last place."""
    root = (a.square() @ b.square().t()).sqrt()
    err = 4 * (a.shape[1] / 16 + 64) * 2 * FP32 * root
    if ea is not None:
        err = err + SIGMAS * (ea.square() @ b.square().t()).sqrt()
    return a @ b.t(), err


def ffn(x, gate_up, down, h_unit=U):
    """(y, its error before rounding, what the backward pass needs) in 64 bits."""
    x, w13, w2 = x.double(), gate_up.double(), down.double()
    I = w2.shape[1]
    a, ea = _product(x, w13)
    g, u, eg, eu = a[:, :I], a[:, I:], ea[:, :I], ea[:, I:]
    s = g * torch.sigmoid(g)
    h = s * u
    eh = 1.1 * eg * (u.abs() + eu) + s.abs() * eu + 8 * FP32 * h.abs()  # silu's slope is at most 1.1
    y, ey = _product(h, w2, eh + h_unit * (h.abs() + eh))
    return y, ey, (x, w13, w2, g, u, eg, eu, h, eh)


def ffn_back(dy, state):
    """[(gradient, its error before rounding)] of x, gate_up and down."""
    x, w13, w2, g, u, eg, eu, h, eh = state
    dy = dy.double()
    dh, edh = _product(dy, w2.t())
    sig = torch.sigmoid(g)
    silu, slope = g * sig, sig * (1 + g * (1 - sig))  # slope at most 1.1, its own slope at most 0.5
    dg, du = dh * u * slope, dh * silu
    edg = 1.1 * (edh * (u.abs() + eu) + dh.abs() * eu) + (dh * u).abs() * 0.5 * eg + 16 * FP32 * dg.abs()
    edu = edh * (silu.abs() + 1.1 * eg) + dh.abs() * 1.1 * eg + 16 * FP32 * du.abs()
    da, eda = torch.cat((dg, du), 1), torch.cat((edg, edu), 1)
    eda = eda + U * (da.abs() + eda)
    eh = eh + U * (h.abs() + eh)
    return [_product(da, w13.t(), eda), _product(da.t(), x.t(), eda.t()),
            tuple(t.t() for t in _product(h.t(), dy.t(), eh.t()))]
