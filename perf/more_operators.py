"""Cases and plain forms of the operators around an MoE layer: the norm before it and the dense feed-forward beside it.

Each case names one operator (``op``):

- ``norm``: the residual's addition and the RMS norm (EpNorm), with rows in the inputs' type for the router and,
  where ``fp8`` is set, rows in 8 bits with a scale per 128 columns, as a dispatch carries them.
- ``norm_back``: its backward pass.
- ``ffn``: the gated feed-forward block (EpFfn), as a dense layer or a shared expert computes it.
- ``ffn_train``: its forward pass for training and its backward pass.

``run`` computes them in elementary torch operations, or with the package's kernels where ``own`` is set.
"""
import math

import torch

own = False

EPS = 1e-6
GROUP = 128  # columns of a scale
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one decoded token before an MoE layer: launch latency counts
        dict(name="norm_one", op="norm", T=1, H=4096, dtype="bf16", residual=True, fp8=True),
        # a decode batch: rows for the router and rows in 8 bits for the dispatch
        dict(name="norm_decode", op="norm", T=128, H=7168, dtype="bf16", residual=True, fp8=True),
        # a prefill's tokens, a ragged count
        dict(name="norm_prefill", op="norm", T=16001, H=7168, dtype="bf16", residual=True, fp8=True),
        # a final norm: no residual, no 8-bit rows, a width that no power of two divides
        dict(name="norm_odd", op="norm", T=4099, H=2056, dtype="fp16", residual=False, fp8=False),
        # a training step's rows
        dict(name="norm_back", op="norm_back", T=8192, H=4096, dtype="bf16", residual=True),
        # a few rows in full precision, without a gradient of the residual stream
        dict(name="norm_back_few", op="norm_back", T=333, H=2048, dtype="fp32", residual=False),
        # one token through a shared expert
        dict(name="ffn_one", op="ffn", T=1, H=7168, I=2048),
        # a decode batch through a shared expert: its weights are the traffic
        dict(name="ffn_decode", op="ffn", T=128, H=7168, I=2048),
        # a ragged batch through a wide dense layer
        dict(name="ffn_batch", op="ffn", T=515, H=4096, I=14336),
        # a prefill's tokens through a shared expert
        dict(name="ffn_prefill", op="ffn", T=8191, H=7168, I=2048),
        # a training step of a small model's layer, sizes that no tile divides
        dict(name="ffn_train_small", op="ffn_train", T=1999, H=2056, I=1400),
        # a training step of a wide dense layer
        dict(name="ffn_train", op="ffn_train", T=4096, H=4096, I=14336),
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of step in [lo, hi], spread over the logarithm."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    return min(max(v, lo), hi)


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_back", "ffn", "ffn", "ffn_train"])
    if op.startswith("norm"):
        c = dict(op=op, T=_spread(rng, 1, 16001), H=_spread(rng, 256, 7168, 8), dtype=rng.choice(sorted(DTYPES)),
                 residual=rng.random() < 0.7)
        return dict(c, fp8=rng.random() < 0.6) if op == "norm" else c
    H, I = _spread(rng, 512, 7168, 8), _spread(rng, 256, 14336, 8)
    if op == "ffn":
        return dict(op=op, T=min(_spread(rng, 1, 16384), 3 * 4096 * 4096 * 14336 // (H * I)), H=H, I=I)
    return dict(op=op, T=min(_spread(rng, 100, 8192), 4096 * 4096 * 14336 // (H * I)), H=H, I=I)


# ---- inputs ------------------------------------------------------------------


def _rows(g, T, H, dtype):
    """Hidden rows: unit variance, a few channels much larger."""
    x = torch.randn(T, H, generator=g, device="cuda")
    x[:, :: max(1, H // 5)] *= 8.0
    return x.to(dtype)


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T, H = case["T"], case["H"]
    if case["op"].startswith("norm"):
        dtype = DTYPES[case["dtype"]]
        d = dict(w=(1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(dtype))
        if case["op"] == "norm":
            d["x"] = _rows(g, T, H, dtype)
            d["residual"] = _rows(g, T, H, dtype) if case["residual"] else None
        else:
            d["h"] = _rows(g, T, H, dtype)
            d["dy"] = torch.randn(T, H, generator=g, device="cuda").mul_(0.1).to(dtype)
            d["dh"] = torch.randn(T, H, generator=g, device="cuda").mul_(0.1).to(dtype) if case["residual"] else None
        return d
    I = case["I"]
    d = dict(x=_rows(g, T, H, torch.bfloat16))
    for name, rows, cols in (("gate_up", 2 * I, H), ("down", H, I)):
        w = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
        d[name] = w.normal_(0.0, 1 / math.sqrt(cols), generator=g)
    if case["op"] == "ffn_train":
        d["dy"] = torch.randn(T, H, generator=g, device="cuda").mul_(0.1).to(torch.bfloat16)
    return d


def prepare(case, seed):
    d = _inputs(case, seed)
    if own:
        import combine_topk_ids_dest_gb300 as ep

        d["call"] = ep.EpNorm(d["w"], eps=EPS) if "w" in d else ep.EpFfn(d["gate_up"], d["down"])
    return dict(case=case, **d)


# ---- plain forms ---------------------------------------------------------------


def _norm(x, residual, w, fp8):
    s = x.float() if residual is None else x.float() + residual.float()
    y = s / torch.sqrt((s * s).mean(1, keepdim=True) + EPS) * w.float()
    out = dict(out=y.to(x.dtype))
    if residual is not None:
        out["residual"] = s.to(x.dtype)
    if fp8:
        T, H = y.shape
        groups = -(-H // GROUP)
        padded = torch.zeros(T, groups * GROUP, device=y.device)
        padded[:, :H] = y
        scales = (padded.view(T, groups, GROUP).abs().amax(2) / 448).clamp(min=2.0 ** -126)
        out["scales"] = scales
        out["q"] = (y / scales.repeat_interleave(GROUP, 1)[:, :H]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return out


def _norm_back(dy, h, dh, w):
    dy, h = dy.float(), h.float()
    rstd = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
    n, g = h * rstd, dy * w.float()
    dx = rstd * (g - n * (g * n).mean(1, keepdim=True))
    return (dx if dh is None else dx + dh.float()), (dy * n).sum(0)


def run(state):
    case, op = state["case"], state["case"]["op"]
    if own:
        call = state["call"]
        if op == "norm":
            r = call(state["x"], state["residual"], quantized=case["fp8"])
            out = dict(out=r.out)
            if case["residual"]:
                out["residual"] = r.residual
            return dict(out, scales=r.scales, q=r.q) if case["fp8"] else out
        if op == "norm_back":
            dx, dweight = call.backward(state["dy"], state["h"], state["dh"])
            return dict(dx=dx, dweight=dweight)
        if op == "ffn":
            return call(state["x"])
        y, saved = call.forward(state["x"])
        dx, dgate_up, ddown = call.backward(state["dy"], state["x"], saved)
        return dict(y=y, dx=dx, dgate_up=dgate_up, ddown=ddown)
    if op == "norm":
        return _norm(state["x"], state["residual"], state["w"], case["fp8"])
    if op == "norm_back":
        dx, dweight = _norm_back(state["dy"], state["h"], state["dh"], state["w"])
        return dict(dx=dx.to(state["h"].dtype), dweight=dweight)
    I, dtype = case["I"], state["x"].dtype
    x, w13, w2 = state["x"].float(), state["gate_up"].float(), state["down"].float()
    a = x @ w13.t()
    gate, up = a[:, :I], a[:, I:]
    sig = 1 / (1 + torch.exp(-gate))
    h = gate * sig * up
    y = (h @ w2.t()).to(dtype)
    if op == "ffn":
        return y
    dy = state["dy"].float()
    dhid = dy @ w2
    da = torch.cat((dhid * up * sig * (1 + gate * (1 - sig)), dhid * gate * sig), 1)
    return dict(y=y, dx=(da @ w13).to(dtype), dgate_up=(da.t() @ x).to(dtype), ddown=(dy.t() @ h).to(dtype))


# ---- work and 64-bit results -----------------------------------------------------


def work(case):
    T, H = case["T"], case["H"]
    if case["op"].startswith("norm"):
        e = DTYPES[case["dtype"]].itemsize
        if case["op"] == "norm":
            b = T * H * e * (4 if case["residual"] else 2) + H * e
            return dict(bytes=b + (T * H + 4 * T * -(-H // GROUP) if case["fp8"] else 0), flops=8 * T * H)
        return dict(bytes=T * H * e * (4 if case["residual"] else 3) + H * (e + 4), flops=12 * T * H)
    I = case["I"]
    if case["op"] == "ffn":
        return dict(bytes=6 * H * I + 4 * T * H, flops=6 * T * H * I)
    return dict(bytes=12 * H * I + 8 * T * H, flops=18 * T * H * I)


def _e4m3(v):
    """v rounded to the nearest number of 4 significant bits from 2^-6 on (steps of 2^-9 below), at most 448."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def exact(case, seed):
    d = {k: None if v is None else v.double() for k, v in _inputs(case, seed).items()}
    if case["op"] == "norm":
        s = d["x"] if d["residual"] is None else d["x"] + d["residual"]
        y = torch.nn.functional.rms_norm(s, (case["H"],), d["w"], EPS)
        out = dict(out=y)
        if case["residual"]:
            out["residual"] = s
        if case["fp8"]:
            parts = y.split(GROUP, 1)
            out["scales"] = torch.stack([p.abs().max(1).values / 448 for p in parts], 1)
            out["q"] = torch.cat([_e4m3(p / out["scales"][:, i:i + 1]) for i, p in enumerate(parts)], 1)
        return out
    with torch.enable_grad():
        if case["op"] == "norm_back":
            h, w = d["h"].requires_grad_(), d["w"].requires_grad_()
            y = torch.nn.functional.rms_norm(h, (case["H"],), w, EPS)
            dx, dweight = torch.autograd.grad(y, (h, w), d["dy"])
            return dict(dx=dx if d["dh"] is None else dx + d["dh"], dweight=dweight)
        x, w13, w2 = (d[k].requires_grad_(case["op"] == "ffn_train") for k in ("x", "gate_up", "down"))
        a = x @ w13.t()
        y = (torch.nn.functional.silu(a[:, : case["I"]]) * a[:, case["I"]:]) @ w2.t()
        if case["op"] == "ffn":
            return y
        dx, dgate_up, ddown = torch.autograd.grad(y, (x, w13, w2), d["dy"])
        return dict(y=y.detach(), dx=dx, dgate_up=dgate_up, ddown=ddown)
