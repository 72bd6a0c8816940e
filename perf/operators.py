"""Cases and plain forms of the MoE layer's operators: router, experts, whole layer, 4-bit linear.

Each case names one operator (``op``):

- ``route``: a token's experts and weights from its hidden row (EpRouter).
- ``layer``: a whole MoE layer for a few tokens, router and experts (EpMoeLayer),
  with bf16 expert weights (``group`` 0) or 4-bit ones with a scale per ``group`` inputs.
- ``linear``: y = x W^T with 4-bit W and group scales (Int4Linear).

``run`` computes them in elementary torch operations, or with the package's kernels where ``own`` is set.
"""
import math

import torch

own = False

SIGMOID_SCALE = 2.5  # the routed experts' factor where sigmoid scores are renormalised


def listed():
    return [
        # routing of one decoded token, 128 experts: launch latency counts
        dict(name="route_one", op="route", T=1, H=4096, E=128, K=8, scoring="softmax", groups=1, top_groups=1,
             dtype="bf16"),
        # one rank's decode batch, 256 experts in 8 groups
        dict(name="route_decode", op="route", T=128, H=7168, E=256, K=8, scoring="sigmoid", groups=8, top_groups=4,
             dtype="bf16"),
        # a prefill's tokens over several ranks, a ragged count
        dict(name="route_prefill", op="route", T=16001, H=7168, E=256, K=8, scoring="sigmoid", groups=8, top_groups=4,
             dtype="bf16"),
        # one token through a small model's layer: the smallest layer call
        dict(name="layer_one_small", op="layer", T=1, H=2048, I=768, E=64, K=8, scoring="softmax", groups=1,
             top_groups=1, group=0, zeros=False),
        # one token through a layer of 256 wide experts: eight experts' weights are the traffic
        dict(name="layer_one", op="layer", T=1, H=7168, I=2048, E=256, K=8, scoring="sigmoid", groups=8, top_groups=4,
             group=0, zeros=False),
        # a few tokens over few, very wide experts: most experts get a token or two
        dict(name="layer_wide", op="layer", T=5, H=4096, I=14336, E=8, K=2, scoring="softmax", groups=1, top_groups=1,
             group=0, zeros=False),
        # a full decode batch: nearly every expert is read
        dict(name="layer_batch", op="layer", T=64, H=4096, I=2048, E=128, K=8, scoring="softmax", groups=1,
             top_groups=1, group=0, zeros=False),
        # one token, 4-bit experts
        dict(name="layer4_one", op="layer", T=1, H=7168, I=2048, E=256, K=8, scoring="sigmoid", groups=8, top_groups=4,
             group=128, zeros=False),
        # a ragged batch, 4-bit experts of an odd width with zero points
        dict(name="layer4_batch", op="layer", T=41, H=4096, I=1408, E=128, K=8, scoring="softmax", groups=1,
             top_groups=1, group=64, zeros=True),
        # a square projection for one token: the smallest 4-bit product
        dict(name="linear4_square", op="linear", T=1, N=4096, K=4096, group=128, zeros=False, dtype="bf16"),
        # a wide feed-forward projection for one token
        dict(name="linear4_wide", op="linear", T=1, N=28672, K=4096, group=128, zeros=True, dtype="bf16"),
        # a long reduction for a ragged batch, small groups
        dict(name="linear4_batch", op="linear", T=47, N=7168, K=18432, group=32, zeros=False, dtype="fp16"),
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of step in [lo, hi], spread over the logarithm; never 3072, nor half of it."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    v = min(max(v, lo), hi)
    return v + step if v in (3072, 1536, 6144) else v


def draw(rng):
    op = rng.choice(["route", "layer", "layer", "layer4", "linear", "linear"])
    if op == "linear":
        group = rng.choice([32, 64, 128])
        return dict(op="linear", T=_spread(rng, 1, 64), N=_spread(rng, 64, 28672), K=_spread(rng, 256, 18432, group),
                    group=group, zeros=rng.random() < 0.5, dtype=rng.choice(["bf16", "fp16"]))
    scoring = rng.choice(["softmax", "sigmoid"])
    groups = rng.choice([1, 1, 2, 4, 8])
    per = _spread(rng, max(2, 8 // groups), 256 // groups)
    E = groups * per
    top_groups = rng.randint(max(1, groups // 2), groups)
    K = rng.randint(1, min(10, per * top_groups))
    c = dict(op="route", T=_spread(rng, 1, 16384), H=_spread(rng, 256, 7168, 8), E=E, K=K, scoring=scoring,
             groups=groups, top_groups=top_groups)
    if op == "route":
        return dict(c, dtype=rng.choice(["bf16", "fp16"]))
    group = 0 if op == "layer" else rng.choice([32, 64, 128])
    step = group or 8
    H, I = _spread(rng, 512, 7168, step), _spread(rng, 256, 4096, step)
    while E * H * I > 128 * 4096 * 2048:  # no larger than the largest listed layer
        E, K = E - groups * ((E // groups + 1) // 2), 1 + (K - 1) // 2
        if E < groups * 2:
            groups, top_groups, E, K, I = 1, 1, 4, 2, step * (2048 // step)
    top_groups = min(top_groups, groups)
    K = min(K, (E // groups) * top_groups)
    T = min(_spread(rng, 1, 64), max(1, 64 * 8 * 4096 * 2048 // (K * H * I)))
    return dict(c, op="layer", T=T, H=H, I=I, E=E, K=K, groups=groups, top_groups=top_groups,
                group=group, zeros=bool(group) and rng.random() < 0.5)


# ---- inputs ------------------------------------------------------------------


def _dtype(case):
    return torch.float16 if case.get("dtype") == "fp16" else torch.bfloat16


def _activations(g, case, T, H):
    """Hidden rows as a norm leaves them: unit variance, a few channels much larger."""
    x = torch.randn(T, H, generator=g, device="cuda")
    x[:, :: max(1, H // 5)] *= 8.0
    return x.to(_dtype(case))


def _choose(scores, bias, case):
    """Selection values [T, E]: scores plus bias, groups that are not among the best set to -inf."""
    T, E = scores.shape
    s = scores if bias is None else scores + bias
    if case["groups"] > 1:
        per = s.view(T, case["groups"], E // case["groups"])
        best = torch.sort(per, dim=2, descending=True).values[:, :, :2].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, : case["top_groups"]]
        keep = torch.zeros_like(best, dtype=torch.bool).scatter(1, kept, True)
        s = torch.where(keep[:, :, None], per, torch.full_like(per, -math.inf)).view(T, E)
    return s


def _scores(logits, scoring):
    if scoring == "sigmoid":
        return 1 / (1 + torch.exp(-logits))
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _close(x, wg, bias, case):
    """Tokens whose choice hangs on rounding: two neighbours among the best K + 1 (or two groups' scores at
    the cut) nearer than 2e-5 of the values' size, in 64 bits."""
    s = _scores(x.double() @ wg.double().t(), case["scoring"])
    top = torch.sort(_choose(s, bias if bias is None else bias.double(), case), dim=1, descending=True).values
    top = top[:, : case["K"] + 1]
    near = (top[:, :-1] - top[:, 1:] < 2e-5 * top[:, :1].abs().clamp(max=1.0)) & torch.isfinite(top[:, 1:])
    bad = near.any(1)
    if case["groups"] > case["top_groups"]:
        b = s if bias is None else s + bias.double()
        best = torch.sort(b.view(len(x), case["groups"], -1), dim=2, descending=True).values[:, :, :2].sum(2)
        best = torch.sort(best, dim=1, descending=True).values
        k = case["top_groups"]
        bad |= best[:, k - 1] - best[:, k] < 2e-5 * best[:, 0].abs().clamp(max=1.0)
    return bad


def _router_inputs(case, g):
    T, H, E = case["T"], case["H"], case["E"]
    wg = (torch.randn(E, H, generator=g, device="cuda") * (1.5 / math.sqrt(H))).to(_dtype(case))
    bias = None
    if case["scoring"] == "sigmoid":  # the correction that balances the experts' load
        bias = torch.randn(E, generator=g, device="cuda") * 0.05
    x = _activations(g, case, T, H)
    for _ in range(20):  # whole numbers are compared for equality: tokens near a tie are drawn again
        bad = _close(x, wg, bias, case)
        n = int(bad.sum())
        if n == 0:
            break
        x[bad] = _activations(g, case, n, H)
    return x, wg, bias


def _quantised(g, rows, K, group, zeros):
    """4-bit codes [rows, K/2] (the low four bits are the even input), bf16 scales and zero points [rows, K/group]."""
    levels = torch.distributions.Normal(0.0, 2.6).icdf((torch.arange(256, device="cuda") + 0.5) / 256)
    levels = (levels.round() + 8).clamp(0, 15).to(torch.uint8)  # codes of normally distributed weights
    codes = torch.empty(rows, K // 2, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // K)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        pick = torch.randint(0, 256, (2, n, K // 2), generator=g, device="cuda", dtype=torch.int32)
        codes[r:r + n] = levels[pick[0]] | (levels[pick[1]] << 4)
    s = torch.randn(rows, K // group, generator=g, device="cuda") * 0.25
    s = (torch.exp(s) * (0.4 / math.sqrt(K))).to(torch.bfloat16)
    z = None
    if zeros:
        z = torch.randint(6, 11, (rows, K // group), generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)
    return codes, s, z


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "linear":
        x = _activations(g, case, case["T"], case["K"])
        return dict(x=x, w=_quantised(g, case["N"], case["K"], case["group"], case["zeros"]))
    x, wg, bias = _router_inputs(case, g)
    d = dict(x=x, wg=wg, bias=bias)
    if case["op"] == "layer":
        H, I, E = case["H"], case["I"], case["E"]
        if case["group"]:
            for name, rows, K in (("w13", 2 * I, H), ("w2", H, I)):
                parts = _quantised(g, E * rows, K, case["group"], case["zeros"])
                d[name] = tuple(None if p is None else p.view(E, rows, -1) for p in parts)
        else:
            for name, rows, K in (("w13", 2 * I, H), ("w2", H, I)):
                w = torch.empty(E, rows, K, dtype=torch.bfloat16, device="cuda")
                d[name] = w.normal_(0.0, 1 / math.sqrt(K), generator=g)
    return d


def _router_args(case):
    return dict(top_k=case["K"], scoring=case["scoring"], num_groups=case["groups"], top_groups=case["top_groups"],
                renormalize=True, scale=SIGMOID_SCALE if case["scoring"] == "sigmoid" else 1.0)


def prepare(case, seed):
    d = _inputs(case, seed)
    if not own:
        return dict(case=case, **d)
    import combine_topk_ids_dest_gb300 as ep

    def weight(w):
        return ep.Int4Weight(*w) if case["group"] else w

    if case["op"] == "linear":
        return dict(case=case, x=d["x"], call=ep.Int4Linear(weight(d["w"]), max_tokens=64))
    router = ep.EpRouter(d["wg"], bias=d["bias"], **_router_args(case))
    if case["op"] == "route":
        return dict(case=case, x=d["x"], call=router)
    experts = ep.EpExperts(weight(d["w13"]), weight(d["w2"]), top_k=case["K"], max_tokens=64)
    return dict(case=case, x=d["x"], call=ep.EpMoeLayer(router, experts))


# ---- plain forms ---------------------------------------------------------------


def _route(x, wg, bias, case, wide):
    """ids and weights, computed in the type `wide`."""
    s = _scores(x.to(wide) @ wg.to(wide).t(), case["scoring"])
    choose = _choose(s, None if bias is None else bias.to(wide), case)
    ids = torch.sort(choose, dim=1, descending=True, stable=True).indices[:, : case["K"]]
    w = s.gather(1, ids)
    w = w / w.sum(1, keepdim=True) * _router_args(case)["scale"]
    return ids, w


def _dequantised(w, wide):
    """(q - z) * s of 4-bit codes [..., K/2], as `wide`."""
    codes, s, z = w
    q = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).to(wide)
    q = q.view(*s.shape, -1) - (8 if z is None else z.to(wide)[..., None])
    return (q * s.to(wide)[..., None]).flatten(-2)


def _picked(w, e, wide):
    """The weights of the experts `e` (a list of ids), in full."""
    if isinstance(w, tuple):
        return _dequantised(tuple(None if p is None else p[e] for p in w), wide)
    return w[e].to(wide)


def _expert_outputs(x, w13, w2, e, wide):
    """Row j: the output of expert e[j] for the row x[j]."""
    gate, up = (_picked(w13, e, wide) @ x.to(wide)[:, :, None])[:, :, 0].chunk(2, dim=1)
    h = gate / (1 + torch.exp(-gate)) * up
    return (_picked(w2, e, wide) @ h[:, :, None])[:, :, 0]


def run(state):
    case, x = state["case"], state["x"]
    if own:
        out = state["call"](x)
        if case["op"] == "linear":
            return out
        return dict(ids=out[-2], weights=out[-1]) if case["op"] == "route" else \
            dict(y=out[0], ids=out[1], weights=out[2])
    wide = torch.float32
    if case["op"] == "linear":
        return (x.to(wide) @ _dequantised(state["w"], wide).t()).to(x.dtype)
    ids, w = _route(x, state["wg"], state["bias"], case, wide)
    out = dict(ids=ids.to(torch.int32), weights=w)
    if case["op"] == "layer":
        K = case["K"]
        o = _expert_outputs(x.repeat_interleave(K, 0), state["w13"], state["w2"], ids.reshape(-1), wide)
        out["y"] = (o.view(-1, K, x.shape[1]) * w[:, :, None]).sum(1).to(x.dtype)
    return out


# ---- work and 64-bit results -----------------------------------------------------


def _weight_bytes(rows, K, group, zeros):
    return rows * K * 2 if not group else rows * K / 2 + rows * (K / group) * (3 if zeros else 2)


def work(case):
    T, K = case["T"], case["K"]
    if case["op"] == "linear":
        N = case["N"]
        return dict(bytes=_weight_bytes(N, K, case["group"], case["zeros"]) + 2 * T * (N + K), flops=2 * T * N * K)
    H, E = case["H"], case["E"]
    b, f = 2 * E * H + 2 * T * H + 8 * T * K, 2 * T * E * H
    if case["op"] == "layer":
        I = case["I"]
        live = E * (1 - (1 - K / E) ** T)  # the expected number of experts that any token chose
        b += 2 * T * H + live * (_weight_bytes(2 * I, H, case["group"], case["zeros"]) +
                                 _weight_bytes(H, I, case["group"], case["zeros"]))
        f += 6 * T * K * H * I
    return dict(bytes=b, flops=f)


def _weights64(w, rows=slice(None)):
    """4-bit or bf16 weights in 64 bits, from the format's definition: nibble by nibble, group by group."""
    if not isinstance(w, tuple):
        return w[rows].double()
    codes, s, z = (None if p is None else p[rows] for p in w)
    n, half = codes.shape
    v = torch.empty(n, 2 * half, dtype=torch.float64, device=codes.device)
    v[:, 0::2], v[:, 1::2] = (codes % 16).double(), torch.div(codes, 16, rounding_mode="floor").double()
    per = 2 * half // s.shape[1]
    v -= 8.0 if z is None else z.double().repeat_interleave(per, 1)
    return v.mul_(s.double().repeat_interleave(per, 1))


def exact(case, seed):
    d = _inputs(case, seed)
    x = d["x"].double()
    if case["op"] == "linear":
        return torch.cat([x @ _weights64(d["w"], slice(r, r + 4096)).t() for r in range(0, case["N"], 4096)], 1)
    T, E, K = case["T"], case["E"], case["K"]
    logits = x @ d["wg"].double().t()
    p = torch.sigmoid(logits) if case["scoring"] == "sigmoid" else torch.softmax(logits, 1)
    rank = p.clone() if d["bias"] is None else p + d["bias"].double()
    if case["groups"] > 1:
        two = rank.view(T, case["groups"], -1).topk(2, dim=2).values.sum(2)
        out = two.topk(case["groups"] - case["top_groups"], dim=1, largest=False).indices
        rank.view(T, case["groups"], -1).scatter_(1, out[:, :, None].expand(-1, -1, E // case["groups"]), -math.inf)
    ids = rank.topk(K, dim=1).indices
    w = p.gather(1, ids)
    w = w / w.sum(1, keepdim=True) * _router_args(case)["scale"]
    result = dict(ids=None, weights=w)
    if case["op"] == "layer":
        y = torch.zeros_like(x)
        for e in torch.unique(ids).tolist():
            t, k = (ids == e).nonzero(as_tuple=True)

            def of(name):
                m = d[name]
                return _weights64(tuple(None if q is None else q[e] for q in m) if isinstance(m, tuple) else m[e])

            a = x[t] @ of("w13").t()
            h = torch.nn.functional.silu(a[:, : case["I"]]) * a[:, case["I"]:]
            y.index_add_(0, t, (h @ of("w2").t()) * w[t, k, None])
        result["y"] = y
    return result
