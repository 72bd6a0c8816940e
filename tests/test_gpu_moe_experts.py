"""EpExperts, EpMoeLayer and Int4Linear against the 64-bit forms, within the bounds that fp32 sums
and one rounding of the result give; odd sizes, empty and doubled choices, layouts, streams, graphs,
refusals, and the layer split over virtual ranks."""
import pytest
import torch

import combine_topk_ids_dest_gb300 as ep
import moe_ref
from combine_topk_ids_dest_gb300 import EpError, EpExperts, EpMoeLayer, EpRouter, Int4Linear, Int4Weight

pytestmark = pytest.mark.gpu


def _case(T, H, I, E, K, group=0, zeros=False, seed=0, ids=None, scale_dtype=torch.bfloat16):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, H, generator=gen, device="cuda").bfloat16()
    if group:
        raw = [moe_ref.make_int4(gen, E, r, c, group=group, zeros=zeros, dtype=scale_dtype) for r, c in ((2 * I, H), (H, I))]
        w = [Int4Weight(*r) for r in raw]
        exact = [moe_ref.dequant(*r) for r in raw]
    else:
        w = [(torch.randn(E, r, c, generator=gen, device="cuda") / c ** 0.5).bfloat16() for r, c in ((2 * I, H), (H, I))]
        exact = [t.double() for t in w]
    if ids is None:
        ids = torch.rand(T, E, generator=gen, device="cuda").argsort(1)[:, :K].int()
    weights = torch.rand(T, K, generator=gen, device="cuda") + 0.1
    return x, ids.contiguous(), weights, w, exact


def _check(x, ids, weights, w, exact, first=0, **kw):
    experts = EpExperts(*w, top_k=ids.shape[1], first_expert=first, **kw)
    y = experts(x, ids, weights)
    moe_ref.close(y, *moe_ref.experts(x, ids, weights, *exact, first), moe_ref.U_BF16)
    return experts, y


@pytest.mark.parametrize("T,H,I,E,K", [
    (1, 8, 8, 1, 1), (1, 256, 128, 4, 2), (2, 128, 136, 3, 3), (5, 520, 264, 6, 2), (8, 192, 64, 16, 4), (9, 640, 1000, 5, 2),
    (17, 72, 328, 40, 3), (33, 1032, 200, 7, 4), (64, 256, 384, 8, 2), (64, 136, 72, 130, 8), (23, 512, 256, 512, 1)])
def test_dense_matches_the_64_bit_form(cuda_device, T, H, I, E, K):
    _check(*_case(T, H, I, E, K, seed=T + H))


@pytest.mark.parametrize("T,H,I,E,K,group,zeros", [
    (1, 32, 32, 1, 1, 32, False), (1, 256, 128, 4, 2, 128, True), (3, 416, 160, 6, 2, 32, True), (4, 128, 64, 3, 3, 64, False),
    (6, 192, 448, 16, 4, 64, True), (8, 128, 384, 9, 2, 128, False), (9, 640, 352, 5, 2, 32, True), (16, 320, 64, 4, 3, 64, True),
    (30, 256, 128, 3, 2, 128, True), (33, 96, 288, 40, 3, 32, False), (64, 256, 384, 8, 2, 128, True),
    (64, 160, 96, 130, 8, 32, True)])
def test_int4_matches_the_64_bit_form(cuda_device, T, H, I, E, K, group, zeros):
    _check(*_case(T, H, I, E, K, group, zeros, seed=T + H))


@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("T", [1, 7, 25, 33, 48, 64])
def test_every_token_to_one_expert(cuda_device, group, T):
    ids = torch.full((T, 1), 2, dtype=torch.int32, device="cuda")
    _check(*_case(T, 320, 192, 4, 1, group, seed=T, ids=ids))


@pytest.mark.parametrize("group,H,I", [(0, 640, 1000), (32, 640, 992), (64, 1152, 704), (128, 512, 384), (32, 96, 64)])
@pytest.mark.parametrize("order", [1, -1])
def test_experts_of_very_different_sizes(cuda_device, group, H, I, order):
    sizes = [1, 4, 5, 8, 9, 16, 17, 24, 25, 32, 33, 64][::order]
    t = torch.arange(64, device="cuda")[:, None]
    e = torch.arange(len(sizes), device="cuda")[None, :]
    ids = torch.where((t + 5 * e) % 64 < torch.tensor(sizes, device="cuda"), e, -1).int()
    _check(*_case(64, H, I, len(sizes), len(sizes), group, seed=H, ids=ids))


@pytest.mark.parametrize("group", [0, 32])
@pytest.mark.parametrize("T", [1, 6, 40])
def test_absent_doubled_and_foreign_ids(cuda_device, group, T):
    gen = torch.Generator(device="cuda").manual_seed(T)
    ids = torch.randint(-3, 14, (T, 5), generator=gen, device="cuda", dtype=torch.int32)  # experts 4..9 are here
    ids[0] = torch.tensor([-1, 3, 10, 2**31 - 1, -2**31], device="cuda")  # nothing
    if T > 1:
        ids[1] = 5  # one expert five times
    case = _case(T, 192, 160, 6, 5, group, ids=ids, seed=T)
    _, y = _check(*case, first=4)
    assert bool((y[0] == 0).all())


@pytest.mark.parametrize("group", [0, 128])
def test_no_token_has_an_expert_here(cuda_device, group):
    x, ids, weights, w, _ = _case(5, 256, 128, 4, 2, group)
    experts = EpExperts(*w, top_k=2, first_expert=100)
    out = torch.full((5, 256), float("nan"), dtype=torch.bfloat16, device="cuda")
    assert experts(x, ids, weights, out=out) is out
    assert bool((out == 0).all())
    assert experts(x[:0], ids[:0], weights[:0]).shape == (0, 256)
    y = EpExperts(*w, top_k=2)(x, ids, weights)
    assert bool((y != 0).any())


@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("T", [3, 20])
def test_nan_and_infinity_keep_to_their_token(cuda_device, group, T):
    x, ids, weights, w, _ = _case(T, 256, 192, 4, 2, group, seed=2)
    experts = EpExperts(*w, top_k=2)
    clean = experts(x, ids, weights)
    bad = x.clone()
    bad[0], bad[2, 5] = float("nan"), float("inf")
    y = experts(bad, ids, weights)
    keep = [t for t in range(T) if t not in (0, 2)]
    assert torch.equal(y[keep], clean[keep])
    assert bool(y[0].isnan().all()) and not bool(y[2].isfinite().all())


@pytest.mark.parametrize("group", [0, 64])
def test_strided_rows_streams_graphs_and_reuse(cuda_device, group):
    x, ids, weights, w, exact = _case(12, 256, 320, 6, 3, group, seed=4)
    experts, want = _check(x, ids, weights, w, exact, max_tokens=12)
    wide = torch.zeros(12, 2, 256, dtype=torch.bfloat16, device="cuda")
    wide[:, 1] = x
    out = torch.zeros(12, 264, dtype=torch.bfloat16, device="cuda")
    experts(wide[:, 1], ids, weights, out=out[:, 3:259])
    assert torch.equal(out[:, 3:259], want) and bool((out[:, :3] == 0).all()) and bool((out[:, 259:] == 0).all())
    for n in (1, 9, 12, 2):  # calls of other sizes leave nothing behind
        assert torch.equal(experts(x[:n], ids[:n], weights[:n])[:1], experts(x[:1], ids[:1], weights[:1])) or n > 8
        assert torch.equal(experts(x, ids, weights), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = experts(x, ids, weights)
    side.synchronize()
    assert torch.equal(got, want)
    sx, si, sw = x.clone(), ids.clone(), weights.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = experts(sx, si, sw)
    for shift in (1, 5):  # the ids of a replay are read when it runs
        sx.copy_(x.roll(shift, 0))
        si.copy_(ids.roll(shift, 0))
        sw.copy_(weights.roll(shift, 0))
        graph.replay()
        moe_ref.close(y, *moe_ref.experts(sx, si, sw, *exact), moe_ref.U_BF16)


@pytest.mark.parametrize("group", [0, 32])
def test_two_handles_on_two_streams(cuda_device, group):
    """Their blocks wait for one another; cooperative launches keep the two from starving each other."""
    cases = [_case(10, 512, 768, 8, 2, group, seed=s) for s in (5, 6)]
    handles = [EpExperts(*c[3], top_k=2) for c in cases]
    want = [h(*c[:3]) for h, c in zip(handles, cases)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(handles[i](*cases[i][:3]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


def test_large_offsets(cuda_device):
    """The last expert's weights begin past 2^32 bytes."""
    E, H, I = 200, 2048, 2752  # 22.5 MB a gate_up
    gate_up = torch.zeros(E, 2 * I, H, dtype=torch.bfloat16, device="cuda")
    down = torch.zeros(E, H, I, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    for e in (0, E - 1):
        gate_up[e] = torch.randn(2 * I, H, generator=gen, device="cuda") / H ** 0.5
        down[e] = torch.randn(H, I, generator=gen, device="cuda") / I ** 0.5
    assert (E - 1) * 2 * I * H * 2 > 2 ** 32
    x = torch.randn(3, H, generator=gen, device="cuda").bfloat16()
    ids = torch.tensor([[E - 1, 0], [E - 1, 1], [0, E - 1]], dtype=torch.int32, device="cuda")
    weights = torch.rand(3, 2, generator=gen, device="cuda")
    y = EpExperts(gate_up, down, top_k=2)(x, ids, weights)
    want = moe_ref.experts(x, torch.where(ids == E - 1, 1, torch.where(ids == 0, 0, -1)), weights,
                           gate_up[[0, E - 1]].double(), down[[0, E - 1]].double())
    moe_ref.close(y, *want, moe_ref.U_BF16)


@pytest.mark.parametrize("group", [0, 32])
def test_refusals(cuda_device, group):
    x, ids, weights, w, _ = _case(6, 256, 128, 4, 2, group)
    experts = EpExperts(*w, top_k=2, max_tokens=6)
    for bad in ((x.half(), ids, weights), (x, ids.long(), weights), (x, ids, weights.double()), (x, ids[:5], weights),
                (x, ids, weights[:, :1]), (x[:, :128], ids, weights), (x.cpu(), ids, weights), (x, ids.t(), weights)):
        with pytest.raises(ValueError):
            experts(*bad)
    with pytest.raises(ValueError):
        experts(x, ids, weights, out=torch.empty(5, 256, dtype=torch.bfloat16, device="cuda"))
    more = torch.cat([x, x]), torch.cat([ids, ids]), torch.cat([weights, weights])
    with pytest.raises(EpError, match="max_tokens"):
        experts(*more)
    with pytest.raises(EpError, match="x_stride|x: stride"):
        experts(torch.zeros(6, 260, dtype=torch.bfloat16, device="cuda")[:, :256], ids, weights)
    with pytest.raises((ValueError, EpError)):
        EpExperts(w[0], w[0], top_k=2)
    with pytest.raises(ValueError):
        EpExperts(w[0], torch.zeros(1, device="cuda") if group else Int4Weight(*moe_ref.make_int4(
            torch.Generator(device="cuda"), 4, 256, 128)), top_k=2)
    experts(x, ids, weights)
    experts.destroy()
    with pytest.raises(EpError) as ei:
        experts(x, ids, weights)
    assert ei.value.status == ep.EP_ERR_STATE


# ---- linear ---------------------------------------------------------------------------


@pytest.mark.parametrize("T,N,K,group,zeros,dtype,scales", [
    (1, 1, 32, 32, False, torch.bfloat16, torch.bfloat16), (1, 128, 128, 128, True, torch.float16, torch.float16),
    (1, 4100, 2048, 128, False, torch.bfloat16, torch.bfloat16), (2, 77, 96, 32, True, torch.bfloat16, torch.float16),
    (7, 300, 1984, 64, True, torch.float16, torch.bfloat16), (8, 129, 640, 128, False, torch.bfloat16, torch.bfloat16),
    (9, 1000, 416, 32, True, torch.bfloat16, torch.bfloat16), (16, 257, 384, 64, False, torch.float16, torch.bfloat16),
    (24, 640, 1088, 64, True, torch.bfloat16, torch.bfloat16), (25, 96, 4224, 128, True, torch.bfloat16, torch.bfloat16),
    (32, 511, 256, 128, False, torch.float16, torch.float16), (33, 200, 608, 32, True, torch.bfloat16, torch.bfloat16),
    (47, 1300, 1056, 32, False, torch.float16, torch.bfloat16), (64, 384, 2304, 64, True, torch.bfloat16, torch.bfloat16)])
def test_linear_matches_the_64_bit_form(cuda_device, T, N, K, group, zeros, dtype, scales):
    gen = torch.Generator(device="cuda").manual_seed(T + N)
    raw = moe_ref.make_int4(gen, N, K, group=group, zeros=zeros, dtype=scales)
    x = torch.randn(T, K, generator=gen, device="cuda").to(dtype)
    linear = Int4Linear(Int4Weight(*raw), max_tokens=64)
    want = moe_ref.linear(x, moe_ref.dequant(*raw))
    y = linear(x)
    assert y.dtype is dtype
    moe_ref.close(y, *want, moe_ref.U_BF16 if dtype is torch.bfloat16 else moe_ref.U_FP16)
    assert torch.equal(linear(x), y)


def test_linear_special_values(cuda_device):
    """Extreme codes, zero points and scales; zeros, infinities and NaN in one token only."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    N, K = 200, 256
    codes, s, z = moe_ref.make_int4(gen, N, K, group=64, zeros=True)
    codes[:8], codes[8:16], z[:4], z[4:8] = 0xFF, 0x00, 0, 15
    s[16:20], s[20:24], s[24:28] = 0.0, -0.5, 1e30
    x = torch.randn(12, K, generator=gen, device="cuda").bfloat16()
    linear = Int4Linear(Int4Weight(codes, s, z))
    want = moe_ref.linear(x, moe_ref.dequant(codes, s, z))
    moe_ref.close(linear(x), *want, moe_ref.U_BF16)
    bad = x.clone()
    bad[3], bad[5, 7], bad[6] = float("nan"), float("inf"), 0.0
    y, clean = linear(bad), linear(x)
    keep = [0, 1, 2, 4, 7, 8, 9, 10, 11]
    assert torch.equal(y[keep], clean[keep])
    assert bool(y[3].isnan().all()) and not bool(y[5].isfinite().any()) and bool((y[6] == 0).all())


def test_linear_layouts_graph_and_refusals(cuda_device):
    gen = torch.Generator(device="cuda").manual_seed(4)
    raw = moe_ref.make_int4(gen, 333, 512, group=128)
    linear = Int4Linear(Int4Weight(*raw), max_tokens=20)
    x = torch.randn(20, 512, generator=gen, device="cuda").bfloat16()
    want = linear(x)
    assert linear(x[:0]).shape == (0, 333)
    wide = torch.zeros(20, 1536, dtype=torch.bfloat16, device="cuda")
    wide[:, 512:1024] = x
    out = torch.zeros(20, 340, dtype=torch.bfloat16, device="cuda")
    linear(wide[:, 512:1024], out=out[:, 5:338])
    assert torch.equal(out[:, 5:338], want) and bool((out[:, :5] == 0).all()) and bool((out[:, 338:] == 0).all())
    static = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = linear(static)
    static.copy_(x.flip(0))
    graph.replay()
    assert torch.equal(y, want.flip(0))
    for bad in (x.float(), x[:, :256], x.cpu(), x.t()):
        with pytest.raises(ValueError):
            linear(bad)
    with pytest.raises(EpError, match="max_tokens"):
        linear(torch.cat([x, x]))
    codes, s, _ = raw
    for args in ((codes.int(), s), (codes, s.float()), (codes, s[:, :3]), (codes, s, s), (codes, s[:100]), (codes.t(), s)):
        with pytest.raises(ValueError):
            Int4Weight(*args)
    with pytest.raises(ValueError):
        Int4Linear(codes)


# ---- whole layer ------------------------------------------------------------------------


@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("T", [1, 11, 64])
def test_layer_is_router_then_experts(cuda_device, group, T):
    x, _, _, w, exact = _case(T, 384, 256, 16, 4, group, seed=T)
    gen = torch.Generator(device="cuda").manual_seed(T)
    wg = (torch.randn(16, 384, generator=gen, device="cuda") / 384 ** 0.5).bfloat16()
    router, experts = EpRouter(wg, 4), EpExperts(*w, top_k=4)
    layer = EpMoeLayer(router, experts)
    y, ids, weights = layer(x)
    for a, b in zip((ids, weights), router(x)):
        assert torch.equal(a, b)
    assert torch.equal(y, experts(x, ids, weights))
    moe_ref.close(y, *moe_ref.experts(x, ids, weights, *exact), moe_ref.U_BF16)
    assert layer(x[:0])[0].shape == (0, 384)
    out = torch.empty_like(y)
    assert layer(x, out=out)[0] is out and torch.equal(out, y)
    with pytest.raises(ValueError):
        EpMoeLayer(EpRouter(wg, 3), experts)


@pytest.mark.parametrize("group", [0, 32])
def test_layer_over_virtual_ranks(cuda_device, group):
    """Router, dispatch, each rank's experts on the rows it received, combine: the whole layer's result, but
    for the rounding of each rank's contribution."""
    ranks, per, H, E, K = 4, 5, 256, 16, 4
    x, _, _, w, exact = _case(ranks * per, H, 128, E, K, group, seed=9)
    gen = torch.Generator(device="cuda").manual_seed(9)
    wg = (torch.randn(E, H, generator=gen, device="cuda") / H ** 0.5).bfloat16()
    router = EpRouter(wg, K, "sigmoid", num_groups=4, top_groups=2)
    local = E // ranks
    part = (lambda t, r: Int4Weight(t.codes[r * local:(r + 1) * local].contiguous(),
                                    t.scales[r * local:(r + 1) * local].contiguous())) if group else \
        (lambda t, r: t[r * local:(r + 1) * local].contiguous())
    experts = [EpExperts(part(w[0], r), part(w[1], r), top_k=K, first_expert=r * local) for r in range(ranks)]
    comm = ep.EpComm(ranks, E, K, H, per, device=cuda_device)
    try:
        ids, weights = router(x)
        split = (lambda t: list(t.view(ranks, per, -1).unbind(0)))
        res = comm.dispatch(split(x), split(ids), split(weights))
        for r, buf in enumerate(comm.get_combine_input_buffer()):
            experts[r](res.hidden_states[r], res.topk_ids[r], res.topk_weights[r], out=buf)
        y = torch.cat(comm.combine())
    finally:
        comm.destroy()
    want, err = moe_ref.experts(x, ids, weights, *exact)
    parts = [moe_ref.experts(x, ids, weights, exact[0][r * local:(r + 1) * local], exact[1][r * local:(r + 1) * local],
                             r * local)[0] for r in range(ranks)]
    each = sum(p.abs() for p in parts) * moe_ref.U_BF16 * 1.01  # a rank's rows are rounded before combine adds them
    moe_ref.close(y, want, err + each, moe_ref.U_BF16)
