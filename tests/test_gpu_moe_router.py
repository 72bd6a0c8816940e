"""EpRouter against the 64-bit form: ids wherever the choice does not hang on rounding, weights
within the bound of fp32 sums, ties, masks, empty rows, layouts, streams and graphs."""
import numpy as np
import pytest
import torch

import combine_topk_ids_dest_gb300 as ep
import moe_ref
from combine_topk_ids_dest_gb300 import EpError, EpRouter

pytestmark = pytest.mark.gpu


def _inputs(T, H, E, dtype=torch.bfloat16, seed=0, bias=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, H, generator=gen, device="cuda").to(dtype)
    w = (torch.randn(E, H, generator=gen, device="cuda") * (1.5 / H ** 0.5)).to(dtype)
    b = torch.randn(E, generator=gen, device="cuda") * 0.1 if bias else None
    return x, w, b


def _check(router, x, w, b, top_k, scoring, groups, top_groups, renormalize=True, scale=1.0):
    ids, weights = router(x)
    assert ids.dtype is torch.int32 and weights.dtype is torch.float32
    l, s, es = moe_ref.scores(x, w, scoring)
    if scoring == "softmax" and b is None and groups == 1:  # ranked by the logits, like their softmax
        want, _ = moe_ref.choice(l, None, top_k)
    else:
        want, _ = moe_ref.choice(s, b, top_k, groups, top_groups)
    # a token counts where every choice value it could have mixed up is further off than the scores' errors:
    # neighbours among the top_k + 1 largest (of all experts, or of the groups that take part)
    c = s if b is None else s + b.double()
    order = moe_ref.choice(s, b, top_k, groups, top_groups)[1][:, :top_k + 1]
    near = ((order[:, :-1] - order[:, 1:]) <= 4 * es.amax(1, keepdim=True)).any(1)
    if groups > 1:
        best = torch.sort(c.view(len(x), groups, -1), dim=2, descending=True).values[:, :, :2].sum(2)
        best = torch.sort(best, dim=1, descending=True).values
        near |= ((best[:, :-1] - best[:, 1:]) <= 8 * es.amax(1, keepdim=True)).any(1)
    sure = ~near
    assert torch.equal(ids[sure].long(), want[sure])
    # whatever was chosen: distinct experts in descending order of the choice value, the weights theirs
    assert all(len(set(r)) == len(r) for r in ids.tolist())
    got_c = c.gather(1, ids.long())
    assert bool((got_c[:, :-1] - got_c[:, 1:] >= -4 * es.amax(1, keepdim=True)).all())
    exact = moe_ref.chosen_weights(s, ids.long(), renormalize, scale)
    rel = (es / s).gather(1, ids.long()).amax(1, keepdim=True)
    err = exact.abs() * (2 * rel + 16 * 2.0 ** -24)
    assert bool(((weights.double() - exact).abs() <= err + 1e-30).all())
    return float(sure.double().mean())


@pytest.mark.parametrize("T", [1, 3, 8, 9, 64, 65, 127, 300, 1217, 3001])
@pytest.mark.parametrize("scoring,bias,E,K,groups,top_groups", [
    ("softmax", False, 64, 8, 1, 1), ("sigmoid", True, 96, 6, 8, 4), ("softmax", True, 40, 3, 4, 2)])
def test_matches_the_64_bit_form(cuda_device, T, scoring, bias, E, K, groups, top_groups):
    x, w, b = _inputs(T, 520, E, seed=T, bias=bias)
    router = EpRouter(w, K, scoring, bias=b, num_groups=groups, top_groups=top_groups, scale=2.5)
    sure = _check(router, x, w, b, K, scoring, groups, top_groups, scale=2.5)
    assert T < 100 or sure > 0.5


@pytest.mark.parametrize("T,H,E,K,groups,top_groups,dtype", [
    (5, 8, 1, 1, 1, 1, torch.bfloat16), (70, 16, 2, 2, 1, 1, torch.float16), (33, 1024, 257, 32, 1, 1, torch.bfloat16),
    (500, 1024, 257, 32, 1, 1, torch.float16), (400, 264, 384, 9, 32, 7, torch.bfloat16), (20000, 64, 12, 2, 3, 2, torch.bfloat16),
    (300, 328, 512, 10, 16, 4, torch.bfloat16), (12, 7168, 256, 8, 8, 4, torch.bfloat16), (129, 72, 17, 1, 1, 1, torch.float16),
    (9800, 200, 64, 4, 32, 5, torch.bfloat16)])
def test_sizes_and_types(cuda_device, T, H, E, K, groups, top_groups, dtype):
    x, w, _ = _inputs(T, H, E, dtype, seed=7)
    for renormalize in (True, False):
        router = EpRouter(w, K, "sigmoid", num_groups=groups, top_groups=top_groups, renormalize=renormalize)
        _check(router, x, w, None, K, "sigmoid", groups, top_groups, renormalize)


@pytest.mark.parametrize("T", [2, 40, 200, 12000])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_equal_experts_tie_to_the_lowest_index(cuda_device, T, scoring):
    x, w, _ = _inputs(T, 256, 4, seed=3)
    router = EpRouter(w.repeat(8, 1).contiguous(), 16, scoring)  # experts e, e + 4, ... are the same
    ids, weights = router(x)
    l = moe_ref.scores(x, w, scoring)[0]
    gap = torch.sort(l, dim=1, descending=True).values
    sure = ((gap[:, :-1] - gap[:, 1:]) > 1e-3).all(1)
    order = torch.sort(l, dim=1, descending=True).indices[:, :2]
    want = torch.cat([order[:, :1] + 4 * torch.arange(8, device="cuda"), order[:, 1:] + 4 * torch.arange(8, device="cuda")], 1)
    assert torch.equal(ids[sure].long(), want[sure])
    assert torch.equal(weights[:, 0], weights[:, 7])


@pytest.mark.parametrize("T", [3, 130, 11000])
@pytest.mark.parametrize("groups", [1, 4])
def test_masked_experts_are_never_chosen(cuda_device, T, groups):
    x, w, _ = _inputs(T, 128, 16, seed=5)
    bias = torch.full((16,), -torch.inf, device="cuda")
    bias[[2, 7, 9]] = 0.0
    bias[9] = float("nan")  # neither is a NaN
    ids, weights = EpRouter(w, 4, "sigmoid", bias=bias, num_groups=groups, top_groups=groups)(x)
    assert set(ids[:, :2].flatten().tolist()) == {2, 7}
    assert bool((ids[:, 2:] == -1).all()) and bool((weights[:, 2:] == 0).all())
    assert torch.allclose(weights.sum(1), torch.ones(T, device="cuda"), atol=1e-6)
    ids, weights = EpRouter(w, 4, "softmax", bias=torch.full_like(bias, -torch.inf))(x)
    assert bool((ids == -1).all()) and bool((weights == 0).all())


@pytest.mark.parametrize("T", [4, 300, 10000])
def test_rows_with_nan_keep_to_themselves(cuda_device, T):
    x, w, _ = _inputs(T, 256, 32, seed=6)
    router = EpRouter(w, 4)
    clean = router(x)
    bad = x.clone()
    bad[1] = float("nan")
    ids, weights = router(bad)
    keep = torch.arange(T, device="cuda") != 1
    assert torch.equal(ids[keep], clean[0][keep]) and torch.equal(weights[keep], clean[1][keep])
    assert bool((ids[1] == -1).all()) and bool((weights[1] == 0).all())


def test_no_rows_and_strided_rows(cuda_device):
    x, w, _ = _inputs(70, 128, 16, seed=8)
    router = EpRouter(w, 4)
    ids, weights = router(x[:0])
    assert ids.shape == weights.shape == (0, 4)
    wide = torch.zeros(70, 3, 128, dtype=torch.bfloat16, device="cuda")
    wide[:, 1] = x
    for n in (5, 70):
        for a, b in zip(router(wide[:n, 1]), router(x[:n])):
            assert torch.equal(a, b)


def test_repeats_are_bit_equal_on_streams_and_in_graphs(cuda_device):
    for T in (1, 64, 200, 11000):
        x, w, _ = _inputs(T, 512, 48, seed=9)
        router = EpRouter(w, 6, "sigmoid")
        want = router(x)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for a, b in zip(router(x), want):
                assert torch.equal(a, b)
        side.synchronize()
        static = x.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = router(static)
        static.copy_(x.flip(0))
        graph.replay()
        for a, b in zip(got, want):
            assert torch.equal(a, b.flip(0))


def test_refusals(cuda_device):
    x, w, _ = _inputs(8, 64, 16)
    router = EpRouter(w, 2)
    for bad in (x.half(), x[:, :32], x.cpu(), x.t(), x[0]):
        with pytest.raises(ValueError):
            router(bad)
    with pytest.raises(EpError) as ei:  # rows 72 elements apart are fine, 68 are not 16-byte aligned
        router(torch.zeros(8, 68, dtype=torch.bfloat16, device="cuda")[:, :64])
    assert ei.value.status == ep.EP_ERR_INVALID_ARG
    with pytest.raises(EpError):
        router(torch.zeros(8 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(8, 64))
    router(x)  # still usable
    router.destroy()
    router.destroy()
    with pytest.raises(EpError) as ei:
        router(x)
    assert ei.value.status == ep.EP_ERR_STATE
    with pytest.raises(ValueError):
        EpRouter(w, 2, scoring="relu")
    with pytest.raises(EpError):
        EpRouter(w, 17)


def test_choices_feed_dispatch(cuda_device):
    """ids and weights go to EpComm.dispatch as they are; slots without an expert route nowhere."""
    x, w, _ = _inputs(24, 256, 8, seed=11)
    bias = torch.zeros(8, device="cuda")
    bias[4:] = -torch.inf  # the second rank's experts
    ids, weights = EpRouter(w, 6, "sigmoid", bias=bias)(x)
    comm = ep.EpComm(2, 8, 6, 256, 12, device=cuda_device)
    try:
        res = comm.dispatch([x[:12], x[12:]], [ids[:12], ids[12:]], [weights[:12], weights[12:]])
        assert torch.equal(res.topk_ids[0], ids) and bool((res.topk_ids[1] == -1).all())
        assert np.array_equal(res.hidden_states[0].view(torch.int16).cpu().numpy(), x.view(torch.int16).cpu().numpy())
        comm.combine()
    finally:
        comm.destroy()
