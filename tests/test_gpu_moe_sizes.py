"""MoE operators at sizes where their plans of tiles, splits and shared memory change, against the
64-bit forms."""
import pytest
import torch

import moe_ref
from combine_topk_ids_dest_gb300 import EpRouter
from test_gpu_moe_experts import _case, _check as _check_experts
from test_gpu_moe_router import _check, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H", [(1152, 1024), (1153, 1024), (1200, 7168), (1300, 7168), (1389, 1024), (1450, 2048), (1621, 1024),
                                 (1768, 1024), (1945, 1024), (2100, 520), (2161, 1024), (2750, 1024), (3242, 1024),
                                 (3891, 1024), (6450, 1024), (6485, 7168), (9728, 1024), (9729, 1024)])
def test_router_where_the_number_of_splits_changes(cuda_device, T, H):
    x, w, b = _inputs(T, H, 256, seed=T, bias=True)
    router = EpRouter(w, 8, "sigmoid", bias=b, num_groups=8, top_groups=4, scale=2.5)
    assert _check(router, x, w, b, 8, "sigmoid", 8, 4, scale=2.5) > 0.5


@pytest.mark.parametrize("T,E,K,group,zeros", [(64, 512, 32, 32, True), (64, 512, 22, 32, True), (58, 504, 32, 32, False),
                                               (64, 384, 26, 64, True), (64, 512, 29, 128, False), (63, 257, 32, 0, False),
                                               (64, 512, 32, 0, False)])
def test_experts_with_long_lists(cuda_device, T, E, K, group, zeros):
    """Lists, sums and rings at their largest: experts of 64 tokens (two entries), of 25 to 32, of a few."""
    gen = torch.Generator(device="cuda").manual_seed(K)
    ids = torch.rand(T, E, generator=gen, device="cuda").argsort(1)[:, :K].int()
    ids[:, :4] = torch.tensor([0, E - 1, E // 2, 3], device="cuda")
    ids[: T // 2, 4] = 5
    _check_experts(*_case(T, 128 if group == 128 else 192, 128 if group else 136, E, K, group, zeros, seed=E + K, ids=ids))


@pytest.mark.parametrize("group", [0, 32])
def test_experts_at_the_end_of_the_ids(cuda_device, group):
    first = 2**31 - 6
    gen = torch.Generator(device="cuda").manual_seed(3)
    ids = torch.randint(first, 2**31, (9, 4), generator=gen, device="cuda").int()
    ids[0] = torch.tensor([-2**31, -2**31 + 5, -1, 0], device="cuda")  # nothing here
    ids[1] = torch.tensor([-2**31, 2**31 - 1, first - 1, first], device="cuda")
    case = _case(9, 192, 160, 6, 4, group, ids=ids, seed=5)
    _, y = _check_experts(*case, first=first)
    assert bool((y[0] == 0).all()) and bool((y[1] != 0).any())


@pytest.mark.parametrize("T,H,E,K,scoring,bias,groups,top_groups,dtype", [
    (10000, 264, 160, 8, "sigmoid", True, 8, 4, torch.bfloat16), (9800, 520, 256, 8, "softmax", True, 1, 1, torch.float16),
    (9900, 264, 256, 8, "softmax", False, 8, 3, torch.bfloat16), (10001, 264, 257, 6, "sigmoid", True, 1, 1, torch.bfloat16),
    (9999, 200, 384, 10, "sigmoid", True, 24, 7, torch.float16), (9999, 200, 384, 32, "softmax", True, 1, 1, torch.bfloat16),
    (12000, 72, 384, 8, "softmax", False, 32, 5, torch.bfloat16), (9800, 264, 300, 4, "softmax", False, 1, 1, torch.float16),
    (30000, 128, 384, 4, "softmax", True, 12, 5, torch.bfloat16)])
def test_router_for_many_tokens_and_experts(cuda_device, T, H, E, K, scoring, bias, groups, top_groups, dtype):
    """Two blocks that multiply together: one instruction up to 256 experts, two above."""
    x, w, b = _inputs(T, H, E, dtype, seed=E, bias=bias)
    router = EpRouter(w, K, scoring, bias=b, num_groups=groups, top_groups=top_groups, scale=2.5)
    _check(router, x, w, b, K, scoring, groups, top_groups, scale=2.5)


@pytest.mark.parametrize("T", [3, 64, 65, 257, 700])
@pytest.mark.parametrize("E,K,scoring,bias,groups,top_groups", [
    (385, 8, "sigmoid", True, 1, 1), (449, 5, "softmax", True, 1, 1), (512, 8, "sigmoid", True, 32, 9),
    (512, 32, "softmax", False, 8, 3), (400, 8, "softmax", False, 1, 1)])
def test_router_of_more_than_384_experts(cuda_device, T, E, K, scoring, bias, groups, top_groups):
    x, w, b = _inputs(T, 520, E, seed=E + T, bias=bias)
    router = EpRouter(w, K, scoring, bias=b, num_groups=groups, top_groups=top_groups)
    _check(router, x, w, b, K, scoring, groups, top_groups)


@pytest.mark.parametrize("T", [40, 300, 10000])
def test_equal_and_masked_experts_among_384(cuda_device, T):
    x, w, _ = _inputs(T, 256, 4, seed=3)
    ids, weights = EpRouter(w.repeat(96, 1).contiguous(), 16, "sigmoid")(x)  # experts e, e + 4, ... are the same
    l = moe_ref.scores(x, w, "sigmoid")[0]
    gap = torch.sort(l, dim=1, descending=True).values
    sure = (gap[:, 0] - gap[:, 1]) > 1e-3
    want = l.argmax(1)[:, None] + 4 * torch.arange(16, device="cuda")
    assert torch.equal(ids[sure].long(), want[sure]) and torch.equal(weights[sure, 0], weights[sure, 15])
    x, w, _ = _inputs(T, 256, 384, seed=4)
    bias = torch.full((384,), -torch.inf, device="cuda")
    left = [1, 127, 128, 255, 256, 383]
    bias[left] = 0.0
    ids, weights = EpRouter(w, 8, "sigmoid", bias=bias)(x)
    assert bool((ids[:, :6].sort(1).values == torch.tensor(left, device="cuda")).all())
    assert bool((ids[:, 6:] == -1).all()) and bool((weights[:, 6:] == 0).all())
