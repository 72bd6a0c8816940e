"""EpRouter at the ends of the scores' range, in each of its kernels: sums of 0, subnormal scores."""
import pytest
import torch

from combine_topk_ids_dest_gb300 import EpRouter

pytestmark = pytest.mark.gpu

TOKENS = [3, 40, 130, 11000]  # few (two widths), many with split inputs, many in pairs


def _logits(T, values, dtype=torch.bfloat16):
    """x and weight whose logits are exactly `values`, for every token."""
    w = torch.zeros(len(values), 8, dtype=dtype, device="cuda")
    w[:, 0] = torch.tensor(values, device="cuda")
    x = torch.zeros(T, 8, dtype=dtype, device="cuda")
    x[:, 0] = 1.0
    assert w[:, 0].tolist() == list(values)
    return x, w


@pytest.mark.parametrize("T", TOKENS)
def test_scores_of_zero_have_weights_of_zero(cuda_device, T):
    """All chosen scores are 0 in fp32: their weights are 0, not 0 / 0."""
    x, w = _logits(T, [200.0] + [0.0] * 15)
    bias = torch.zeros(16, device="cuda")
    bias[0] = -torch.inf  # the expert whose score is 1 may not be chosen; the others' are exp(-200)
    bias[5], bias[9] = 2.0, 1.0
    for router, scale in ((EpRouter(w, 4, "softmax", bias=bias), 1.0), (EpRouter(w, 4, "softmax", bias=bias, scale=2.5), 2.5)):
        ids, weights = router(x)
        assert ids.tolist() == [[5, 9, 1, 2]] * T and bool((weights == 0).all())
    x, w = _logits(T, [-200.0] * 16)
    ids, weights = EpRouter(w, 4, "sigmoid", num_groups=4, top_groups=2, scale=2.5)(x)
    assert ids.tolist() == [[0, 1, 2, 3]] * T and bool((weights == 0).all())
    x, w = _logits(T, [-200.0, -1.0, -200.0, 1.0])  # one of them is not 0
    ids, weights = EpRouter(w, 3, "sigmoid")(x)
    assert ids.tolist() == [[3, 1, 0]] * T and bool((weights[:, 2] == 0).all())
    assert torch.allclose(weights.sum(1), torch.ones(T, device="cuda"), atol=1e-6)


@pytest.mark.parametrize("T", TOKENS)
def test_subnormal_sigmoid_scores(cuda_device, T):
    """sigmoid(l) down to fp32's smallest numbers. Exponential and quotient are within 2 units each, or 2^-149 where the
    result is subnormal; the sum and the division by it add a few units more."""
    values = [-86.0 - 0.5 * e for e in range(20)]  # exp(-95.5) is 2300 times 2^-149
    x, w = _logits(T, values)
    s = torch.sigmoid(torch.tensor(values, dtype=torch.float64, device="cuda"))
    off = 8 * 2.0 ** -24 + 3 * 2.0 ** -149 / s
    order = [e for e in range(20) if e > 11][:6]
    bias = torch.zeros(20, device="cuda")
    bias[order] = torch.arange(6, 0, -1, device="cuda").float()
    for scale in (1.0, 2.5):
        ids, weights = EpRouter(w, 6, "sigmoid", bias=bias, scale=scale)(x)
        assert ids.tolist() == [order] * T
        want = s[order] / s[order].sum() * scale
        assert bool(((weights.double() - want).abs() <= want * (off[order] + off[order].max() + 8 * 2.0 ** -24)).all())
    ids, weights = EpRouter(w, 20, "sigmoid", renormalize=False)(x)
    assert ids.tolist() == [list(range(20))] * T
    assert bool(((weights.double() - s).abs() <= s * off).all())
