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
