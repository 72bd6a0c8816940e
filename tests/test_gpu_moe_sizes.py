"""MoE operators at sizes where their plans of tiles, splits and shared memory change, against the
64-bit forms."""
import pytest
import torch

from combine_topk_ids_dest_gb300 import EpRouter
from test_gpu_moe_router import _check, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H", [(1152, 1024), (1153, 1024), (1200, 7168), (1300, 7168), (1389, 1024), (1450, 2048), (1621, 1024),
                                 (1768, 1024), (1945, 1024), (2100, 520), (2161, 1024), (2750, 1024), (3242, 1024),
                                 (3891, 1024), (6450, 1024), (6485, 7168), (9728, 1024), (9729, 1024)])
def test_router_where_the_number_of_splits_changes(cuda_device, T, H):
    x, w, b = _inputs(T, H, 256, seed=T, bias=True)
    router = EpRouter(w, 8, "sigmoid", bias=b, num_groups=8, top_groups=4, scale=2.5)
    assert _check(router, x, w, b, 8, "sigmoid", 8, 4, scale=2.5) > 0.5
