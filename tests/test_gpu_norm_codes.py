"""Which of two neighbouring codes a value of the norm's 8-bit rows takes."""
import pytest
import torch

from combine_topk_ids_dest_gb300 import EpNorm
from test_gpu_norm import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H", [(40000, 1024), (7, 7168), (3001, 200)])
def test_codes_are_the_nearest_of_the_quotients(cuda_device, T, H):
    """Rows in fp32 come out as they are divided: the codes are those of the fp32 quotients, exactly."""
    x, residual, w, _, _ = make(T, H, torch.float32, seed=T)
    r = EpNorm(w)(x, residual, quantized=True)
    wide = r.scales.repeat_interleave(128, 1)[:, :H]
    want = (r.out / wide).clamp(-448, 448).to(torch.float8_e4m3fn)
    differ = int((want.view(torch.uint8) != r.q.view(torch.uint8)).sum())
    assert differ == 0, f"{differ} of {T * H}"
