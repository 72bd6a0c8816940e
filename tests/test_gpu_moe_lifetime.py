"""MoE handles that go while calls on another stream are queued: the calls finish first."""
import pytest
import torch

import moe_ref
from combine_topk_ids_dest_gb300 import EpExperts, EpRouter, Int4Linear, Int4Weight
from test_gpu_moe_experts import _case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["router", "dense", "int4", "linear"])
def test_memory_is_given_back_after_queued_calls(cuda_device, kind):
    x, ids, weights, w, _ = _case(40, 256, 320, 6, 3, 64 if kind == "int4" else 0, seed=4)
    gen = torch.Generator(device="cuda").manual_seed(1)
    if kind == "router":
        handle = EpRouter((torch.randn(48, 256, generator=gen, device="cuda") / 16).bfloat16(), 4)
        call = lambda h: h(x)[1]  # noqa: E731
    elif kind == "linear":
        handle = Int4Linear(Int4Weight(*moe_ref.make_int4(gen, 333, 256)))
        call = lambda h: h(x)  # noqa: E731
    else:
        handle = EpExperts(*w, top_k=3)
        call = lambda h: h(x, ids, weights)  # noqa: E731
    want = call(handle)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)  # some 25 ms
        got = call(handle)
    assert not side.query()
    del handle, call
    assert side.query()
    assert torch.equal(got, want)
