"""The same call again gives the same bits: the 4-bit kernel where its rings have few stages, and each stage of an
expert-parallel decoding step, eager and replayed, so that a difference names the stage."""
import pytest
import torch

import moe_ref
from combine_topk_ids_dest_gb300 import EpComm, EpExperts, EpRouter, Int4Linear, Int4Weight

pytestmark = pytest.mark.gpu


def _same(a, b):
    """Equal bits, NaN included."""
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def _differ(first, call, times):
    """How many of `times` further calls differ from the first; other data passes through L2 in between."""
    flush = torch.empty(160 << 20, dtype=torch.uint8, device="cuda")
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(times):
        if i % 4 == 0:
            flush.fill_(i & 255)
        differ += (call().view(torch.int16) != first.view(torch.int16)).any()
    return int(differ)


@pytest.mark.parametrize("T,N,K", [(64, 8000, 2048), (33, 1000, 4096), (24, 7168, 1024), (16, 2056, 2048), (3, 4096, 2048)])
def test_linear_again(cuda_device, T, N, K):
    gen = torch.Generator(device="cuda").manual_seed(T)
    raw = moe_ref.make_int4(gen, 1, N, K, group=128)
    codes, scales = raw[0][0], raw[1][0]
    x = torch.randn(T, K, generator=gen, device="cuda").bfloat16()
    call = Int4Linear(Int4Weight(codes, scales))
    y = call(x)
    moe_ref.close(y, *moe_ref.linear(x, moe_ref.dequant(codes, scales)), moe_ref.U_BF16)
    assert _differ(y, lambda: call(x), 200) == 0


@pytest.mark.parametrize("T,E,most", [(64, 32, 0), (64, 8, 0), (40, 8, 0), (16, 16, 0), (8, 8, 0), (48, 6, 32), (24, 4, 24)])
def test_experts_again(cuda_device, T, E, most):
    """most: as many tokens for expert 0, the others' choices at random."""
    H, I, K = 1024, 384, min(8, E)
    gen = torch.Generator(device="cuda").manual_seed(T + E)
    raw = [moe_ref.make_int4(gen, E, r, c, group=128) for r, c in ((2 * I, H), (H, I))]
    ids = torch.rand(T, E, generator=gen, device="cuda").argsort(1)[:, :K].int().contiguous()
    if most:
        ids = torch.randint(1, E, (T, 1), generator=gen, device="cuda", dtype=torch.int32)
        ids[:most] = 0
        K = 1
    x = torch.randn(T, H, generator=gen, device="cuda").bfloat16()
    weights = torch.rand(T, K, generator=gen, device="cuda") + 0.1
    call = EpExperts(*[Int4Weight(*r) for r in raw], top_k=K)
    y = call(x, ids, weights)
    moe_ref.close(y, *moe_ref.experts(x, ids, weights, *[moe_ref.dequant(*r) for r in raw]), moe_ref.U_BF16)
    assert _differ(y, lambda: call(x, ids, weights), 200) == 0


def test_every_stage_of_a_replayed_step(cuda_device):
    ranks, tokens, E, K, H, I = 4, 16, 32, 8, 2048, 768
    gen = torch.Generator(device="cuda").manual_seed(7)
    weights4 = [Int4Weight(*moe_ref.make_int4(gen, E, r, c, group=128)) for r, c in ((2 * I, H), (H, I))]
    router = EpRouter((torch.randn(E, H, generator=gen, device="cuda") / H ** 0.5).bfloat16(), K, scoring="sigmoid")
    raw = moe_ref.make_int4(gen, 1, 4000, H, group=128)
    head = Int4Linear(Int4Weight(raw[0][0], raw[1][0]))
    x = torch.randn(ranks * tokens, H, generator=gen, device="cuda").bfloat16()
    comm, local = EpComm(ranks, E, K, H, tokens, device="cuda"), E // ranks
    owned = [EpExperts(*[Int4Weight(w.codes[r * local:(r + 1) * local], w.scales[r * local:(r + 1) * local]) for w in weights4],
                       top_k=K, max_tokens=ranks * tokens, first_expert=r * local) for r in range(ranks)]

    def step():
        ids, weights = router(x)
        out = dict(ids=ids, weights=weights)
        got = comm.dispatch(*([t[r * tokens:(r + 1) * tokens] for r in range(ranks)] for t in (x, ids, weights)))
        for r, y in enumerate(comm.get_combine_input_buffer()):
            chosen = got.topk_ids[r].clone()
            there = ((chosen >= r * local) & (chosen < (r + 1) * local)).any(1, keepdim=True)
            out[f"ids of rank {r}"] = chosen
            out[f"rows of rank {r}"] = torch.where(there, got.hidden_states[r], torch.zeros_like(got.hidden_states[r]))
            owned[r](got.hidden_states[r], got.topk_ids[r], got.topk_weights[r], out=y)
            out[f"experts of rank {r}"] = torch.where(there, y, torch.zeros_like(y))
        out["combined"] = torch.cat(comm.combine())
        out["logits"] = head(out["combined"])
        return out

    want = step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(30):
        graph.replay()
        differ = [name for name, t in got.items() if not _same(t, want[name])]
        assert differ == [], differ
    again = step()
    differ = [name for name, t in again.items() if not _same(t, want[name])]
    comm.destroy()
    assert differ == [], differ
