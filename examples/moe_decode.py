"""One decoding step of an MoE layer, as one GPU serves it and as an expert-parallel group does.

    python examples/moe_decode.py [--int4]

A few tokens per rank choose their experts (EpRouter). Each rank's rows go to
the ranks that own those experts (EpComm.dispatch), every rank computes its own
experts on what it received (EpExperts with its ids' range) into the combine
buffer, and EpComm.combine adds the ranks' rows up. The same layer as one call
on one GPU (EpMoeLayer) gives the same result but for one rounding per rank.
A 4-bit projection (Int4Linear) follows. The step is captured in a CUDA graph
and replayed. Weights and tokens are random.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from combine_topk_ids_dest_gb300 import (EpComm, EpExperts, EpMoeLayer, EpRouter, Int4Linear,  # noqa: E402
                                         Int4Weight)


def random_int4(gen, *shape, group=128):
    """Random 4-bit weights [..., rows, cols] whose products keep the size of their inputs."""
    *lead, cols = shape
    codes = torch.randint(0, 256, (*lead, cols // 2), dtype=torch.uint8, device="cuda", generator=gen)
    scales = torch.rand((*lead, cols // group), device="cuda", generator=gen) * 0.4 / cols ** 0.5
    return Int4Weight(codes, scales.bfloat16())


def random_bf16(gen, *shape):
    return (torch.randn(shape, device="cuda", generator=gen) / shape[-1] ** 0.5).bfloat16()


def part(w, first, n):
    """Experts first .. first + n - 1 of a weight [experts, rows, cols]."""
    if isinstance(w, Int4Weight):
        return Int4Weight(w.codes[first:first + n], w.scales[first:first + n])
    return w[first:first + n]


def main(int4=False, ranks=4, tokens=16, experts=32, top_k=8, hidden=2048, intermediate=768, vocabulary=8000):
    gen = torch.Generator("cuda").manual_seed(1)
    make = random_int4 if int4 else random_bf16
    gate_up, down = make(gen, experts, 2 * intermediate, hidden), make(gen, experts, hidden, intermediate)
    router = EpRouter(random_bf16(gen, experts, hidden), top_k, scoring="sigmoid", num_groups=4, top_groups=2,
                      bias=0.1 * torch.randn(experts, device="cuda", generator=gen), scale=2.5)
    head = Int4Linear(random_int4(gen, vocabulary, hidden))
    x = torch.randn((ranks * tokens, hidden), device="cuda", generator=gen).bfloat16()

    # one GPU: router and all experts in one call, at most 64 tokens
    layer = EpMoeLayer(router, EpExperts(gate_up, down, top_k, max_tokens=ranks * tokens))
    y, ids, weights = layer(x)

    # the expert-parallel group: rank r owns experts r * local ..
    local = experts // ranks
    comm = EpComm(ranks, experts, top_k, hidden, tokens, device="cuda")
    owned = [EpExperts(part(gate_up, r * local, local), part(down, r * local, local), top_k,
                       max_tokens=ranks * tokens, first_expert=r * local) for r in range(ranks)]
    rows = [slice(r * tokens, (r + 1) * tokens) for r in range(ranks)]

    def step():
        ids, weights = router(x)  # of all ranks' tokens; a rank's own router would see its rows
        got = comm.dispatch([x[s] for s in rows], [ids[s] for s in rows], [weights[s] for s in rows])
        for r, out in enumerate(comm.get_combine_input_buffer()):
            owned[r](got.hidden_states[r], got.topk_ids[r], got.topk_weights[r], out=out)
        z = torch.cat(comm.combine())
        return z, head(z)

    z, logits = step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z2, logits2 = step()
    graph.replay()
    torch.cuda.synchronize()
    off = ((z.double() - y.double()).norm() / y.double().norm()).item()
    print(f"{'4-bit' if int4 else 'bf16'} experts, {ranks} ranks x {tokens} tokens: ranks against one GPU {off:.1e}, "
          f"replay {'equal' if torch.equal(z, z2) and torch.equal(logits, logits2) else 'different'}, "
          f"next tokens {logits[:4].argmax(-1).tolist()}")
    comm.destroy()
    return off, torch.equal(z, z2) and torch.equal(logits, logits2)


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--int4", action="store_true", help="4-bit experts instead of bf16")
    main(ap.parse_args().int4)
