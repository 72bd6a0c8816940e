"""A block as it is used: norm, router, dispatch of 8-bit rows, the routed experts, the shared expert, and the next norm."""
import pytest
import torch

import block_ref
import moe_ref
from combine_topk_ids_dest_gb300 import EpComm, EpExperts, EpFfn, EpMoeLayer, EpNorm, EpRouter

pytestmark = pytest.mark.gpu
E, K, H, I, SHARED, EPS = 16, 4, 512, 256, 768, 1e-5


def _weights(gen):
    def w(*shape):
        return (torch.randn(shape, generator=gen, device="cuda") / shape[-1] ** 0.5).bfloat16()

    return dict(gate=w(E, H), gate_up=w(E, 2 * I, H), down=w(E, H, I), shared_up=w(2 * SHARED, H), shared_down=w(H, SHARED),
                before=(1 + 0.1 * torch.randn(H, generator=gen, device="cuda")).bfloat16(),
                after=(1 + 0.1 * torch.randn(H, generator=gen, device="cuda")).bfloat16())


def test_block_with_a_shared_expert(cuda_device):
    gen = torch.Generator("cuda").manual_seed(1)
    w = _weights(gen)
    x, residual = (torch.randn(48, H, generator=gen, device="cuda").bfloat16() for _ in range(2))
    before, after = EpNorm(w["before"], eps=EPS), EpNorm(w["after"], eps=EPS)
    layer = EpMoeLayer(EpRouter(w["gate"], K), EpExperts(w["gate_up"], w["down"], K))
    shared = EpFfn(w["shared_up"], w["shared_down"])

    def step(x, residual):
        n = before(x, residual)
        y, ids, weights = layer(n.out)
        return n, y, ids, weights, shared(n.out), after(y, n.residual)

    n, y, ids, weights, z, last = step(x, residual)
    s, want = block_ref.norm(x, residual, w["before"], EPS)
    block_ref.check(n.out, want, block_ref.NORM * want.abs(), "norm")
    want, err = moe_ref.experts(n.out, ids, weights, w["gate_up"].double(), w["down"].double())
    moe_ref.close(y, want, err, block_ref.U)
    want, err, _ = block_ref.ffn(n.out, w["shared_up"], w["shared_down"])
    block_ref.check(z, want, err, "shared expert")
    _, want = block_ref.norm(y, n.residual, w["after"], EPS)
    block_ref.check(last.out, want, block_ref.NORM * want.abs(), "next norm")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = step(x, residual)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in ((again[1], y), (again[4], z), (again[5].out, last.out), (again[5].residual, last.residual)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("hidden", [512, 7168])
def test_rows_in_8_bits_are_what_a_dispatch_carries(cuda_device, hidden):
    """q and scales go into EpComm.dispatch as they are, and arrive at the rows of every rank that owns a chosen expert."""
    ranks, tokens = 4, 24
    gen = torch.Generator("cuda").manual_seed(2)
    x = torch.randn(ranks * tokens, hidden, generator=gen, device="cuda").bfloat16()
    norm = EpNorm((1 + 0.1 * torch.randn(hidden, generator=gen, device="cuda")).bfloat16())
    router = EpRouter((torch.randn(E, hidden, generator=gen, device="cuda") / hidden ** 0.5).bfloat16(), K)
    n = norm(x, quantized=True)
    ids, weights = router(n.out)
    comm = EpComm(ranks, E, K, hidden, tokens, dtype=torch.float8_e4m3fn, device="cuda")
    rows = [slice(r * tokens, (r + 1) * tokens) for r in range(ranks)]
    got = comm.dispatch([n.q[s] for s in rows], [ids[s] for s in rows], [weights[s] for s in rows],
                        hidden_states_scale=[n.scales[s] for s in rows])
    torch.cuda.synchronize()
    for d in range(ranks):
        here = ((ids >= d * E // ranks) & (ids < (d + 1) * E // ranks)).any(1)
        q = got.hidden_states[d].view(torch.uint8).view(ranks * tokens, hidden)
        assert torch.equal(q[here], n.q.view(torch.uint8)[here])
        assert torch.equal(got.hidden_states_scale[d].view(ranks * tokens, -1)[here], n.scales[here])
    comm.destroy()


def test_training_step_of_a_dense_layer(cuda_device):
    """Norm, block and residual stream forward and backward: the gradients of the whole against 64 bits."""
    T = 200
    gen = torch.Generator("cuda").manual_seed(3)
    w = _weights(gen)
    x, residual, dz = (torch.randn(T, H, generator=gen, device="cuda").bfloat16() for _ in range(3))
    dz = (dz * 0.1).bfloat16()
    norm, ffn = EpNorm(w["before"], eps=EPS), EpFfn(w["shared_up"], w["shared_down"])
    n = norm(x, residual)
    y, saved = ffn.forward(n.out)
    dn, dup, ddown = ffn.backward(dz, n.out, saved)  # z = y + residual stream: dz reaches both
    dx, dweight = norm.backward(dn, n.residual, dz)
    leaves = [t.double().requires_grad_() for t in (x, residual, w["before"], w["shared_up"], w["shared_down"])]
    s = leaves[0] + leaves[1]
    h = s / (s.square().mean(1, keepdim=True) + EPS).sqrt() * leaves[2]
    a = h @ leaves[3].t()
    z = (torch.nn.functional.silu(a[:, :SHARED]) * a[:, SHARED:]) @ leaves[4].t() + s
    want = torch.autograd.grad(z, leaves, dz.double())
    assert torch.equal(want[0], want[1])
    # bf16 roundings between the operators (s, n, h, the gradients of g and u, dn, the result): six of half a step each,
    # independent of one another, so far below their sum in the norm of a whole tensor
    for name, got, ref in (("dx", dx, want[0]), ("dweight", dweight, want[2]), ("dgate_up", dup, want[3]), ("ddown", ddown, want[4])):
        off = ((got.double() - ref).norm() / ref.norm()).item()
        assert off < 6 * block_ref.U, (name, off)
