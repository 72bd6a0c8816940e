"""The feed-forward block where it can go wrong: strides, rows that are not finite, what is not asked for, gradients in fp32 and
added up, weights that change, graphs, streams, offsets past 32 bits, refusals."""
import pytest
import torch

import block_ref
from combine_topk_ids_dest_gb300 import EP_ERR_INVALID_ARG, EpError, EpFfn
from test_gpu_ffn import make

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("T,H,I", [(3, 136, 72), (130, 264, 520), (700, 1024, 9000)])
def test_strides_and_rows_beside(cuda_device, T, H, I):
    """Rows of wider buffers, results at odd places too, give the same; what lies beside stays as it was."""
    x, gate_up, down, dy = make(T, H, I, seed=2)
    ffn = EpFfn(gate_up, down)
    y, saved = ffn.forward(x)
    grads = ffn.backward(dy, x, saved)
    for pad in (8, 40):
        wide = torch.full((T + 3, H + pad), float("nan"), dtype=BF16, device="cuda")
        wide[:T, :H] = x
        wdy = torch.full((T + 3, H + pad), float("nan"), dtype=BF16, device="cuda")
        wdy[:T, :H] = dy
        assert _same(ffn(wide[:T, :H]), y)
        y2, saved2 = ffn.forward(wide[:T, :H])
        assert _same(y2, y) and _same(saved2, saved)
        for a, b in zip(grads, ffn.backward(wdy[:T, :H], wide[:T, :H], saved)):
            assert _same(a, b)
    for pad, shift in ((0, 0), (8, 0), (1, 0), (3, 1), (4, 4), (2, 1)):  # 16-byte, 8-byte, 2-byte aligned rows
        flat = torch.full(((T + 2) * (H + pad) + 8,), 7.0, dtype=BF16, device="cuda")
        rows = flat[shift:shift + (T + 2) * (H + pad)].view(T + 2, H + pad)
        out = rows[:T, :H]
        assert ffn(x, out=out) is out
        assert _same(out, y)
        left = flat.clone()
        left[shift:shift + (T + 2) * (H + pad)].view(T + 2, H + pad)[:T, :H] = 7.0
        assert bool((left == 7.0).all())


@pytest.mark.parametrize("T,H,I", [(5, 264, 136), (300, 1032, 520), (1999, 2056, 1400)])
def test_rows_that_are_not_finite_stay_in_their_rows(cuda_device, T, H, I):
    x, gate_up, down, dy = make(T, H, I, seed=3)
    ffn = EpFfn(gate_up, down)
    want, (_, saved) = ffn(x), ffn.forward(x)
    dx = ffn.backward(dy, x, saved, need_weights=False)[0]
    bad, bdy = x.clone(), dy.clone()
    bad[1, 3], bad[T - 1, H - 1], bdy[2, 0], bdy[T - 2, H - 1] = float("nan"), float("inf"), float("nan"), float("-inf")
    got = ffn(bad)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[[1, T - 1]] = False
    assert _same(got[keep], want[keep]) and bool(got[1].isnan().all())
    got = ffn.backward(bdy, x, saved, need_weights=False)[0]
    keep[:] = True
    keep[[2, T - 2]] = False
    assert _same(got[keep], dx[keep]) and bool(got[2].isnan().all())


@pytest.mark.parametrize("T", [6, 400])
@pytest.mark.parametrize("spread", [50.0, 1e4, 1e12])
def test_gates_far_from_zero(cuda_device, T, spread):
    """Gates up to some 10^13: silu is then the gate, or nothing, and its slope 1 or 0."""
    x, gate_up, down, dy = make(T, 256, 200, seed=4, spread=spread)
    ffn = EpFfn(gate_up, down)
    want, err, state = block_ref.ffn(x, gate_up, down)
    y, saved = ffn.forward(x)
    block_ref.check(y, want, err, "y")
    for name, got, (g, e) in zip(("dx", "dgate_up", "ddown"), ffn.backward(dy, x, saved), block_ref.ffn_back(dy, state)):
        assert bool(got.isfinite().all())
        block_ref.check(got, g, e, name)


@pytest.mark.parametrize("T,H,I", [(9, 136, 72), (1999, 2056, 1400)])
def test_what_is_not_asked_for(cuda_device, T, H, I):
    x, gate_up, down, dy = make(T, H, I, seed=5)
    ffn = EpFfn(gate_up, down)
    _, saved = ffn.forward(x)
    dx, dgate_up, ddown = ffn.backward(dy, x, saved)
    a = ffn.backward(dy, x, saved, need_weights=False)
    assert _same(a[0], dx) and a[1] is None and a[2] is None
    a = ffn.backward(dy, x, saved, need_dx=False)
    block_ref_close = [(a[1], dgate_up), (a[2], ddown)]
    assert a[0] is None
    for got, want in block_ref_close:  # other products in the launch: parts of sums may be cut elsewhere
        off = (got.double() - want.double()).abs()
        assert bool((off <= 2.0 ** -7 * want.double().abs() + 2.0 ** -12 * want.double().abs().mean()).all())


@pytest.mark.parametrize("T,H,I", [(100, 256, 4096), (16, 1024, 5000), (3, 72, 16384), (300, 520, 8192), (9001, 264, 256), (700, 2048, 768)])
def test_few_tiles_shared_by_many_blocks(cuda_device, T, H, I):
    """dx alone, the weights' gradients alone and all: tiles whose K goes over many blocks, and shares that some blocks lack."""
    x, gate_up, down, dy = make(T, H, I, seed=11)
    ffn = EpFfn(gate_up, down)
    _, _, state = block_ref.ffn(x, gate_up, down)
    want = block_ref.ffn_back(dy, state)
    _, saved = ffn.forward(x)
    calls = [ffn.backward(dy, x, saved, **kw) for kw in (dict(), dict(need_weights=False), dict(need_dx=False))]
    for got in calls:
        for name, t, (g, e) in zip(("dx", "dgate_up", "ddown"), got, want):
            if t is not None:
                block_ref.check(t, g, e, name)
    for kw, first in zip((dict(), dict(need_weights=False), dict(need_dx=False)), calls):
        for t, again in zip(first, ffn.backward(dy, x, saved, **kw)):
            assert t is None and again is None or torch.equal(t, again)


@pytest.mark.parametrize("T,H,I", [(1, 72, 40), (70, 264, 136), (1100, 520, 1032)])
def test_gradients_in_fp32_and_added_up(cuda_device, T, H, I):
    x, gate_up, down, dy = make(T, H, I, seed=6)
    ffn = EpFfn(gate_up, down)
    state = block_ref.ffn(x, gate_up, down)[2]
    _, saved = ffn.forward(x)
    wide = [torch.full(w.shape, float("nan"), device="cuda") for w in (gate_up, down)]
    dx, *got = ffn.backward(dy, x, saved, dgate_up=wide[0], ddown=wide[1])
    assert got[0] is wide[0] and got[1] is wide[1]
    once = [w.clone() for w in wide]
    for name, g, (want, err) in zip(("dgate_up", "ddown"), once, block_ref.ffn_back(dy, state)[1:]):
        block_ref.check(g, want, err, name)
    narrow = ffn.backward(dy, x, saved)
    assert _same(narrow[0], dx)
    for a, b in zip(narrow[1:], once):
        assert _same(a, b.bfloat16())
    start = [torch.randn_like(w) for w in wide]
    sums = [s.clone() for s in start]
    ffn.backward(dy, x, saved, dgate_up=sums[0], ddown=sums[1], accumulate=True)
    for s, a, b in zip(sums, start, once):
        assert _same(s, a + b)  # one rounding


def test_no_rows(cuda_device):
    x, gate_up, down, dy = make(4, 136, 72)
    ffn = EpFfn(gate_up, down)
    assert ffn(x[:0]).shape == (0, 136)
    y, saved = ffn.forward(x[:0])
    assert y.shape == (0, 136) and saved.shape == (0, 144)
    dx, a, b = ffn.backward(dy[:0], x[:0], saved)
    assert dx.shape == (0, 136) and bool((a == 0).all()) and bool((b == 0).all())
    sums = [torch.randn(w.shape, device="cuda") for w in (gate_up, down)]
    kept = [s.clone() for s in sums]
    ffn.backward(dy[:0], x[:0], saved, dgate_up=sums[0], ddown=sums[1], accumulate=True)
    assert all(_same(a, b) for a, b in zip(sums, kept))


@pytest.mark.parametrize("T", [3, 300])
def test_weights_that_change_between_calls(cuda_device, T):
    """A step that changes the weights in place, right before the next call on the same stream, and in a replayed graph."""
    H, I = 1032, 1400
    x, gate_up, down, dy = make(T, H, I, seed=7)
    w = [gate_up.clone(), down.clone()]
    ffn = EpFfn(*w)
    other = make(T, H, I, seed=8)[1:3]
    a, b = ffn(x), EpFfn(*other)(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, saved = ffn.forward(x)
        grads = ffn.backward(dy, x, saved)
    for _ in range(3):
        for new, want in ((other, b), ((gate_up, down), a)):
            for t, v in zip(w, new):
                t.copy_(v)
            assert _same(ffn(x), want)
            y.zero_()
            for t, v in zip(w, new):
                t.copy_(v)
            graph.replay()
            assert _same(y, want)
            f = EpFfn(*new)
            for g, h in zip(grads, f.backward(dy, x, f.forward(x)[1])):
                assert _same(g, h)


def test_other_streams(cuda_device):
    """One handle on two streams with events between them, and two handles at the same time."""
    x, gate_up, down, dy = make(515, 1024, 4000, seed=9)
    ffn, second = EpFfn(gate_up, down), EpFfn(gate_up, down)
    y, saved = ffn.forward(x)
    grads = ffn.backward(dy, x, saved)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(6):
        s, before = streams[i % 2], streams[1 - i % 2]
        s.wait_stream(before)
        with torch.cuda.stream(s):
            y2, saved2 = ffn.forward(x)
            got = ffn.backward(dy, x, saved2)
    torch.cuda.synchronize()
    assert _same(y, y2) and all(_same(a, b) for a, b in zip(grads, got))
    for _ in range(5):
        outs = []
        for f, s in zip((ffn, second), streams):
            with torch.cuda.stream(s):
                y2, saved2 = f.forward(x)
                outs.append((y2, *f.backward(dy, x, saved2)))
        torch.cuda.synchronize()
        for o in outs:
            assert _same(o[0], y) and all(_same(a, b) for a, b in zip(grads, o[1:]))


def test_two_graphs_of_one_block(cuda_device):
    """Two captured calls with different numbers of rows, replayed in turn."""
    x, gate_up, down, _ = make(700, 1024, 9000, seed=10)
    ffn = EpFfn(gate_up, down)
    graphs, outs, sizes = [], [], (700, 90)
    want = [ffn(x[:n]) for n in sizes]
    for n in sizes:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(ffn(x[:n]))
        graphs.append(g)
    for _ in range(4):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(_same(a, b) for a, b in zip(want, outs))


def test_offsets_past_32_bits(cuda_device):
    """300000 rows: 2 * 8192 kept values a row are 4.9e9, 20 GB; and weights' gradients over all of them."""
    T, H, I = 300000, 128, 8192
    x, gate_up, down, dy = make(T, H, I, seed=11)
    ffn = EpFfn(gate_up, down)
    y, saved = ffn.forward(x)
    dx, dgate_up, ddown = ffn.backward(dy, x, saved)
    picks = torch.tensor([0, 131071, 131072, 262143, 262144, T - 1], device="cuda")
    want, err, state = block_ref.ffn(x[picks], gate_up, down)
    block_ref.check(y[picks], want, err, "y")
    block_ref.check(saved[picks], torch.cat(state[3:5], 1), torch.cat(state[5:7], 1), "saved")
    block_ref.check(dx[picks], *block_ref.ffn_back(dy[picks], state)[0], "dx")
    total = [torch.zeros(w.shape, dtype=torch.float64, device="cuda") for w in (gate_up, down)]
    squares = [torch.zeros_like(t) for t in total]
    for i in range(0, T, 20000):
        part = block_ref.ffn_back(dy[i:i + 20000], block_ref.ffn(x[i:i + 20000], gate_up, down)[2])[1:]
        for k, (g, e) in enumerate(part):
            total[k] += g
            squares[k] += e.square()
    for got, want, sq in zip((dgate_up, ddown), total, squares):
        # independent errors of the chunks' rows; the accumulator's own grow with the number of additions
        block_ref.check(got, want, sq.sqrt() * (1 + (T / 16 + 64) / (20000 / 16 + 64) / 4), "weights")


def test_refusals(cuda_device):
    x, gate_up, down, dy = make(8, 136, 72)
    ffn = EpFfn(gate_up, down)
    _, saved = ffn.forward(x)
    f32 = [torch.zeros(w.shape, device="cuda") for w in (gate_up, down)]
    for bad in (lambda: ffn(x.half()), lambda: ffn(x[:, :128]), lambda: ffn(x, out=x[:4]), lambda: ffn(x.cpu()),
                lambda: ffn.backward(dy[:4], x, saved), lambda: ffn.backward(dy, x, saved[:4]),
                lambda: ffn.backward(dy, x, saved.bfloat16()), lambda: ffn.backward(dy, x, saved, dgate_up=f32[0]),
                lambda: ffn.backward(dy, x, saved, dgate_up=f32[0], ddown=down.clone()),
                lambda: ffn.backward(dy, x, saved, accumulate=True),
                lambda: ffn.backward(dy, x, saved, dgate_up=gate_up.clone(), ddown=down.clone(), accumulate=True),
                lambda: ffn.backward(dy, x, saved, dgate_up=gate_up.half(), ddown=down.half()),
                lambda: ffn.backward(dy, x, saved, need_weights=False, dgate_up=f32[0], ddown=f32[1]),
                lambda: EpFfn(gate_up, down.t()), lambda: EpFfn(gate_up[:143], down), lambda: EpFfn(gate_up.float(), down.float()),
                lambda: EpFfn(gate_up[:, ::2], down)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: ffn(x, out=x), lambda: EpFfn(torch.zeros(16, 12, dtype=BF16, device="cuda"), torch.zeros(12, 8, dtype=BF16, device="cuda")),
                lambda: ffn(torch.zeros(8, 140, dtype=BF16, device="cuda")[:, :136])):
        with pytest.raises(EpError) as e:
            bad()
        assert e.value.status == EP_ERR_INVALID_ARG
    ffn.destroy()
    ffn.destroy()
    with pytest.raises(EpError):
        ffn(x)
