"""The norm where it can go wrong: strides, rows in place, rows that are not finite or too large to square, graphs,
streams, offsets past 32 bits, refusals."""
import pytest
import torch

import block_ref
from combine_topk_ids_dest_gb300 import EpNorm, EP_ERR_INVALID_ARG
from combine_topk_ids_dest_gb300._lib import EpError
from test_gpu_norm import EPS, make

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _same(a, b):
    """Equal bits, NaN included."""
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("T,H", [(3, 264), (400, 2056), (900, 256)])
def test_strides_and_rows_beside(cuda_device, T, H):
    """Rows of wider buffers give the same results; what lies beside them, and rows after the last, stay as they were."""
    x, residual, w, dy, dh = make(T, H, BF16, seed=3)
    call = EpNorm(w, eps=EPS)
    want, back = call(x, residual, quantized=True), call.backward(dy, x, dh)

    def wide(t, pad):
        b = torch.full((T + 2, H + pad), 7.0, dtype=BF16, device="cuda")
        b[:T, :H] = t
        return b, b[:T, :H]

    (_, wx), (_, wr), (_, wdy), (_, wdh) = wide(x, 8), wide(residual, 64), wide(dy, 16), wide(dh, 40)
    (bo, out), (br, residual_out), (bd, dx) = wide(x * 0, 24), wide(x * 0, 8), wide(x * 0, 72)
    got = call(wx, wr, quantized=True, out=out, residual_out=residual_out)
    assert got.out is out and got.residual is residual_out
    for a, b in zip(want, got):
        assert _same(a, b)
    got = call.backward(wdy, wx, wdh, dx=dx)
    assert _same(got[0], back[0]) and _same(got[1], back[1])
    for b in (bo, br, bd):
        assert bool((b[T:] == 7).all()) and bool((b[:, H:] == 7).all())


def test_in_place(cuda_device):
    x, residual, w, dy, dh = make(500, 1032, BF16, seed=4)
    call = EpNorm(w, eps=EPS)
    want, back = call(x, residual, quantized=True), call.backward(dy, x, dh)
    for o, r in ((0, 1), (1, 0)):
        t = [x.clone(), residual.clone()]
        got = call(*t, quantized=True, out=t[o], residual_out=t[r])
        for a, b in zip(want, got):
            assert _same(a, b)
    for k in range(3):
        t = [dy.clone(), x.clone(), dh.clone()]
        got = call.backward(*t, dx=t[k])
        assert _same(got[0], back[0]) and _same(got[1], back[1])


@pytest.mark.parametrize("T", [4, 700])
@pytest.mark.parametrize("H", [200, 256, 1000, 4104])
def test_rows_that_are_not_finite_stay_in_their_rows(cuda_device, T, H):
    x, residual, w, dy, dh = make(T, H, BF16, seed=5)
    call = EpNorm(w, eps=EPS)
    clean, back = call(x, residual, quantized=True), call.backward(dy, x, dh)
    bad = x.clone()
    bad[1, 5], bad[2, H - 1], bad[3, 0] = float("nan"), float("inf"), float("-inf")
    got = call(bad, residual, quantized=True)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[1:4] = False
    for a, b in zip(clean, got):
        assert _same(a[keep], b[keep])
    assert bool(got.out[1].isnan().all()) and bool(got.scales[1].isnan().all()) and bool(got.q[1].float().isnan().all())
    # an infinity is NaN itself, the other columns are 0 beside it, as in the formula; its group's scale says so
    for row, col in ((2, H - 1), (3, 0)):
        o = got.out[row].clone()
        assert bool(o[col].isnan())
        o[col] = 0
        assert bool((o == 0).all())
        groups = got.scales[row].isnan()
        assert bool(groups[col // 128]) and int(groups.sum()) == 1
        q = got.q[row].float()
        assert bool(q[col // 128 * 128:col // 128 * 128 + 128].isnan().all()) and not bool(q.isnan().all() if H > 128 else False)
    dx, _ = call.backward(dy, bad, dh)
    assert _same(dx[keep], back[0][keep])
    assert bool(dx[1].isnan().all())


@pytest.mark.parametrize("dtype,size", [(BF16, 1e30), (torch.float32, 3e37), (torch.float16, 6e4), (BF16, 1e-30), (torch.float32, 1e-38)])
@pytest.mark.parametrize("H", [128, 1000, 7168])
def test_ends_of_the_range(cuda_device, H, dtype, size):
    """Squares that exceed fp32, or vanish: the values are those of 64 bits all the same."""
    x, _, w, dy, dh = make(5, H, torch.float32, seed=6)
    x = (x / 64 * size).to(dtype)
    w, dy, dh = w.to(dtype), dy.to(dtype), dh.to(dtype)
    call = EpNorm(w, eps=EPS)
    _, y = block_ref.norm(x, None, w, EPS)
    got = call(x, quantized=True)
    # where the type has subnormals y may be one: fp32's own, half a step of 2^-149, times the products behind it
    block_ref.check(got.out, y, block_ref.NORM * y.abs() + 2.0 ** -140, "out")
    assert bool((got.scales >= 2.0 ** -126).all()) and bool(got.q.float().abs().max() <= 448)
    dx, edx, dw, edw = block_ref.norm_back(dy, x, dh, w, EPS)
    gdx, gdw = call.backward(dy, x, dh)
    block_ref.check(gdx, dx, edx + 2.0 ** -140, "dx")
    block_ref.check(gdw, dw, edw + 2.0 ** -140, "dweight")


def test_rows_of_zeros(cuda_device):
    x, _, w, dy, _ = make(6, 300 // 8 * 8, BF16, seed=7)
    x[2] = 0
    r = EpNorm(w, eps=EPS)(x, quantized=True)
    assert bool((r.out[2] == 0).all()) and bool((r.q[2].float() == 0).all()) and bool((r.scales[2] == 2.0 ** -126).all())
    dx, edx, _, _ = block_ref.norm_back(dy, x, None, w, EPS)
    block_ref.check(EpNorm(w, eps=EPS).backward(dy, x)[0], dx, edx, "dx")


def test_no_rows(cuda_device):
    x, residual, w, dy, _ = make(4, 264, BF16)
    call = EpNorm(w, eps=EPS)
    r = call(x[:0], residual[:0], quantized=True)
    assert r.out.shape == r.residual.shape == r.q.shape == (0, 264) and r.scales.shape == (0, 3)
    dx, dw = call.backward(dy[:0], x[:0])
    assert dx.shape == (0, 264) and bool((dw == 0).all())


def test_results_do_not_depend_on_the_call(cuda_device):
    """A row's results are the same whatever the rows beside it; the weight's gradient is the same from call to call."""
    x, residual, w, dy, dh = make(3001, 2056, BF16, seed=8)
    call = EpNorm(w, eps=EPS)
    a = call.backward(dy, x, dh)
    for _ in range(5):
        b = call.backward(dy, x, dh)
        assert _same(a[0], b[0]) and _same(a[1], b[1])
    assert _same(call(x, residual).residual[:700], call(x[:700], residual[:700]).residual)


def test_another_stream_and_a_graph(cuda_device):
    x, residual, w, dy, dh = make(640, 1032, BF16, seed=9)
    call = EpNorm(w, eps=EPS)
    want, back = call(x, residual, quantized=True), call.backward(dy, x, dh)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        got, gback = call(x, residual, quantized=True), call.backward(dy, x, dh)
    stream.synchronize()
    for a, b in zip((*want, *back), (*got, *gback)):
        assert _same(a, b)
    inputs = [torch.zeros_like(t) for t in (x, residual, dy, dh)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = call(inputs[0], inputs[1], quantized=True)
        b = call.backward(inputs[2], inputs[0], inputs[3])
        twice = call(r.out, r.residual)  # overlaps the kernel before it
    for t, v in zip(inputs, (x, residual, dy, dh)):
        t.copy_(v)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for u, v in zip((*want, *back), (*r, *b)):
        assert _same(u, v)
    assert _same(call(want.out, want.residual).out, twice.out)


def test_two_calls_at_once(cuda_device):
    """Calls have no state of their own: two streams may run them at the same time."""
    sets = [make(4000, 2048, BF16, seed=s) for s in (1, 2)]
    calls = [EpNorm(t[2], eps=EPS) for t in sets]
    want = [(*c(t[0], t[1], quantized=True), *c.backward(t[3], t[0], t[4])) for c, t in zip(calls, sets)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = []
        for c, t, s in zip(calls, sets, streams):
            with torch.cuda.stream(s):
                got.append((*c(t[0], t[1], quantized=True), *c.backward(t[3], t[0], t[4])))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(_same(u, v) for u, v in zip(a, b))


def test_offsets_past_32_bits(cuda_device):
    """600000 rows of 4096: 2.4e9 values, 4.9e9 bytes."""
    T, H = 600000, 4096
    gen = torch.Generator("cuda").manual_seed(1)
    x = torch.empty(T, H, dtype=BF16, device="cuda").normal_(generator=gen)
    w = (1 + 0.2 * torch.randn(H, generator=gen, device="cuda")).bfloat16()
    call = EpNorm(w, eps=EPS)
    r = call(x, x, quantized=True)
    picks = torch.tensor([0, 1, 524287, 524288, 524289, T - 1], device="cuda")
    s, y = block_ref.norm(x[picks], x[picks], w, EPS)
    block_ref.check(r.residual[picks], s, block_ref.FP32 * s.abs())
    block_ref.check(r.out[picks], y, block_ref.NORM * y.abs())
    block_ref.check_quantized(r.q[picks], r.scales[picks], y)
    dx, dw = call.backward(r.out, x, r.residual)
    want, err, _, _ = block_ref.norm_back(r.out[picks], x[picks], r.residual[picks], w, EPS)
    block_ref.check(dx[picks], want, err)
    total, size = torch.zeros(H, dtype=torch.float64, device="cuda"), torch.zeros(H, dtype=torch.float64, device="cuda")
    for i in range(0, T, 50000):
        _, _, part, bound = block_ref.norm_back(r.out[i:i + 50000], x[i:i + 50000], None, w, EPS)
        total += part
        size += bound / (2 * block_ref.NORM + (50000 / 128 + 64) * block_ref.FP32)
    block_ref.check(dw, total, (2 * block_ref.NORM + (T / 128 + 64) * block_ref.FP32) * size)


def test_refusals(cuda_device):
    x, residual, w, dy, _ = make(8, 256, BF16)
    call = EpNorm(w, eps=EPS)
    for bad in (lambda: call(x.float()), lambda: call(x[:, :128]), lambda: call(x.t()), lambda: call(x, residual[:4]),
                lambda: call(x, out=x[:4]), lambda: call(x, residual_out=x), lambda: call(x, plain=False, out=x),
                lambda: call(x.cpu()), lambda: call.backward(dy, x[:3]), lambda: call.backward(dy, x, dy[:2]),
                lambda: call.backward(dy, x, dx=dy[:2]), lambda: EpNorm(w.half(), dtype=BF16), lambda: EpNorm(w[None]),
                lambda: EpNorm(w[::2]), lambda: EpNorm(w.int())):
        with pytest.raises(ValueError):
            bad()
    wide = torch.zeros(9, 264, dtype=BF16, device="cuda")
    for bad in (lambda: call(wide.view(-1)[4:4 + 8 * 264].view(8, 264)[:, :256]), lambda: call(x, residual, out=residual[0:8], residual_out=residual),
                lambda: EpNorm(w, eps=0.0), lambda: EpNorm(torch.ones(4, device="cuda")),
                lambda: EpNorm(torch.ones(16392, device="cuda")),
                lambda: call(torch.zeros(8, 260, dtype=BF16, device="cuda")[:, :256])):
        with pytest.raises(EpError) as e:
            bad()
        assert e.value.status == EP_ERR_INVALID_ARG
