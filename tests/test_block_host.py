"""CPU checks of the norm's and the feed-forward block's host side, over a stand-in runtime: refusals, what is launched,
devices; and the 64-bit forms' gradients against differences."""
import ctypes

import pytest
import torch

import block_ref
import combine_topk_ids_dest_gb300 as ep
from combine_topk_ids_dest_gb300 import _lib
from fake_runtime import Fake

INVALID, OK = _lib.EP_ERR_INVALID_ARG, _lib.EP_OK
AT = [k << 40 for k in range(1, 12)]  # addresses of operands, far from one another; nothing reads them
H, T = 256, 5


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    return Fake(tmp_path_factory.mktemp("fake"))


@pytest.fixture(autouse=True)
def clean(fake):
    fake.L.fake_device(0)
    fake.L.fake_sms(152)
    fake.L.fake_clear()


def _cfg(**kw):
    b = dict(hidden=H, dtype=0, weight_dtype=0, eps=1e-6, weight=AT[0])
    b.update(kw)
    return _lib.EpNormConfigC(*b.values())


def _norm(fake, cfg=None, n=T, **kw):
    b = dict(x=AT[1], x_stride=H, residual=AT[2], residual_stride=H, residual_out=AT[3], residual_out_stride=H, out=AT[4],
             out_stride=H, q=AT[5], scales=AT[6])
    b.update(kw)
    return fake.L.ep_norm_run(ctypes.byref(cfg or _cfg()), ctypes.byref(_lib.EpNormRowsC(*b.values())), n, None)


@pytest.mark.parametrize("kw,frag", [
    (dict(hidden=0), "hidden"), (dict(hidden=12), "hidden"), (dict(hidden=16392), "hidden"), (dict(dtype=1), "dtype"),
    (dict(weight_dtype=2), "weight_dtype"), (dict(dtype=3, weight_dtype=0), "weight_dtype"), (dict(eps=0.0), "eps"),
    (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(eps=float("inf")), "eps"), (dict(weight=0), "weight"),
    (dict(weight=AT[0] + 8), "weight"),
])
def test_norm_configurations_refused(fake, kw, frag):
    assert _norm(fake, _cfg(**kw)) == INVALID and frag in fake.message()
    n = ctypes.c_size_t(0)
    assert fake.L.ep_norm_backward_workspace_size(ctypes.byref(_cfg(**kw)), T, ctypes.byref(n)) == INVALID
    assert fake.launches() == []


@pytest.mark.parametrize("kw,frag", [
    (dict(x=0), "x"), (dict(x=AT[1] + 8), "x"), (dict(x_stride=H - 8), "x"), (dict(x_stride=H + 4), "x"),
    (dict(residual_stride=H - 8), "residual"), (dict(out=AT[4] + 2), "out"), (dict(out_stride=0), "out"),
    (dict(residual=0), "residual_out without residual"), (dict(q=0), "together"), (dict(scales=0), "together"),
    (dict(q=AT[5] + 4), "aligned"), (dict(scales=AT[6] + 2), "aligned"),
    (dict(out=AT[1] + 16), "overlaps"), (dict(out=AT[1], out_stride=2 * H), "overlaps"), (dict(out=AT[3]), "overlaps"),
    (dict(residual_out=AT[2] + 2 * H), "overlaps"), (dict(q=AT[1]), "overlaps"), (dict(scales=AT[5]), "overlaps"),
    (dict(n=-1), "num_tokens"),
])
def test_norm_rows_refused(fake, kw, frag):
    assert _norm(fake, **kw) == INVALID and frag in fake.message(), fake.message()
    assert fake.launches() == []


@pytest.mark.parametrize("kw", [dict(out=AT[0]), dict(residual_out=AT[0] + 16), dict(q=AT[0] + 2 * H - 8), dict(scales=AT[0])])
def test_norm_results_on_the_weight_refused(fake, kw):
    assert _norm(fake, **kw) == INVALID and "overlaps weight" in fake.message(), fake.message()
    assert fake.launches() == []


def test_norm_in_place_and_without_rows(fake):
    for kw in (dict(), dict(out=AT[1]), dict(residual_out=AT[2]), dict(residual_out=AT[1], out=AT[2]),
               dict(residual=0, residual_out=0), dict(q=0, scales=0), dict(out=0)):
        fake.L.fake_clear()
        assert _norm(fake, **kw) == OK, fake.message()
        assert len(fake.launches()) == 1
    fake.L.fake_clear()
    assert _norm(fake, n=0, x=0) == OK and fake.launches() == []


def test_norm_blocks_hold_every_row(fake):
    """Any number of rows up to the largest; threads and rows of a block within what the kernel is made for."""
    for dtype in (0, 2, 3):
        for hidden in (8, 128, 256, 264, 512, 2048, 2056, 4096, 7168, 8200, 16384):
            for n in (1, 3, 304, 305, 16001, 2**31 - 1):
                fake.L.fake_clear()
                rows = dict(x_stride=hidden, residual=0, residual_out=0, out=1 << 56, out_stride=hidden, q=0, scales=0)
                assert _norm(fake, _cfg(hidden=hidden, dtype=dtype, weight_dtype=dtype), n, **rows) == OK, fake.message()
                (name, _, grid, block, _), = fake.launches()
                units = int(name[name.index("Li") + 2])
                assert block[0] % 32 == 0 and block[0] * units >= hidden // 8 and block[0] * block[1] <= 1024
                assert block[1] == 1 or (block[0] == 32 and block[1] <= 4)
                assert grid[0] * block[1] >= n and grid[0] <= 2**31 - 1


def _back(fake, cfg=None, n=T, workspace=AT[8], bytes=1 << 30, **kw):
    b = dict(dy=AT[1], dy_stride=H, h=AT[2], h_stride=H, dh=AT[3], dh_stride=H, dx=AT[4], dx_stride=H, dweight=AT[5])
    b.update(kw)
    v = list(b.values())
    return fake.L.ep_norm_backward(ctypes.byref(cfg or _cfg()), *v[:6], n, *v[6:], workspace, bytes, None)


@pytest.mark.parametrize("kw,frag", [
    (dict(dy=0), "dy"), (dict(h=0), "h"), (dict(dy_stride=H + 1), "dy"), (dict(dh_stride=8), "dh"), (dict(dx=AT[4] + 2), "dx"),
    (dict(dweight=AT[5] + 1), "dweight"), (dict(workspace=None), "workspace"), (dict(workspace=AT[8] + 16), "workspace"),
    (dict(bytes=16), "workspace"), (dict(dx=AT[2] + 16), "overlaps"), (dict(dweight=AT[1]), "overlaps"),
    (dict(dweight=AT[4]), "overlaps"), (dict(n=-5), "num_tokens"),
])
def test_norm_backward_refused(fake, kw, frag):
    assert _back(fake, **kw) == INVALID and frag in fake.message(), fake.message()
    assert fake.launches() == []


@pytest.mark.parametrize("kw", [dict(dx=AT[0]), dict(dweight=AT[0])])
def test_norm_gradients_on_the_weight_refused(fake, kw):
    assert _back(fake, **kw) == INVALID and "overlaps weight" in fake.message(), fake.message()
    assert fake.launches() == []


def test_norm_backward_launches(fake):
    for kw, kernels in ((dict(), 2), (dict(dx=0), 2), (dict(dweight=0, workspace=None), 1), (dict(dx=AT[1]), 2),
                        (dict(dx=AT[3]), 2), (dict(dh=0, dh_stride=0), 2), (dict(dx=0, dweight=0), 0), (dict(n=0), 1),
                        (dict(n=0, dweight=0), 0)):
        fake.L.fake_clear()
        assert _back(fake, **kw) == OK, fake.message()
        assert len(fake.launches()) == kernels, kw
    size = ctypes.c_size_t(0)
    for dtype in (0, 2, 3):
        for hidden in (8, 256, 512, 520, 4096, 7168, 8192, 8200, 16384):
            cfg = _cfg(hidden=hidden, dtype=dtype, weight_dtype=3)
            for n in (1, 7, 152, 153, 1000, 2**31 - 1):
                fake.L.fake_clear()
                assert fake.L.ep_norm_backward_workspace_size(ctypes.byref(cfg), n, ctypes.byref(size)) == OK
                strides = dict(dy_stride=hidden, h_stride=hidden, dh_stride=hidden, dx_stride=hidden)
                big = dict(zip(("dy", "h", "dh", "dx", "dweight"), (k << 52 for k in range(1, 6))))
                assert _back(fake, cfg, n, bytes=size.value, **strides, **big) == OK, fake.message()
                (_, _, grid, block, smem), (_, _, sums, _, _) = fake.launches()
                assert grid[0] <= min(n, 152) and size.value >= grid[0] * hidden * 4
                assert smem <= 227 * 1024 - 6000 and block[0] == 544 and sums[0] * 32 >= hidden


def test_norm_on_two_devices(fake):
    """A kernel's shared-memory limit belongs to the device that was current when it was set."""
    for device in (1, 0, 1):
        fake.L.fake_device(device)
        fake.L.fake_clear()
        assert _norm(fake) == OK and _back(fake) == OK, fake.message()
        assert [l[1] for l in fake.launches()] == [device] * 3


# ---- feed-forward ------------------------------------------------------------------------

I = 128


def _ffn(fake, **kw):
    b = dict(hidden=H, intermediate=I, gate_up=AT[0], down=AT[1])
    b.update(kw)
    h = ctypes.c_void_p()
    st = fake.L.ep_ffn_create(ctypes.byref(_lib.EpFfnConfigC(*b.values())), ctypes.byref(h))
    return st, h.value


@pytest.fixture
def ffn(fake):
    st, h = _ffn(fake)
    assert st == OK, fake.message()
    fake.L.fake_clear()
    yield h
    assert fake.L.ep_ffn_destroy(h) == OK


@pytest.mark.parametrize("kw,frag", [
    (dict(hidden=0), "hidden"), (dict(hidden=12), "hidden"), (dict(hidden=65544), "hidden"), (dict(intermediate=4), "intermediate"),
    (dict(intermediate=65544), "intermediate"), (dict(gate_up=0), "gate_up"), (dict(gate_up=AT[0] + 8), "gate_up"),
    (dict(down=0), "down"), (dict(down=AT[1] + 2), "down"),
])
def test_ffn_configurations_refused(fake, kw, frag):
    st, h = _ffn(fake, **kw)
    assert st == INVALID and h is None and frag in fake.message()


def _run(fake, h, n=T, workspace=AT[8], bytes=1 << 36, **kw):
    b = dict(x=AT[2], x_stride=H, saved=None, out=AT[3], out_stride=H)
    b.update(kw)
    return fake.L.ep_ffn_run(h, b["x"], b["x_stride"], n, b["saved"], b["out"], b["out_stride"], workspace, bytes, None)


@pytest.mark.parametrize("kw,frag", [
    (dict(n=-1), "num_tokens"), (dict(n=16777217), "num_tokens"), (dict(x=None), "x"), (dict(x=AT[2] + 2), "x"),
    (dict(x_stride=H - 8), "x"), (dict(x_stride=H + 2), "x"), (dict(out=None), "out"), (dict(out=AT[3] + 1), "out"),
    (dict(out_stride=H - 1), "out"), (dict(saved=AT[4] + 4), "saved"), (dict(out=AT[2]), "overlaps"),
    (dict(saved=AT[2]), "overlaps"), (dict(saved=AT[3]), "overlaps"), (dict(workspace=None), "workspace"),
    (dict(workspace=AT[8] + 128), "workspace"), (dict(bytes=64), "workspace"),
])
def test_ffn_runs_refused(fake, ffn, kw, frag):
    assert _run(fake, ffn, **kw) == INVALID and frag in fake.message(), fake.message()
    assert fake.launches() == []


def _backward(fake, h, n=T, workspace=AT[8], bytes=1 << 36, **kw):
    b = dict(dy=AT[2], dy_stride=H, x=AT[3], x_stride=H, saved=AT[4], dx=AT[5], dx_stride=H, dgate_up=AT[6], ddown=AT[7],
             grad_dtype=0, accumulate=0)
    b.update(kw)
    return fake.L.ep_ffn_backward(h, ctypes.byref(_lib.EpFfnGradsC(*b.values())), n, workspace, bytes, None)


@pytest.mark.parametrize("kw,frag", [
    (dict(dy=0), "dy"), (dict(x=0), "x"), (dict(saved=0), "saved"), (dict(saved=AT[4] + 8), "saved"), (dict(dy_stride=8), "dy"),
    (dict(x_stride=H + 2), "x"), (dict(dx_stride=H - 1), "dx"), (dict(dx=AT[5] + 1), "dx"), (dict(grad_dtype=2), "grad_dtype"),
    (dict(accumulate=1), "accumulate"), (dict(dgate_up=AT[6] + 8), "aligned"), (dict(ddown=AT[7] + 2), "aligned"),
    (dict(dx=AT[2]), "overlaps"), (dict(dx=AT[3]), "overlaps"), (dict(dgate_up=AT[4]), "overlaps"),
    (dict(ddown=AT[6]), "overlaps"), (dict(workspace=None), "workspace"), (dict(bytes=1 << 10), "workspace"),
    (dict(n=-3), "num_tokens"),
])
def test_ffn_backward_refused(fake, ffn, kw, frag):
    assert _backward(fake, ffn, **kw) == INVALID and frag in fake.message(), fake.message()
    assert fake.launches() == []


@pytest.mark.parametrize("kw,frag", [
    (dict(out=AT[0]), "out overlaps gate_up"), (dict(out=AT[1] + 2), "out overlaps down"),
    (dict(saved=AT[0] + 4 * H * I - 16), "saved overlaps gate_up"), (dict(saved=AT[1]), "saved overlaps down"),
])
def test_ffn_results_on_the_weights_refused(fake, ffn, kw, frag):
    assert _run(fake, ffn, **kw) == INVALID and frag in fake.message(), fake.message()
    assert fake.launches() == []


@pytest.mark.parametrize("kw,frag", [
    (dict(dx=AT[1]), "dx overlaps down"), (dict(dgate_up=AT[0]), "dgate_up overlaps gate_up"),
    (dict(ddown=AT[1]), "ddown overlaps down"), (dict(ddown=AT[0] + 4 * H * I - 16), "ddown overlaps gate_up"),
])
def test_ffn_gradients_on_the_weights_refused(fake, ffn, kw, frag):
    assert _backward(fake, ffn, **kw) == INVALID and frag in fake.message(), fake.message()
    assert fake.launches() == []


def test_ffn_launches(fake, ffn):
    for n, kw, kernels in ((T, dict(), 2), (1000, dict(), 2), (1000, dict(saved=AT[4]), 2), (0, dict(x=None), 0)):
        fake.L.fake_clear()
        assert _run(fake, ffn, n, **kw) == OK, fake.message()
        assert len(fake.launches()) == kernels
    for n, kw, kernels in ((T, dict(), 2), (1000, dict(), 2), (T, dict(dx=0), 2), (T, dict(dgate_up=0, ddown=0), 2),
                           (T, dict(dx=0, dgate_up=0, ddown=0), 0), (0, dict(), 2), (0, dict(ddown=0), 1),
                           (0, dict(grad_dtype=3, accumulate=1), 0)):
        fake.L.fake_clear()
        assert _backward(fake, ffn, n, **kw) == OK, fake.message()
        assert len(fake.launches()) == kernels, kw


def test_ffn_workspace_and_shared_memory(fake):
    """A launch fits the device, and a call of one size does not use what is kept of another size's plan."""
    size = ctypes.c_size_t(0)
    for hidden, intermediate in ((8, 8), (2056, 1400), (4096, 14336), (65536, 65536)):
        st, h = _ffn(fake, hidden=hidden, intermediate=intermediate)
        assert st == OK
        seen = {}
        for n in (1, 500, 8191, 1, 500, 77, 8191):
            for call in range(3):
                assert fake.L.ep_ffn_workspace_size(h, call, n, ctypes.byref(size)) == OK
                rows = n * intermediate * 2 * (3 if call == 2 else 1)
                assert size.value >= rows
                fake.L.fake_clear()
                far = [k << 48 for k in range(1, 10)]
                if call == 2:
                    st = _backward(fake, h, n, bytes=size.value, dy_stride=hidden, x_stride=hidden, dx_stride=hidden,
                                   **dict(zip(("dy", "x", "saved", "dx", "dgate_up", "ddown"), far)))
                else:
                    st = _run(fake, h, n, bytes=size.value, x=far[0], x_stride=hidden, out=far[1], out_stride=hidden,
                              saved=far[2] if call else None)
                assert st == OK, fake.message()
                made = [l[2:] for l in fake.launches()]
                assert len(made) == 2 and all(l[-1] <= 227 * 1024 for l in made)
                assert seen.setdefault((n, call), made) == made
        assert fake.L.ep_ffn_workspace_size(h, 3, 1, ctypes.byref(size)) == INVALID
        assert fake.L.ep_ffn_destroy(h) == OK


def test_ffn_handles_of_two_devices(fake):
    made = []
    for device in (0, 1):
        fake.L.fake_device(device)
        made.append(_ffn(fake)[1])
    for device, h in enumerate(made):
        fake.L.fake_device(device)
        fake.L.fake_clear()
        assert _run(fake, h) == OK and _run(fake, h, 1000) == OK and _backward(fake, h) == OK
        assert {l[1] for l in fake.launches()} == {device}
        fake.L.fake_device(1 - device)
        fake.L.fake_clear()
        assert _run(fake, h) == INVALID and "device" in fake.message()
        assert _backward(fake, h) == INVALID and fake.launches() == []
    for device, h in enumerate(made):
        fake.L.fake_device(1 - device)
        fake.L.fake_clear()
        assert fake.L.ep_ffn_destroy(h) == OK
        assert fake.calls()[0] == f"cudaDeviceSynchronize {device}"


def test_ffn_reports_a_wait_that_ran_out_once(fake, ffn):
    words = fake.L.fake_error_words()
    words[0] = words[4] = 1
    assert _run(fake, ffn) == _lib.EP_ERR_CUDA and "ran out" in fake.message() and fake.launches() == []
    assert _run(fake, ffn) == OK
    words[0] = words[4] = 1
    assert _backward(fake, ffn) == _lib.EP_ERR_CUDA and fake.launches() == [] or len(fake.launches()) == 2


def test_null_arguments(fake):
    L = fake.L
    assert L.ep_norm_run(None, None, 1, None) == INVALID
    assert L.ep_norm_run(ctypes.byref(_cfg()), None, 1, None) == INVALID
    assert L.ep_norm_backward_workspace_size(ctypes.byref(_cfg()), 1, None) == INVALID
    assert L.ep_ffn_create(None, None) == INVALID
    assert L.ep_ffn_run(None, None, 0, 1, None, None, 0, None, 0, None) == INVALID
    assert L.ep_ffn_backward(None, None, 1, None, 0, None) == INVALID
    assert L.ep_ffn_workspace_size(None, 0, 1, None) == INVALID
    assert L.ep_ffn_destroy(None) == OK


def test_binding_wants_cuda_tensors():
    w = torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ep.EpNorm(w)
    with pytest.raises(ValueError, match="CUDA"):
        ep.EpFfn(w, w)


# ---- the forms that the GPU tests compare with -----------------------------------------------


def test_norm_gradients_against_differences():
    gen = torch.Generator().manual_seed(1)
    h, dy, dh = (torch.randn(3, 16, generator=gen, dtype=torch.float64) for _ in range(3))
    w = torch.rand(16, generator=gen, dtype=torch.float64) + 0.5
    dx, _, dw, _ = block_ref.norm_back(dy, h, dh, w, 1e-3)

    def loss(h, w):
        return (block_ref.norm(h, None, w, 1e-3)[1] * dy).sum() + (h * dh).sum()

    _against_differences(loss, [h, w], [dx, dw])


def test_ffn_gradients_against_differences():
    gen = torch.Generator().manual_seed(2)
    x, dy = (torch.randn(3, 8, generator=gen, dtype=torch.float64) for _ in range(2))
    w13, w2 = torch.randn(12, 8, generator=gen, dtype=torch.float64), torch.randn(8, 6, generator=gen, dtype=torch.float64)
    state = block_ref.ffn(x, w13, w2)[2]
    grads = [g for g, _ in block_ref.ffn_back(dy, state)]
    _against_differences(lambda *a: (block_ref.ffn(*a)[0] * dy).sum(), [x, w13, w2], grads)


def _against_differences(loss, inputs, grads, step=1e-5):
    for i, (t, g) in enumerate(zip(inputs, grads)):
        for k in range(0, t.numel(), 5):
            d = torch.zeros_like(t).view(-1)
            d[k] = step
            d = d.view_as(t)
            up, down = ([u + d * s if j == i else u for j, u in enumerate(inputs)] for s in (1, -1))
            want = (loss(*up) - loss(*down)) / (2 * step)
            # central differences: the third derivative's term, and the losses' own rounding over the step
            assert abs(float(want - g.reshape(-1)[k])) < 1e-7 * (1 + abs(float(want)))
