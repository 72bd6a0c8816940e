"""What the MoE operators' host code launches, on the CPU over a stand-in runtime: sizes that the
kernels' buffers hold, for every accepted call."""
import ctypes

import pytest
import torch

from combine_topk_ids_dest_gb300 import EpRouter, _lib
from fake_runtime import Fake


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    return Fake(tmp_path_factory.mktemp("fake"))


@pytest.fixture(autouse=True)
def clean(fake):
    fake.L.fake_device(0)
    fake.L.fake_sms(152)
    fake.L.fake_clear()


@pytest.mark.parametrize("sms", [148, 152, 160])
@pytest.mark.parametrize("hidden,E", [(64, 40), (520, 256), (1024, 384), (7168, 256)])
def test_router_tiles_hold_their_rows(fake, sms, hidden, E):
    """A tile has room for 128 rows in shared memory, tensor memory and the parts; a tile's splits run together."""
    fake.L.fake_sms(sms)
    h = fake.router(hidden=hidden, num_experts=E)
    args = (ctypes.c_int * 2)()
    for n in [*range(65, 9000), *range(9000, 40000, 37)]:
        fake.L.fake_clear()
        st, workspace = fake.route(h, n, hidden)
        assert st == _lib.EP_OK, fake.message()
        (name, _, (tiles, splits, _), _, _), = fake.launches()
        assert "many_kernel" in name
        fake.L.fake_router_args(0, args)
        rows, stages = args
        assert 1 <= rows <= 128 and fake.box()[:2] == (64, rows), (n, rows, fake.box())
        assert tiles * rows >= n and stages >= 2
        if splits > 1:
            assert tiles * splits <= sms and splits <= -(-hidden // 64)
            assert workspace >= tiles * splits * 128 * E * 4
    assert fake.L.ep_router_destroy(h) == _lib.EP_OK


def test_int4_rings_have_two_stages(fake):
    """Two pairs of groups step through the weights' ring by two, each from its own stage on: one stage would let them
    read past the block's memory. Every number of tokens, choices and experts, every kind of tile and entry."""
    v = (ctypes.c_int * 10)()
    fake.L.fake_int4_walk(64, 32, 512, v)
    least_a, least_b1, least_b2, *where, past = v
    assert least_a >= 2 and least_b1 >= 2 and least_b2 >= 2, (least_a, least_b1, least_b2, where)
    assert past <= 0


def test_experts_of_the_largest_size_launch(fake):
    args = (ctypes.c_int * 3)()
    for group, zeros in ((0, 0), (32, 1), (128, 0)):
        h = fake.experts(group, zeros, num_experts=512, top_k=32)
        fake.L.fake_clear()
        assert fake.run_experts(h, 64) == _lib.EP_OK, fake.message()
        (name, _, grid, _, smem), = fake.launches()
        assert grid == (152, 1, 1) and smem <= 227 * 1024
        if group:
            fake.L.fake_int4_args(0, args)
            assert "int4_kernel" in name and args[0] == smem
        else:
            fake.L.fake_experts_args(0, args)
            assert "experts_kernel" in name and args[0] >= 2 and args[1] >= 2
        assert fake.L.ep_experts_destroy(h) == _lib.EP_OK


def test_handles_of_two_devices_launch_on_both(fake):
    """A kernel's shared-memory limit belongs to the device that was current when it was set."""
    made = []
    for device in (0, 1, 0):
        fake.L.fake_device(device)
        made.append((device, fake.router(hidden=256), fake.experts(), fake.experts(64), fake.linear()))
    for device, router, dense, int4, linear in made:
        fake.L.fake_device(device)
        fake.L.fake_clear()
        for n in (1, 60, 300, 20000):
            assert fake.route(router, n, 256)[0] == _lib.EP_OK, (device, n, fake.message())
        for h in (dense, int4):
            assert fake.run_experts(h, 5) == _lib.EP_OK, (device, fake.message())
        assert fake.run_linear(linear, 5) == _lib.EP_OK, (device, fake.message())
        assert [l[1] for l in fake.launches()] == [device] * 7
    for device, router, dense, int4, linear in made:
        fake.L.fake_device(device)
        assert fake.L.ep_router_destroy(router) == fake.L.ep_experts_destroy(dense) == _lib.EP_OK
        assert fake.L.ep_experts_destroy(int4) == fake.L.ep_linear_destroy(linear) == _lib.EP_OK


def test_layer_queues_nothing_unless_both_calls_will_be(fake):
    router, h = fake.router(hidden=256), fake.experts()
    words = fake.L.fake_error_words()  # of the experts, which were made last
    fake.L.fake_clear()
    words[0] = words[7] = 1  # a wait of an earlier call ran out
    assert fake.run_layer(router, h, 3) == _lib.EP_ERR_CUDA and "ran out" in fake.message()
    assert fake.launches() == []
    assert fake.run_layer(router, h, 3) == _lib.EP_OK and len(fake.launches()) == 2
    fake.L.fake_device(1)
    elsewhere = fake.experts()
    fake.L.fake_device(0)
    fake.L.fake_clear()
    for n in (0, 3):
        assert fake.run_layer(router, elsewhere, n) == _lib.EP_ERR_INVALID_ARG and "device 1" in fake.message()
    assert fake.launches() == []
    for x in (h, elsewhere):
        fake.L.ep_experts_destroy(x)
    fake.L.ep_router_destroy(router)


def test_destroy_waits_for_the_handles_device(fake):
    """Queued work still uses a handle's workspace, which its owner may hand out again once destroy has returned, and its
    error words, which destroy frees."""
    fake.L.fake_device(1)
    made = [("ep_router_destroy", fake.router(hidden=256)), ("ep_experts_destroy", fake.experts()),
            ("ep_experts_destroy", fake.experts(64)), ("ep_linear_destroy", fake.linear())]
    fake.L.fake_device(0)  # the device that is current at destroy may be another
    for destroy, h in made:
        fake.L.fake_clear()
        assert getattr(fake.L, destroy)(h) == _lib.EP_OK
        calls = fake.calls()
        assert calls[0] == "cudaDeviceSynchronize 1" and "cudaFreeHost" in calls[1:], calls
    h = fake.router(hidden=256)
    fake.L.fake_clear()
    assert fake.route(h, 1, 256)[0] == _lib.EP_OK
    assert fake.launches()[0][1] == 0  # the current device is as it was
    fake.L.ep_router_destroy(h)


def test_rows_that_the_kernels_cannot_count_are_refused(fake):
    """Rows are int32 in the kernels, with a tile's or a slice's room above the last one."""
    for E in (64, 512):  # tiles of many tokens; slices of 256
        h = fake.router(hidden=8, num_experts=E)
        for n in (2**31 - 1, 2**31 - 511):
            fake.L.fake_clear()
            size = ctypes.c_size_t(0)
            assert fake.L.ep_router_workspace_size(h, n, ctypes.byref(size)) == _lib.EP_ERR_INVALID_ARG
            assert fake.L.ep_router_run(h, 4096, 8, n, 4096, 4096, 4096, 1 << 40, None) == _lib.EP_ERR_INVALID_ARG
            assert "num_tokens" in fake.message() and fake.launches() == []
        fake.L.ep_router_destroy(h)
    h = fake.router(hidden=8, num_experts=64)
    fake.L.fake_clear()
    assert fake.route(h, 2**31 - 512, 8)[0] == _lib.EP_OK, fake.message()
    (_, _, (tiles, splits, _), _, _), = fake.launches()
    args = (ctypes.c_int * 2)()
    fake.L.fake_router_args(0, args)
    assert splits == 1 and args[0] <= 128 and 2**31 - 512 <= tiles * args[0] <= 2**31 - 1
    fake.L.ep_router_destroy(h)


def test_binding_refuses_rows_that_do_not_fit_the_abi():
    """The C ABI's counts are int: 2^32 + 5 rows would be taken for 5."""
    h = EpRouter.__new__(EpRouter)
    h._h, h._index, h.device = None, -1, torch.device("cpu")
    x = torch.zeros(1, 8, dtype=torch.bfloat16)
    assert h._rows(x.expand(2**31 - 1, 8), 8, torch.bfloat16)[0] == 2**31 - 1
    for n in (2**31, 2**32 + 5):
        with pytest.raises(ValueError, match="rows"):
            h._rows(x.expand(n, 8), 8, torch.bfloat16)


def test_experts_past_the_ids_are_refused(fake):
    """An id is int32: with experts numbered past 2^31 - 1, id - first_expert of a negative id wrapped to one of them."""
    size = ctypes.c_size_t(0)

    def status(first, E):
        w = [_lib.EpWeightC(4096, 0, 0, 0)] * 2
        cfg = _lib.EpExpertsConfigC(E, first, 2, 64, 64, 8, *w)
        return fake.L.ep_experts_workspace_size(ctypes.byref(cfg), ctypes.byref(size))

    for first, E in ((0, 512), (2**31 - 8, 8), (2**31 - 1, 1)):
        assert status(first, E) == _lib.EP_OK, fake.message()
    for first, E in ((2**31 - 7, 8), (2**31 - 1, 2), (2**31 - 4, 512)):
        assert status(first, E) == _lib.EP_ERR_INVALID_ARG and "first_expert" in fake.message()
