"""What the MoE operators' host code launches, on the CPU over a stand-in runtime: sizes that the
kernels' buffers hold, for every accepted call."""
import ctypes

import pytest

from combine_topk_ids_dest_gb300 import _lib
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
