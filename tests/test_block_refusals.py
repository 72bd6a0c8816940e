"""CPU checks, over a stand-in runtime, of which calls of the norm and the feed-forward block are refused and which are not:
results beside their operands, calls without rows, waits that ran out, workspaces."""
import ctypes

import pytest

from combine_topk_ids_dest_gb300 import _lib
from test_block_host import AT, H, I, T, _back, _backward, _ffn, _norm, _run, clean, fake, ffn  # noqa: F401

INVALID, OK = _lib.EP_ERR_INVALID_ARG, _lib.EP_OK


def test_gradients_of_no_rows_on_the_weights_refused(fake, ffn):
    """They are written (0) without any row too."""
    assert _back(fake, n=0, dweight=AT[0]) == INVALID and "dweight overlaps weight" in fake.message(), fake.message()
    for kw, frag in ((dict(dgate_up=AT[0]), "dgate_up overlaps gate_up"), (dict(ddown=AT[1] + 32), "ddown overlaps down"),
                     (dict(ddown=AT[0]), "ddown overlaps gate_up"), (dict(ddown=AT[6] + 64), "ddown overlaps dgate_up")):
        assert _backward(fake, ffn, n=0, **kw) == INVALID and frag in fake.message(), fake.message()
    assert fake.launches() == []
    # operands that have no rows may be anything
    assert _back(fake, n=0, dy=0, h=0, dh=0, dx=0) == OK, fake.message()
    assert _backward(fake, ffn, n=0, dy=0, x=0, saved=0, dx=0, workspace=None) == OK, fake.message()


def test_columns_of_one_buffer_do_not_overlap(fake, ffn):
    """x and its results as columns of a wider buffer's rows: no element is both."""
    wide, at = 2 * H, AT[1]
    rows = dict(x=at, x_stride=wide, residual=AT[2], residual_stride=wide, residual_out=at + 2 * H, residual_out_stride=wide,
                out=AT[2] + 2 * H, out_stride=wide)
    assert _norm(fake, **rows) == OK, fake.message()
    for kw in (dict(residual_out=at + 2 * H - 16), dict(residual_out=at + 16), dict(residual_out=at + 4 * H - 16),
               dict(residual_out=at + 2 * H, residual_out_stride=wide + 8), dict(residual_out=at + 2 * H, residual_out_stride=H)):
        assert _norm(fake, **dict(rows, **kw)) == INVALID and "overlaps" in fake.message(), (kw, fake.message())
    # a row further on, the columns beside still, or not
    assert _norm(fake, **dict(rows, residual_out=at + 2 * wide + 2 * H)) == OK, fake.message()
    assert _norm(fake, **dict(rows, residual_out=at + 2 * wide)) == INVALID
    assert _norm(fake, **dict(rows, residual_out=at - 2 * wide + 2 * H)) == OK, fake.message()
    assert _norm(fake, **dict(rows, residual_out=at - 2 * wide)) == INVALID
    back = dict(dy=at, dy_stride=wide, dx=at + 2 * H, dx_stride=wide)
    assert _back(fake, **back) == OK, fake.message()
    assert _back(fake, **dict(back, dx=at + 16)) == INVALID
    at = AT[9]  # AT[0] and AT[1] are the block's weights
    assert _run(fake, ffn, x=at, x_stride=wide, out=at + 2 * H, out_stride=wide) == OK, fake.message()
    at = AT[9]  # AT[0] and AT[1] are the block's weights
    assert _run(fake, ffn, x=at, x_stride=wide, out=at + 2 * H - 2, out_stride=wide) == INVALID
    assert _backward(fake, ffn, dy=at, dy_stride=wide, dx=at + 2 * H, dx_stride=wide) == OK, fake.message()
    # rows of another kind may lie between, too: a row of the weights' gradients is no row of x
    assert _backward(fake, ffn, dy=at, dy_stride=wide, dgate_up=at + 2 * H) == INVALID


def _size(fake, h, call, n):
    size = ctypes.c_size_t(0)
    assert fake.L.ep_ffn_workspace_size(h, call, n, ctypes.byref(size)) == OK
    return size.value


def test_ffn_workspaces_are_what_the_calls_use(fake):
    """h's rows; for the gradients those of gate and up, and parts of tiles only where pairs share them."""
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    shared = 0
    for hidden, intermediate in ((8, 8), (2056, 1400), (512, 8192), (4096, 14336)):
        st, h = _ffn(fake, hidden=hidden, intermediate=intermediate, gate_up=AT[9], down=AT[10])
        assert st == OK
        for n in (1, 64, 300, 700, 1999, 4096):
            rows = up(n * intermediate * 2)
            assert _size(fake, h, 0, n) == _size(fake, h, 1, n) == rows
            both = rows + up(n * intermediate * 4)
            size = _size(fake, h, 2, n)
            assert size == both or size == both + 2 * 76 * 256 * 128 * 4
            shared += size > both
            # it is enough for any of the gradients, one byte less is refused where a call uses all
            far = dict(zip(("dy", "x", "saved", "dx", "dgate_up", "ddown"), (k << 48 for k in range(1, 7))))
            strides = dict(dy_stride=hidden, x_stride=hidden, dx_stride=hidden)
            for skip in ((), ("dx",), ("dgate_up",), ("ddown",), ("dx", "ddown"), ("dgate_up", "ddown"), ("dx", "dgate_up")):
                ops = dict(far, **{k: 0 for k in skip})
                assert _backward(fake, h, n, bytes=size, **strides, **ops) == OK, fake.message()
            refused = [_backward(fake, h, n, bytes=size - 1, **strides, **dict(far, **{k: 0 for k in skip})) == INVALID
                       for skip in ((), ("dx",), ("dgate_up",), ("ddown",), ("dx", "ddown"), ("dgate_up", "ddown"), ("dx", "dgate_up"))]
            assert any(refused)
        assert _size(fake, h, 2, 0) == _size(fake, h, 0, 0) == 0
        assert fake.L.ep_ffn_destroy(h) == OK
    assert 0 < shared < 24


def test_ffn_backward_reports_a_wait_that_ran_out_once(fake, ffn):
    words = fake.L.fake_error_words()
    fake.L.fake_clear()
    words[0] = words[4] = 1
    assert _backward(fake, ffn) == _lib.EP_ERR_CUDA and "ran out" in fake.message() and fake.launches() == []
    assert _backward(fake, ffn) == OK and len(fake.launches()) == 2
