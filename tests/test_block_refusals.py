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
