"""The plans of the feed-forward block's launches, on the CPU: every chunk of every tile is multiplied once, within the
buffers, and what a pair of blocks waits for, last of all, is written by a lower one that does not wait before."""
import ctypes
import os
import random
import subprocess

import pytest

from combine_topk_ids_dest_gb300 import build
from fake_runtime import CUDA, ROOT, Fake


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    folder = tmp_path_factory.mktemp("plans")
    Fake(folder)  # builds the objects
    so = os.path.join(str(folder), "libffn_plan.so")
    objects = [os.path.join(build.BUILD, os.path.basename(s) + ".o") for s in build.sources()]
    cmd = ["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-I", os.path.join(CUDA, "include"), "-I",
           build.INCLUDE, "-I", build.CSRC, os.path.join(ROOT, "tests", "c", "ffn_plan.cpp"),
           os.path.join(ROOT, "tests", "c", "fake_runtime.cpp"), *objects, "-o", so, "-ldl", "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return ctypes.CDLL(so)


def _look(plans, T, H, I, sms=152, wanted=7):
    v = (ctypes.c_longlong * 8)()
    bad = plans.ffn_look(T, H, I, sms, wanted, v)
    assert bad == 0, (bad, T, H, I, sms, wanted)
    return list(v)


@pytest.mark.parametrize("H,I", [(8, 8), (72, 40), (136, 264), (520, 200), (1032, 520), (2056, 1400), (4096, 14336),
                                 (7168, 2048), (65536, 8), (8, 65536)])
def test_any_number_of_rows(plans, H, I):
    for T in [*range(1, 70), *range(70, 2200, 37), 4096, 8191, 16384, 20011]:
        _look(plans, T, H, I, wanted=1 + T % 7)


def test_drawn_sizes_and_machines(plans):
    rng = random.Random(1)
    for _ in range(1500):
        T, H, I = (max(1, int(2 ** rng.uniform(0, 13))) for _ in range(3))
        _look(plans, T, 8 * H, 8 * I if H * I < 1 << 18 else 8, sms=rng.choice([2, 20, 132, 148, 152, 160, 200]),
              wanted=rng.randint(1, 7))


@pytest.mark.parametrize("T,H,I", [(1999, 2056, 1400), (4096, 4096, 14336), (700, 1024, 9000)])
def test_gradients_shares_are_even(plans, T, H, I):
    """Tiles of T / 64 and of 2 I / 64 chunks over 76 pairs: whole ones alone would differ by a tile. What is left are edges
    that are not cut because a few chunks are behind them."""
    v = _look(plans, T, H, I)
    assert v[3] <= 1.1 * v[7] / 76
