"""The rings of the 4-bit kernel on the CPU: its barriers' phases in a model, for the stage counts that calls have.

Two pairs of worker groups take the units of a ring in turn: a pair waits for every second unit only. A wait on a
barrier's parity passes when the phase that is under way has the other parity, so it also passes where the phase before
the one that is meant has not completed yet. Copies may land in any order."""
import os
import shutil
import subprocess

import pytest

from combine_topk_ids_dest_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")


def early(stages, rounds=3):
    """A unit that some order of landing copies lets a pair take before its copy has landed, or None.

    Unit u lies in stage u % stages and is phase u // stages of that stage's barrier. The copies are issued in order, each
    once its stage's unit before has been taken; every order of issuing, landing and taking is gone through."""
    units = rounds * stages
    begin = (0, (0, 1), 0)  # units issued, each pair's next one, the set of those that have landed
    todo, seen = [begin], {begin}
    while todo:
        issued, nexts, landed = todo.pop()
        after = []
        if issued < units:
            before = issued - stages
            if before < 0 or before < nexts[before % 2]:
                after.append((issued + 1, nexts, landed))
        for u in range(max(0, issued - stages), issued):
            if not landed >> u & 1:
                after.append((issued, nexts, landed | 1 << u))
        for pair in (0, 1):
            u = nexts[pair]
            if u >= units:
                continue
            phase, done = u // stages, 0  # the barrier's phases that have completed
            while done * stages + u % stages < issued and landed >> (done * stages + u % stages) & 1:
                done += 1
            if (done & 1) != (phase & 1):  # the wait passes
                if not landed >> u & 1:
                    return u
                moved = (u + 2, nexts[1]) if pair == 0 else (nexts[0], u + 2)
                after.append((issued, moved, landed))
        for s in after:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return None


def test_the_model_tells_odd_rings_from_even_ones():
    assert [early(s, 2) is None for s in (2, 3, 4, 5, 6)] == [True, False, True, False, True]


@pytest.fixture(scope="module")
def rings(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("rings") / "int4_rings")
    r = subprocess.run(["g++", "-std=c++17", "-O2", "-I", os.path.join(CUDA, "include"), "-I", build.INCLUDE, "-I", build.CSRC,
                        os.path.join(ROOT, "tests", "c", "int4_rings.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    return [tuple(map(int, line.split())) for line in out.splitlines()]


def test_no_wait_passes_before_its_copy_has_landed(rings):
    counts = sorted({n for r in rings for n in r})
    assert rings and counts[0] >= 2
    for n in counts:
        if n <= 6:
            assert early(n, 2) is None, f"a ring of {n} stages"
        # with an even number a pair's stages are its own: it has waited for each of their phases
        assert n % 2 == 0, f"a ring of {n} stages: {[r for r in rings if n in r][:4]}"
