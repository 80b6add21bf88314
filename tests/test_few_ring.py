"""Which copies a block of the few-row attention waits for before it ends when a wait of
its readers gave up: every copy that nobody has seen arrive, by the phase that its stage is in.
The rule (csrc/few_ring.h, plain C++) is run here over random orders of events.
"""

import ctypes
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "w8a16_linear_gb300", "csrc")


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    d = tmp_path_factory.mktemp("few_ring")
    src, lib = d / "f.cpp", d / "f.so"
    src.write_text('#include "few_ring.h"\nextern "C" int f(int n, int o, int s, int r, int j) '
                   '{ return w8::unread_filling(n, o, s, r, j); }\n')
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    subprocess.run([cxx, "-std=c++17", "-shared", "-fPIC", f"-I{CSRC}", str(src), "-o", str(lib)], check=True)
    return ctypes.CDLL(str(lib)).f


@pytest.mark.parametrize("step,ring", [(1, 2), (1, 3), (2, 3), (2, 5)])
def test_copies_that_nobody_has_seen(rule, step, ring):
    rng = random.Random(ring * 10 + step)
    for _ in range(3000):
        following = list(range(step))                # the copiers' next fillings
        filled, read, landed = set(), set(), set()
        for _ in range(rng.randrange(60)):
            who = rng.randrange(step)
            e = following[who]
            if rng.random() < 0.5:                   # a copy, where the stage's reader has released it
                if e < ring or e - ring in read:
                    filled.add(e)
                    following[who] += step
            else:                                    # a copier's fillings are read in their order
                left = sorted(x for x in filled - read if x % step == who)
                if left:
                    read.add(left[0])
        landed = read | {e for e in filled if rng.random() < 0.5}
        asked = set()
        for who in range(step):
            for j in range(1, ring + 1):
                e = rule(following[who], following[1 - who] if step == 2 else 0, step, ring, j)
                if e >= 0:
                    asked.add(e)
        assert filled - read <= asked <= filled
        for e in asked:
            # the barrier's phases that are complete are those of the stage's landed fillings: a wait for
            # a phase's parity ends when that phase, and not the next, is the last complete one
            later = [x for x in filled if x % ring == e % ring and x > e]
            assert not later
            complete = sum(1 for x in landed if x % ring == e % ring)
            assert complete in (e // ring, e // ring + 1)
