"""The accounts that a CTA pair settles before it ends after a wait ran out (stage_debt in
csrc/pair_drain.cuh, compiled for the host), on a model of the pair's ring of stages: whichever uses the
two CTAs had come to, and however many of their copies had landed, each barrier's phase ends with the last
copy under way -- not before, and not never."""
from __future__ import annotations

import ctypes
import itertools
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "tests", "pair_drain_host.cu")
CSRC = os.path.join(ROOT, "mixture_experts_ffn_renorm_gb300", "csrc")
LIB = os.path.join(ROOT, "_build", "libpair_drain_host.so")
STAGES = 6


@pytest.fixture(scope="module")
def debt():
    cc = next((c for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc")
               if c and os.path.exists(c)), None)
    if cc is None:
        pytest.skip("nvcc not found")
    os.makedirs(os.path.dirname(LIB), exist_ok=True)
    subprocess.check_call([cc, "-gencode", "arch=compute_103a,code=sm_103a", "-O1", "-std=c++17", "-shared", "-Xcompiler",
                           "-fPIC", "-I", os.path.join(ROOT, "include"), "-I", CSRC, SRC, "-o", LIB])
    lib = ctypes.CDLL(LIB)
    fn, gathers = lib.stage_debt_host, lib.gather_debt_host
    gathers.restype = ctypes.c_uint

    def run(i, even, odd, size):
        out = (ctypes.c_uint * 3)()
        fn(i, even, odd, size, out)
        return out[0], out[1], out[2]
    run.gathers = gathers
    return run


class Barrier:
    """One phase of an mbarrier: ends when no arrival is pending and no bytes are outstanding."""

    def __init__(self, arrivals):
        self.pending, self.tx, self.ended = arrivals, 0, False

    def settle(self):
        if self.pending == 0 and self.tx == 0:
            self.ended = True

    def arrive(self, expect=0):
        assert self.pending > 0 and not self.ended
        self.tx += expect
        self.pending -= 1
        self.settle()

    def complete(self, size):
        assert not self.ended
        self.tx -= size
        self.settle()


@pytest.mark.parametrize("base", [0, 4, 29])
def test_every_phase_ends_with_its_last_copy(debt, base):
    rnd = random.Random(base)
    consumed = base                               # every role has come to here, and no further than STAGES on
    for even, odd in itertools.product(range(consumed, consumed + STAGES + 1), repeat=2):
        n = max(even, odd)
        for i in range(max(0, n - STAGES), n):
            size = rnd.choice([20480, 24576, 32768])
            if i < consumed:                      # landed, and used
                assert debt(i, even, odd, size) == (1, 0, 0)
                continue
            for landed in itertools.product([False, True], repeat=2):
                bar, under_way = Barrier(1), 0
                for cta, upto in enumerate((even, odd)):
                    if i < upto:
                        if cta == 0:
                            bar.arrive(2 * size)  # armed for both
                        if landed[cta]:
                            bar.complete(size)
                        else:
                            under_way += 1
                is_open, expect, complete = debt(i, even, odd, size)
                assert is_open == (1 if i < even or i < odd else 0)
                if not is_open:
                    assert expect == complete == 0
                    continue
                if complete:
                    bar.complete(complete)
                if expect:
                    bar.arrive(expect)
                while under_way:
                    assert not bar.ended
                    under_way -= 1
                    bar.complete(size)
                assert bar.ended and bar.tx == 0 and bar.pending == 0


def test_gathered_rows_arrivals_are_made_up(debt):
    # even, odd: copies; the even CTA's two gatherer warps and the odd one's relay stopped anywhere in the ring
    rnd = random.Random(7)
    for even, odd, warp0, warp1, relay in (tuple(rnd.randint(9, 9 + STAGES) for _ in range(5)) for _ in range(4000)):
        n = max(even, odd)
        for i in range(n - STAGES, n):
            if i < 9:
                assert debt.gathers(i, warp0, warp1, relay) == 0
                continue
            bar, size, under_way = Barrier(1 + 64 + 1), 16384, []
            if i < even:
                bar.arrive(2 * size)
            for there, k in ((i < warp0, 32), (i < warp1, 32), (i < relay, 1)):
                # a gatherer's arrival comes when its own copies have landed
                under_way += [bar.arrive] * k if there else []
            under_way += [lambda: bar.complete(size)] * ((i < even) + (i < odd))
            rnd.shuffle(under_way)
            for _ in range(rnd.randint(0, len(under_way))):
                under_way.pop()()
            _, expect, complete = debt(i, even, odd, size)
            if complete:
                bar.complete(complete)
            if expect:
                bar.arrive(expect)
            for _ in range(debt.gathers(i, warp0, warp1, relay)):
                bar.arrive()
            while under_way:
                assert not bar.ended
                under_way.pop()()
            assert bar.ended and bar.tx == 0 and bar.pending == 0
