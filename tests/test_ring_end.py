"""The end of a ring of copies after an expired wait (csrc/vh_ring.cuh): whoever asked for copies stopped where it was, and what a
stage's phase then lacks is made up for, so that it ends when the copies have landed.  The counts against a model of the barriers on
the CPU; the barriers and copies themselves in a small kernel."""
import ctypes
import itertools
import os
import random
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "verify_head_gb300", "csrc")

WRAP = """
#include "vh_ring.cuh"
extern "C" void lack(unsigned j, const unsigned* asked, int ctas, unsigned bytes, unsigned* out) {
    const unsigned one[1] = {asked[0]}, two[2] = {asked[0], ctas > 1 ? asked[1] : 0u};
    const vh::ring::Lack l = ctas == 1 ? vh::ring::lack<1>(j, one, bytes) : vh::ring::lack<2>(j, two, bytes);
    out[0] = l.arrive; out[1] = l.expect; out[2] = l.give;
}
"""


@pytest.fixture(scope="module")
def lack(tmp_path_factory):
    d = tmp_path_factory.mktemp("ring")
    src, lib = d / "lack.cpp", d / "lack.so"
    src.write_text(WRAP)
    subprocess.run(["g++", "-x", "c++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I" + CSRC, str(src), "-o", str(lib)], check=True)
    f = ctypes.CDLL(str(lib)).lack

    def call(j, asked, size):
        out = (ctypes.c_uint * 3)()
        f(j, (ctypes.c_uint * len(asked))(*asked), len(asked), size, out)
        return tuple(out)
    return call


def phase_ends(lack, j, counts, sizes, rng):
    """One phase of a barrier of two arrivals, in a random order of what happens to it: the askers' arrivals, the landing copies, and what
    settling adds.  Returns whether it ends, and whether a copy had not landed by then."""
    events = []  # (arrivals, bytes expected, bytes that land, whether a copy)
    for asked, size in zip(counts, sizes):
        ctas = len(asked)
        if j < asked[0]:
            events.append((1, ctas * size, 0, False))
        events += [(0, 0, size, True) for n in asked if j < n]
        arrive, expect, give = lack(j, asked, size)
        if give:
            events.append((0, 0, give, False))
        if arrive:
            events.append((1, expect, 0, False))
    rng.shuffle(events)
    pending, tx, ended, landed_after = 2, 0, False, False
    for a, e, b, copy in events:
        landed_after |= ended and copy
        tx += e - b
        pending -= a
        ended |= pending == 0 and tx == 0
    return ended and pending == 0 and tx == 0, landed_after


@pytest.mark.parametrize("ctas", [1, 2])
def test_every_phase_that_was_asked_for_ends(lack, ctas):
    rng = random.Random(ctas)
    sizes, stages, taken = (18432, 20480), 3, 4  # `taken` uses are over; nobody is more than the ring's length ahead
    for n in itertools.product(range(taken, taken + stages + 1), repeat=2 * ctas):
        counts = (n[:ctas], n[ctas:])
        for j in range(taken, max(n)):
            for _ in range(4):
                ended, early = phase_ends(lack, j, counts, sizes, rng)
                assert ended and not early, (counts, j)


def test_nothing_is_added_where_all_have_asked(lack):
    assert lack(5, (6,), 100) == (0, 0, 0) and lack(5, (6, 6), 100) == (0, 0, 0)
    assert lack(5, (6, 5), 100) == (0, 0, 100) and lack(5, (5, 6), 100) == (1, 100, 0) and lack(5, (5, 5), 100) == (1, 0, 0)


@pytest.mark.gpu
def test_on_the_gpu(tmp_path):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from verify_head_gb300 import buildlib
    lib = str(tmp_path / "ring_end.so")
    subprocess.run([buildlib.nvcc(), *buildlib.ARCH, *buildlib.NVCC_FLAGS, "-shared", "-cudart", "shared", "-I" + CSRC,
                    os.path.join(HERE, "ring_end.cu"), "-o", lib, "-Xlinker", "-rpath=/usr/local/cuda/lib64"], check=True)
    f = ctypes.CDLL(lib).ring_end
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    stages, size = 4, 4096
    rng = random.Random(0)
    for ctas in (1, 2):
        total = stages * 2 * ctas * size
        src = torch.randint(1, 256, (total,), dtype=torch.uint8, device="cuda")
        every = list(itertools.product(range(stages + 1), repeat=2 * ctas))
        for n in every if ctas == 1 else rng.sample(every, 60):
            counts = torch.tensor(n, dtype=torch.int32, device="cuda")
            done, out = torch.zeros(stages, dtype=torch.int32, device="cuda"), torch.empty_like(src)
            torch.cuda.synchronize()
            assert f(p(src), p(counts), ctas, p(done), p(out)) == 0
            torch.cuda.synchronize()
            assert done.tolist() == [int(j < max(n)) for j in range(stages)], n
            asked = torch.tensor([[[j < n[o * ctas + c] for c in range(ctas)] for o in range(2)] for j in range(stages)])
            assert torch.equal(out.view(-1, size), src.view(-1, size) * asked.view(-1, 1).cuda()), n
