"""The tiles of the products in 8-bit integers, checked on the host against their
source: the waits on copies into LDS, what a copy may overwrite, and that the GPU
tests' sizes reach every kernel that the choice knows."""

import math
import os
import re

import pytest

import test_gpu_int8 as G

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = open(os.path.join(ROOT, "nf4_bit_weight_amd", "csrc", "nf4_int8.hip")).read()
TILES = {n: tuple(int(x) for x in v.split(",")) for n, v in re.findall(r"using (Tile\w+) = Tile<([\d, ]+)>;", SRC)}


def wait_count(pattern):
    m = re.search(pattern, SRC)
    assert m, pattern
    return m.group(1)


LATER = wait_count(r'if \(later\) asm volatile\("s_waitcnt vmcnt\(%0\)\\n\\ts_barrier" :: "n"\(([^"]+)\) :')
FIRST = wait_count(r'if \(steps >= NS - 1\) asm volatile\("s_waitcnt vmcnt\(%0\)\\n\\ts_barrier" :: "n"\(([^"]+)\) :')


def replay(NS, S, C, steps):
    """One wave's copies in the order the kernel issues them (all waves alike).  Checks that a
    step has landed before its first read and that no copy lands on a step that may still be read."""
    env = dict(NS=NS, C=C)
    later, first = eval(LATER, {}, env), eval(FIRST, {}, env)
    assert 0 <= later < 64 and 0 <= first < 64                  # what the counter holds
    issued, done = [], 0                                        # the step of each copy, how many have surely landed
    passed = -1                                                 # steps up to here are read by nobody any more

    def copy(step):
        assert step - NS <= passed, f"step {step} copied over step {step - NS} too early"
        issued.append(step)

    def wait(n):
        nonlocal done
        done = max(done, len(issued) - n)

    def landed(step):
        assert issued.count(step) == C, f"step {step} is not copied yet"
        assert max(i for i, s in enumerate(issued) if s == step) < done, f"step {step} is read before it landed"

    for k in range(min(steps, NS - 1)):
        for _ in range(C):
            copy(k)
    if steps == 0:
        return
    wait(first if steps >= NS - 1 else 0)
    landed(0)
    part = -(-C // S)

    def step(k, more, fetch, rest):
        nonlocal passed
        for s in range(S):
            last = s == S - 1
            if last and more:
                wait(later if fetch else 0)
                passed = max(passed, k - 1)                     # behind the barrier every wave is done with step k - 1
                landed(k + 1)
            at = 0 if last else (s + 1) * part
            if fetch if last else rest:
                for i in range(at, min(at + part, C)):
                    copy(k - 1 + NS if last else k - 2 + NS)
    k = 0
    if NS - 1 < steps:
        step(0, True, True, False)
        k = 1
        while k + NS - 1 < steps:
            step(k, True, True, True)
            k += 1
        step(k, True, False, True)
        k += 1
    while k + 1 < steps:
        step(k, True, False, False)
        k += 1
    if k < steps:
        step(k, False, False, False)
    assert issued.count(steps - 1) == C and len(issued) == C * steps


@pytest.mark.parametrize("name", sorted(TILES))
def test_copies_land_before_they_are_read(name):
    BM, BN, WX, WY, BK, NS = TILES[name]
    C = (BM + BN) // (1024 // BK) // (WX * WY)
    assert NS >= 3 and BM % (1024 // BK * WX * WY) == 0 and BN % (1024 // BK * WX * WY) == 0
    assert NS * (BM + BN) * BK <= 160 * 1024
    for steps in range(0, 40):
        replay(NS, BK // 32, C, steps)


def test_the_replay_sees_a_lost_wait():
    for wrong in ("(NS - 2) * C", "(NS - 3) * C + 1"):
        global LATER
        kept, LATER = LATER, wrong
        try:
            with pytest.raises(AssertionError):
                replay(5, 4, 4, 20)
        finally:
            LATER = kept


def table(name):
    m = re.search(name + r"\[\] = \{(.*?)\};", SRC)
    return [tuple(int(x) for x in t.split(",")) for t in re.findall(r"\{([\d, ]+)\}", m.group(1))]


def best_shape(M, N, E=0, cus=256):
    best = None
    for i, (bm, bn, cost) in enumerate(table("kGroupedShapes" if E else "kShapes")):
        if not bm:
            continue
        rows = -(-M // bm)
        if E:
            experts = min(E, M)
            rows = experts * max(1.1, M / experts / bm + 0.5)
        c = math.ceil(rows * -(-N // bn) / cus) * cost
        if best is None or c < best[1]:
            best = (i, c)
    return best[0]


def few_rows(M, N, cus=256):
    return M <= 16 or (M <= 64 and (N + 63) // 64 < cus // 2)


def channels(M, N, K, cus=256):
    blocks = -(-K // 128)
    groups = 8 // (8 if blocks >= 8 else 4 if blocks >= 4 else 2 if blocks >= 2 else 1)

    def fills(mt, nt):
        return -(-M // (16 * mt)) * -(-N // (16 * nt * groups)) * 8 >= cus * 7
    for shape in ((2, 2), (2, 1)) if M > 16 else ((1, 4), (1, 2)):
        if fills(*shape):
            return shape
    return 1, 1


def test_the_sizes_reach_every_kernel():
    """The choice of nf4_int8.hip once more, in Python, on 256 compute units."""
    assert re.search(r"a\.M <= 16 \|\| \(a\.M <= 64 && \(a\.N \+ 63\) / 64 < cus / 2\)", SRC)
    tiles = {best_shape(M, N) for M, N, K in G.SHAPES if not few_rows(M, N)}
    assert tiles == {0, 1, 2, 3, 4}
    few = {channels(M, N, K) for M, N, K in G.SHAPES if few_rows(M, N)}
    assert few == {(1, 1), (1, 2), (1, 4), (2, 1), (2, 2)}
    one = {M == 1 for M, N, K in G.SHAPES if few_rows(M, N) and M * -(-K // 128) * 128 <= (16384 if M == 1 else 8192)}
    assert one == {True, False}                                 # the form of one launch, with one row and with several
    grouped = {best_shape(T * k, N, E) for T, E, k, N, K, empty in G.GROUPED}
    assert grouped == {0, 2, 4}
