"""The tolerance of a row's sum in fp32, rows_reference.sum_tol(V) = (ceil(V / 512) + 72) * 2^-24, from what the kernels
do, at every launch shape.

A block has 256 threads (224 of them read in distillation) and a row between 1 and 16 blocks; from some 300 rows on it
is one block, so that a thread has more columns than V / 512.  They are not added one after another: a thread sums a
tile of kVecs vectors of N columns first, in two halves (or, where a value needs a guard, in one run), and adds the
tile's sum to its own.  A term thus goes through at most
    kVecs N (a guarded tile) + the thread's tiles + 5 (the warp's shuffles)
additions of half a step, 2^-24 each, before the sums go on in 64 bits; references are powers of two and scale exactly.
To these come 2^-22 for the exponential and the rounding of its argument, 2^-24 ln 2 of |argument|, whose average over
the row's distribution is at most log2 V + 1 < 22."""
import math
import os
import re

import pytest

from tests.rows_reference import sum_tol

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "draft_block_causal_b200", "csrc")


def constant(source: str, name: str) -> int:
    with open(os.path.join(CSRC, source)) as f:
        text = f.read()
    (value,) = re.findall(rf"constexpr int {name} = (\d+);", text)
    return int(value)


def units(tiles: int, vecs: int, N: int) -> float:
    return vecs * N + tiles + 5 + 4 + 22 * math.log(2)


@pytest.mark.parametrize("source,idle", [("top_scan.cuh", 0), ("distill.cu", 32)])
@pytest.mark.parametrize("N", [4, 8])
def test_sum_tolerance_covers_every_launch_shape(source, idle, N):
    threads, per = constant(source, "kThreads") - idle, constant(source, "kVecs")
    assert (threads, per) == (256 - idle, 4)
    for V in list(range(1, 3000, 7)) + [2 ** e + d for e in range(12, 21) for d in (-1, 0)] + [50001, 151936]:
        vecs = -(-V // N)
        for cluster in (1, 2, 4, 8, 16):  # one block is the most that a thread can have to add
            tiles = -(-(-(-vecs // cluster)) // (threads * per))
            assert units(tiles, per, N) * 2.0 ** -24 <= sum_tol(V), (V, cluster)


def test_a_thread_of_a_long_row_has_more_columns_than_512_threads_would_leave_it():
    """400 rows of 151936 fp32 have a block each: 596 columns a thread in 38 tiles, 79 units of the 369 allowed."""
    vecs = 151936 // 4
    assert -(-vecs // 256) * 4 == 596 > math.ceil(151936 / 512) + 32
    assert 78 < units(-(-vecs // 1024), 4, 4) < 79 and sum_tol(151936) * 2 ** 24 == 369
