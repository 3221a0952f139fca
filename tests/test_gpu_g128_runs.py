"""The product with a scale per 128 on both sides of the mean run length (rows of one source for one expert) from which whole
halves of a tile are read where they arrived, on the GPU against float64.  Bounds: tests/g128_ref.py."""

import pytest

from test_gpu_g128 import _lib, run, split  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,qtype", [("bf16", "e4m3fn"), ("fp16", "e5m2")])
@pytest.mark.parametrize("W,e,sizes,K,N", [
    (2, 3, [480, 280, 380], 256, 328), (2, 3, [500, 300, 410], 256, 328), (4, 2, [900, 0], 384, 136), (4, 2, [900, 780], 384, 136),
    (8, 2, [1700, 1500], 512, 520), (2, 4, [3, 1900, 0, 5], 128, 1032), (16, 1, [3100], 256, 264), (3, 2, [700, 640], 1152, 72)])
def test_runs_around_the_limit(W, e, sizes, K, N, dt, qtype):
    run(W, e, split(19, W, e, sizes), K, N, dt, qtype)


@pytest.mark.parametrize("counts", [
    # runs that end inside a half, at its end and one row off it; a source without rows, an expert from one source only
    [128, 256, 127, 129, 384, 1, 255, 640], [0, 0, 1000, 128, 300, 600, 129, 0], [1536, 0, 0, 0, 0, 0, 0, 1], [256, 256, 256, 256, 256, 256, 256, 256]])
def test_runs_of_chosen_lengths(counts):
    run(4, 2, counts, 384, 264, "bf16", "e4m3fn")
