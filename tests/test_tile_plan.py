"""The division of a tiled product over tiles and ranges of k, against an exhaustive
search of its own estimate (no GPU)."""
import math
import random

import pytest

import kronecker_factored_gptq_amd as bk


def sizes(seed, count):
    """Outputs M x N and steps of products of every size, spread over their logarithm."""
    r = random.Random(seed)
    any_of = lambda hi: int(math.exp(r.uniform(0, math.log(hi))))
    return [(any_of(130000), any_of(8192), any_of(2100)) for _ in range(count)]


@pytest.mark.parametrize("pairs,kmajor", [(1, False), (1, True), (3, True), (6, True), (6, False)])
def test_plan_is_the_least_of_its_estimate(pairs, kmajor):
    for M, N, steps in sizes(pairs, 250) + [(16384, 20, 128), (2048, 20, 128), (64, 1, 2004), (1, 1, 1), (1, 1, 0)]:
        tile, splits, us = bk.debug_plan(M, N, steps, pairs, kmajor)
        if tile == 256:
            continue
        for t in (128, 64):
            for n in range(1, 1025):
                other = bk.debug_plan(M, N, steps, pairs, kmajor, True, t, n)[2]
                if other == math.inf and n % 3 == 0:
                    break  # too many, and so is any more
                assert us <= other, (M, N, steps, (tile, splits, us), (t, n, other))
        unsplit = bk.debug_plan(M, N, steps, pairs, kmajor, False)
        assert unsplit[1] == 1 and unsplit[2] >= us


@pytest.mark.parametrize("pairs", [1, 3, 6])
def test_large_tiles_are_not_mostly_empty(pairs):
    """256 x 256 tiles multiply at most a quarter more than 128 x 128 ones, and are taken where
    they fill the chip so."""
    up = lambda x, t: -(-x // t) * t
    for M, N, steps in sizes(7, 400) + [(128256, n, 8) for n in (1, 64, 65, 100, 128, 129, 256, 300, 1000)] + [(20, 131072, 9)]:
        tile = bk.debug_plan(M, N, steps, pairs, True)[0]
        large, small = up(M, 256) * up(N, 256), up(M, 128) * up(N, 128)
        assert (tile == 256) == (large >= 192 * 65536 and large <= 1.25 * small), (M, N, steps)


def test_hook_refuses_what_no_call_takes():
    assert bk.debug_plan(100, 100, 40, tile=96, splits=1)[2] == math.inf
    assert bk.debug_plan(100, 100, 40, tile=64, splits=21)[2] == math.inf  # less than two steps each
    assert bk.debug_plan(4096, 4096, 4000, tile=128, splits=2)[2] == math.inf  # more than the chip holds
    assert bk.debug_plan(100, 100, 40, tile=64, splits=0)[2] == math.inf
    assert bk.debug_plan(0, 100, 40)[2] == math.inf
    # several pairs of planes: ranges that meet the same k
    assert bk.debug_plan(100, 100, 40, 3, tile=64, splits=4)[2] == math.inf
    assert bk.debug_plan(100, 100, 40, 3, tile=64, splits=6)[2] < math.inf
