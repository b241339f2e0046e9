"""GPU checks of the 8-bit cache's tree attention where queries and keys are far from one, in
opposite directions: the scores are ordinary."""
import numpy as np
import pytest
import torch

from tests.test_gpu_kv8_bounds import D, _bf16, _cache, _check, _trees

pytestmark = pytest.mark.gpu


def _times(x, power):
    return (x.double() * 2.0 ** power).bfloat16()


@pytest.mark.parametrize("n,Hq", [(1, 4), (6, 4), (50, 4)])
@pytest.mark.parametrize("power", [-110, -60, -45, -36, 40, 55])
def test_queries_and_keys_of_opposite_size(power, n, Hq):
    L = [333]
    q, kt, vt = _times(_bf16((1, n, Hq, D), 41), power), _times(_bf16((1, n, 1, D), 42), -power), _bf16((1, n, 1, D), 43)
    codes, scales = _cache(1, 1, L, 352, 44)
    _check(q, (codes, scales * 2.0 ** -power), _cache(1, 1, L, 352, 45), kt, vt, L, _trees(1, n, 46))


@pytest.mark.parametrize("power", [45, 70, 110])
def test_large_queries_and_small_keys_of_the_tree(power):
    n, L = 30, [0]
    q, kt, vt = _times(_bf16((1, n, 4, D), 51), power), _times(_bf16((1, n, 2, D), 52), -power), _bf16((1, n, 2, D), 53)
    _check(q, _cache(1, 2, L, 32, 54), _cache(1, 2, L, 32, 55), kt, vt, L, _trees(1, n, 56))


@pytest.mark.parametrize("qp,kp,scale", [(30, 30, 2.0 ** -64), (60, 60, 2.0 ** -124), (-50, -50, 2.0 ** 96), (-60, -40, 2.0 ** 97)])
def test_factor_of_the_softmax_far_from_one(qp, kp, scale):
    n, L = 5, [150]
    q, kt, vt = _times(_bf16((1, n, 2, D), 61), qp), _times(_bf16((1, n, 1, D), 62), kp), _bf16((1, n, 1, D), 63)
    codes, scales = _cache(1, 1, L, 160, 64)
    _check(q, (codes, scales * 2.0 ** kp), _cache(1, 1, L, 160, 65), kt, vt, L, _trees(1, n, 66), scale=scale)
