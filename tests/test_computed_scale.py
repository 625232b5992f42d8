"""The scale of computed values takes its quotient by one correction step down
to 2^-126: exact there for every amax, by the emulation that the division's
tests use."""
import multiprocessing as mp
import os

import numpy as np

from tests.test_scale_division import _scale_binade, reciprocal_division

F32 = np.float32


def test_one_step_on_every_amax_down_to_the_floor():
    # amax / 448 >= 2^-126 from 2^-117.2 on: the binades from 2^-117 up whole, those below 2^-100 that the given tensors' quantiser leaves out
    workers = max(1, min(8, os.cpu_count() or 1))
    with mp.get_context("spawn").Pool(workers) as pool:
        assert sum(pool.map(_scale_binade, range(-117, -100))) == 0


def test_around_the_floor_and_where_the_quotient_is_0():
    """Next to 448 * 2^-126 the floor hides what a step could lose; amax / 448 rounds to 0 up to 448 * 2^-150."""
    at = F32(448.0 * 2.0 ** -126).view(np.uint32)
    a = np.arange(int(at) - (1 << 20), int(at) + (1 << 20), dtype=np.uint32).view(F32)
    q, _ = reciprocal_division(a, np.full_like(a, F32(448.0)), 1)
    assert np.array_equal(np.maximum(q, F32(2.0 ** -126)), np.maximum(a / F32(448.0), F32(2.0 ** -126)))
    a = np.arange(0, 1 << 12, dtype=np.uint32).view(F32)
    assert np.array_equal(a / F32(448.0) == 0, a <= F32(float.fromhex("0x1.cp-142")))
