"""Calls of the paged cache that its documentation allows, at the edges of its rules."""
import ctypes
import os
import subprocess
import sys
from pathlib import Path

import numpy as np
import pytest
import torch

from pool_parity import Both, bf16, ints

pytestmark = pytest.mark.gpu
ROOT = Path(__file__).resolve().parent.parent


def test_lists_are_checked_where_there_is_nothing_to_move():
    """A budget that no sequence can pass, and tokens of length zero."""
    b = Both(pages=8, page=16, heads=2, d=64, sequences=4, max_pages=2)
    b.write([0, 1], 20)
    b.check()
    b.compact([0, 1], 16, 16)
    b.check()
    b.compact([0, 7, 0], 30, 30)  # outside the pool; named before
    b.check(errors=16)
    b.write([1, -1, 2], 0)
    b.check()
    b.write([1, -3, 1], 0)
    b.check(errors=16)
    b.write([1, 2], 0, [1, 0])  # longer than T
    b.check(errors=4)
    b.close()


def test_a_budget_beyond_the_capacity_checks_all_layers():
    import h2o_heavy_hitter_gb300 as h2o
    pool = h2o.h2o_pool_create(3, 8, 16, 2, 64, 4, 2)
    h2o.h2o_pool_compact(pool, -1, ints([0, -1, 3]), 16, 17)
    h2o.h2o_pool_sync_check(pool)
    h2o.h2o_pool_view(pool, 2)["meta"][1, 0] = 33  # longer than its table
    h2o.h2o_pool_compact(pool, -1, ints([0, 1]), 16, 17)
    with pytest.raises(h2o.H2OError, match="word 0x2 "):
        h2o.h2o_pool_sync_check(pool)
    pool.close()
