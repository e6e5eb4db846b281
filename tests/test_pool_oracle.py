"""The paged cache's oracle on calls where the order of its own steps could show."""
import numpy as np
import pytest

from oracle import kv_pool


@pytest.mark.parametrize("share", [True, False])
def test_forks_read_their_sources_as_they_were_before_the_call(share):
    p = kv_pool.Pool(12, 16, 2, 8, 5, 4)
    x = np.random.default_rng(0).standard_normal((2, 1, 2, 40, 8))
    p.write([0], x[0], x[1])
    p.fork([0, 1, 2, 0], [1, 2, 3, 4], share)
    assert p.meta.tolist() == [[40, 40], [40, 40], [0, 0], [0, 0], [40, 40]]
    assert p.errors == 0 and (p.table[[2, 3]] == -1).all()
    held = np.bincount(p.table[p.table >= 0], minlength=12)
    assert np.array_equal(held, p.ref)
