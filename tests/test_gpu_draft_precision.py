"""How exact drafts are: a tree of one node is a single token's attention, and what keeping it adds to the
scores is what that adds, so both are held to the paged attention's bounds, which are made of the
roundings that its kernels document and a tree's share."""
import numpy as np
import pytest
import torch

import test_gpu_pool_precision as single
from pool_parity import bf16, ints

pytestmark = pytest.mark.gpu


class OneNode:
    """The library, with the attention and the scores of each sequence's last token as a draft's."""

    def __init__(self, h2o):
        self.h2o = h2o

    def __getattr__(self, name):
        return getattr(self.h2o, name)

    def h2o_pool_attend(self, pool, layer, seqs, q, prefix):
        q = q[:, None]
        out, lse = self.h2o.h2o_pool_attend_tree(pool, layer, seqs, q, prefix)
        self.h2o.h2o_pool_accept(pool, layer, seqs, 1, torch.zeros_like(seqs)[:, None], q=q, lse=lse, prefix=prefix)
        return out[:, 0], lse[:, 0]


@pytest.fixture(autouse=True)
def one_node(monkeypatch):
    def filled(*args):
        b = fill(*args)
        b.h2o = OneNode(b.h2o)
        return b

    fill = single.filled
    monkeypatch.setattr(single, "filled", filled)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("path", single.PATHS)
def test_values_that_cancel(path, d, kv):
    single.test_values_that_cancel(*path, d, kv)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("path", single.PATHS)
def test_outputs_and_scores_of_ordinary_values(path, d, kv):
    single.test_outputs_and_scores_of_ordinary_values(*path, d, kv)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("exponent", [-118, -100, 100])
@pytest.mark.parametrize("path", [single.PATHS[1], single.PATHS[4], single.PATHS[6], single.PATHS[8], single.PATHS[10]])
def test_queries_and_keys_of_opposite_magnitudes(path, exponent, kv):
    single.test_queries_and_keys_of_opposite_magnitudes(*path, exponent, kv)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("exponent", [-119, 111, 115, 118, 119])
@pytest.mark.parametrize("d", [64, 128])
def test_queries_beyond_what_a_sum_of_codes_holds(d, exponent, kv):
    """(And the other way round.) Keys of nearly 2^-119, the least that an E4M3 pool stores, against queries of that order: a sum of d codes up to
    448 times the query leaves fp32 where the logit does not."""
    rng = np.random.default_rng(d)
    sign = lambda *s: np.where(rng.random(s) < 0.5, -1.0, 1.0) * (1 + rng.random(s))  # noqa: E731
    K = lambda n, T: sign(n, 2, T, d) * 2.0 ** -exponent  # noqa: E731
    V = lambda n, T: rng.standard_normal((n, 2, T, d))  # noqa: E731
    b = single.filled(3, 2, 200, 90, d, kv, K, V)
    q64 = sign(3, 6, d) * 2.0 ** exponent
    single.attend_and_compare(b, 3, 2, 3, 3, *bf16(q64))
    b.close()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("path", single.PATHS)
def test_an_infinite_value_gives_an_infinite_output(path, d):
    """Among the drafts too: the last token's."""
    single.test_an_infinite_value_gives_an_infinite_output(*path, d)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("batch,heads,group,prefix,own", [single.PATHS[0], single.PATHS[5]])
def test_the_same_of_single_tokens(batch, heads, group, prefix, own, kv):
    """What `attend_and_compare` was told here is what a tree does: both ways, out and lse agree to a rounding."""
    rng = np.random.default_rng(own)
    some = lambda n, T: rng.standard_normal((n, heads, T, 64))  # noqa: E731
    b = single.filled(batch, heads, prefix, own, 64, kv, some, some)
    _, q = bf16(rng.standard_normal((batch, heads * group, 64)))
    at = batch if prefix else -1
    a, la = b.h2o.h2o.h2o_pool_attend(b.pool, 0, ints(range(batch)), q, prefix=at, accumulate=False)
    t, lt = b.h2o.h2o_pool_attend(b.pool, 0, ints(range(batch)), q, prefix=at)
    assert torch.allclose(la, lt, atol=2.0 ** -18, rtol=0)
    assert torch.allclose(a.float(), t.float(), atol=2.0 ** -9, rtol=2.0 ** -7)
    b.close()
