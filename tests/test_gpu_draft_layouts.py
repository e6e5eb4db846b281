"""Queries and normalisers of drafts in other orders than contiguous ones."""
import numpy as np
import pytest
import torch

from draft_parity import random_paths
from pool_parity import ints
from test_gpu_tree import filled

pytestmark = pytest.mark.gpu


def laid_out(x, how):
    """x's values in another order of strides, or inside something larger."""
    if how == "heads first":
        return x.transpose(1, 2).contiguous().transpose(1, 2)
    if how == "every other entry":
        y = torch.full((2 * x.shape[0], *x.shape[1:]), float("nan"), dtype=x.dtype, device=x.device)
        y[::2] = x
        return y[::2]
    y = torch.full((x.shape[0], x.shape[1] + 3, x.shape[2] + 8, *x.shape[3:]), float("nan"), dtype=x.dtype, device=x.device)
    view = y[:, 2:-1, 8:]
    view.copy_(x)
    return view


@pytest.mark.parametrize("how", ["heads first", "every other entry", "inside a batch"])
@pytest.mark.parametrize("group,kv", [(1, "bf16"), (4, "fp8")])
def test_any_strides_of_queries_and_normalisers(how, group, kv):
    """The same bits as from contiguous tensors."""
    import h2o_heavy_hitter_gb300 as h2o
    lens, nodes, T = [40, 0, 130, 7], [9, 3, 12, 1], 12
    states = []
    for strided in (False, True):
        b, _, q, up = filled(lens, nodes, 2 * group, 16, 2, 64, kv, prefix=50, seed=1)
        parent = torch.tensor(up, dtype=torch.int32, device="cuda")
        q = laid_out(q, how) if strided else q
        assert q.is_contiguous() != strided
        out, lse = torch.full((4, T, 2 * group, 64), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((4, T, 2 * group), 7.0, device="cuda")
        h2o.h2o_pool_attend_tree(b.pool, 0, ints(range(4)), q, 4, ints(nodes), parent, out, lse)
        mine, more = h2o.h2o_pool_attend_tree(b.pool, 0, ints(range(4)), q, 4, ints(nodes), parent)
        live = (torch.arange(T) < torch.tensor(nodes)[:, None]).cuda()
        assert mine.is_contiguous() and torch.equal(mine[live], out[live]) and torch.equal(more[live], lse[live])
        path = torch.tensor(random_paths(np.random.default_rng(4), up, nodes, 5), dtype=torch.int32, device="cuda")
        h2o.h2o_pool_accept(b.pool, 0, ints(range(4)), T, path, ints(nodes), q, laid_out(lse, how) if strided else lse, 4)
        h2o.h2o_pool_sync_check(b.pool)
        states.append([out, lse] + [x.clone() for x in b.view.values()])
        b.close()
    for x, y in zip(*states):
        assert torch.equal(x, y)


def test_a_normaliser_of_another_order_in_a_captured_call():
    import h2o_heavy_hitter_gb300 as h2o
    got = []
    for captured in (False, True):
        b, _, q, _ = filled([60], [6], 4, 16, 2, 64, parent="chain", seed=2)
        _, lse = h2o.h2o_pool_attend_tree(b.pool, 0, ints([0]), q)
        lse, seqs, path = laid_out(lse, "heads first"), ints([0]), ints([0, 1, 2]).view(1, 3)
        call = lambda: h2o.h2o_pool_accept(b.pool, 0, seqs, 6, path, q=q, lse=lse)  # noqa: E731
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                call()
            graph.replay()
        else:
            call()
        h2o.h2o_pool_sync_check(b.pool)
        got.append(b.view["score"].clone())
        b.close()
    assert torch.equal(*got)


def test_what_the_strides_do_not_excuse():
    import h2o_heavy_hitter_gb300 as h2o
    pool = h2o.h2o_pool_create(1, 8, 16, 2, 64, 4, 8)
    q, lse = torch.zeros(1, 4, 3, 64, dtype=torch.bfloat16, device="cuda").transpose(1, 2), torch.zeros(1, 4, 3, device="cuda").transpose(1, 2)
    h2o.h2o_pool_accept(pool, 0, ints([-1]), 3, q=q, lse=lse)
    for args in (dict(q=q[:, :2], lse=lse), dict(q=q, lse=lse[:, :, :2]), dict(q=q.float(), lse=lse), dict(q=q, lse=lse.half()),
                 dict(q=q.cpu(), lse=lse), dict(q=q, lse=lse.cpu()), dict(q=q, lse=None)):
        with pytest.raises((ValueError, TypeError)):
            h2o.h2o_pool_accept(pool, 0, ints([-1]), 3, **args)
    for args in (dict(q=q.float()), dict(q=q.cpu()), dict(q=q, out=torch.zeros_like(q)), dict(q=q, lse=lse)):
        with pytest.raises((ValueError, TypeError)):
            h2o.h2o_pool_attend_tree(pool, 0, ints([-1]), **args)
    h2o.h2o_pool_sync_check(pool)
    pool.close()
