"""What a call refuses of a round must not be taken for drafts by the calls behind it: tokens, scores and
the prefix's scores stay what they would be had the entry been -1. Against the fp64 oracle, and against a
second pool whose lists have -1 in these places."""
import numpy as np
import pytest
import torch

from draft_parity import Drafts, Rotation, random_parents, random_paths
from pool_parity import ints

pytestmark = pytest.mark.gpu

H, GROUP, D, PAGE = 2, 3, 64, 16


def pool_of(lens, spare, max_pages, prefix, kv, sequences=None, seed=3):
    """Sequences 0 .. of `lens` tokens, the prefix behind them, and `spare` free pages."""
    every = list(lens) + [prefix]
    b = Drafts(pages=sum(-(-t // PAGE) for t in every) + spare, page=PAGE, heads=H, d=D,
               sequences=sequences or len(every) + 2, max_pages=max_pages, kv=kv, seed=seed)
    b.write(range(len(every)), max(every), every)
    return b


def one_round(b, seqs, T, lens, prefix, most=4, rotation=None):
    """Append, attend, accept with scores: the rows of q and lse that no call wrote hold 7."""
    up = random_parents(b.rng, len(seqs), T)
    paths = random_paths(b.rng, up, lens, most)
    q64, q = b.append(seqs, T, H * GROUP, rotation, lens=lens, parent=up)
    _, lse = b.tree(seqs, q64, q, prefix, lens, up)
    b.accept(seqs, T, paths, lens, q64, q, lse, prefix)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("cause", ["pages", "longest"])
def test_a_round_with_an_entry_that_got_no_pages(cause, kv):
    """Entry 1's drafts are refused, for want of a free page or as longer than a sequence can be: the round
    passes it over. Then it has room again, and its next round is an ordinary one."""
    lens = [40, 76, 21] if cause == "longest" else [44, 40, 21]
    b = pool_of(lens, 1 if cause == "pages" else 9, 5 if cause == "longest" else 8, 70, kv)
    nodes = [3, 20, 5] if cause == "longest" else [5, 20, 3]  # (of pages: all entries behind the one that got none)
    one_round(b, [0, 1, 2], 20, nodes, 3)
    b.check(errors=8)
    assert b.oracle.meta[1].tolist() == [lens[1], lens[1]] and not b.oracle.refused.any()
    if cause == "pages":
        b.free([0])
    else:
        b.compact([1], 10, 10)
    one_round(b, [1, 2], 9, [9, 9], 3, rotation=Rotation(D, D))
    b.check()
    b.close()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_writes_that_are_refused_leave_no_drafts(kv):
    """Drafts that came by a write, as h2o_pool_accept takes them too."""
    b = pool_of([40, 60, 33], 1, 5, 30, kv)
    b.write([0, 1], 20, [20, 20])  # one page for the first, none for the second
    b.check(errors=8)
    b.accept([0, 1], 20, [[0, 7], [0, 7]], [20, 20])
    b.check()
    assert b.oracle.meta[:2, 0].tolist() == [42, 60]
    b.accept([1], 20, [[0, 7]], [20])  # the last call ended its round: these are its own tokens now
    b.check()
    assert b.oracle.meta[1, 0] == 42
    b.close()


def test_all_layers_remember_for_themselves():
    import h2o_heavy_hitter_gb300 as h2o
    pool = h2o.h2o_pool_create(2, 4, PAGE, H, D, 3, 8)
    x = torch.randn(1, 40, H, D, device="cuda").to(torch.bfloat16)
    up = torch.full((1, 10), -1, dtype=torch.int32, device="cuda")
    for layer, filled in ((0, 30), (1, 9)):  # layer 0 has no page left for the drafts
        h2o.h2o_pool_append(pool, layer, ints([0]), None, x[:, :30], x[:, :30])
        h2o.h2o_pool_append(pool, layer, ints([1]), None, x[:, :filled], x[:, :filled])
        h2o.h2o_pool_append(pool, layer, ints([0]), None, x[:, :10], x[:, :10], parent=up)
    with pytest.raises(h2o.H2OError, match="word 0x8 "):
        h2o.h2o_pool_sync_check(pool)
    before = h2o.h2o_pool_view(pool)["K"][0].clone()
    h2o.h2o_pool_accept(pool, -1, ints([0]), 10, path=ints([9]).view(1, 1))
    h2o.h2o_pool_sync_check(pool)
    v = h2o.h2o_pool_view(pool)
    assert v["meta"][:, 0].tolist() == [[30, 30], [31, 31]] and torch.equal(v["K"][0], before)
    pool.close()


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n,kv", [(2, "bf16"), (2, "fp8"), (40, "bf16")])
def test_a_step_whose_queries_were_not_written(n, kv, accumulate):
    """Single tokens: h2o_pool_attend passes over what h2o_pool_append refused with its queries, and attends
    as before to a sequence whose write, or append without queries, was refused."""
    b = pool_of([32 if i % 2 else 30 for i in range(n)], 0, 4, 40, kv)
    seqs = list(range(n))
    b.append(seqs, 1, H * GROUP)  # the odd ones want a page, and all behind the first are refused
    assert b.oracle.errors == 8 and b.oracle.refused[:n].any()
    b.attend(seqs, H * GROUP, n, accumulate)  # (rows that hold 7 before and after)
    b.check(errors=8)
    b.write(seqs, 1, [0 if i % 2 == 0 else 1 for i in seqs])
    assert b.oracle.errors == 8
    b.attend(seqs, H * GROUP, n, accumulate)  # all of them
    b.check(errors=8)
    b.close()


def test_appends_without_queries_leave_attention_as_it_was():
    b = pool_of([32, 30], 0, 4, 40, "bf16")
    x = torch.randn(1, 1, H, D, device="cuda").to(torch.bfloat16)
    b.h2o.h2o_pool_append(b.pool, 0, ints([0]), None, x, x)
    b.oracle.append([0], 1, None, None, None, queries=False)
    b.attend([0, 1], H * GROUP, 2)
    b.check(errors=8)
    b.close()


@pytest.mark.parametrize("way", ["append", "write", "free", "fork", "nothing to write"])
def test_what_ends_a_refusal(way):
    """Tokens that are served, and an empty sequence that is filled again, are drafts like any others."""
    b = pool_of([48, 40, 25], 0, 5, 16, "bf16", sequences=6)
    b.append([0], 9, H * GROUP, parent=[list(range(-1, 8))])
    b.check(errors=8)
    assert b.oracle.refused[0] == 3
    if way == "fork":
        b.append([4], 20, 2)  # refused: there is no page for an empty sequence either
        b.check(errors=8)
        b.free([1])
        b.fork([2], [4])
        seq = 4
    else:
        seq = 0
        b.free([1])
        if way == "append":
            b.append([0], 9, 2, parent=[list(range(-1, 8))])
        elif way == "write":
            b.write([0], 9)
        elif way == "free":
            b.free([0])
            b.write([0], 12)
        else:
            b.write([0], 9, [0])
    b.check()
    assert b.oracle.refused[seq] == 0
    q64, q = torch.zeros(1, 9, H * GROUP, D).double().numpy(), torch.zeros(1, 9, H * GROUP, D, dtype=torch.bfloat16, device="cuda")
    _, lse = b.tree([seq], q64, q)
    assert np.isfinite(lse.cpu().numpy()).all() and not (lse == 7).any()
    b.accept([seq], 9, [[0, 4]])
    b.check()
    b.close()


def state_bits(view):
    return {name: x.view(torch.int16 if x.dtype is torch.bfloat16 else torch.int32 if x.dtype is torch.float32 else x.dtype)
            for name, x in view.items()}


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_captured_rounds_pass_over_what_runs_out(kv):
    """Rounds in a graph, which the host does not look into, until the pages are gone: bit for bit the state
    of a second pool that gets -1 in the place of every entry that would be refused."""
    import h2o_heavy_hitter_gb300 as h2o
    n, T, rounds = 4, 12, 9
    lens = [44, 30, 15, 60]
    gen = torch.Generator("cuda").manual_seed(7)
    rng = np.random.default_rng(7)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    prompt = randn(2, n + 1, H, 70, D)
    pools = []
    for _ in range(2):
        pool = h2o.h2o_pool_create(1, sum(-(-t // PAGE) for t in lens + [70]) + 4, PAGE, H, D, n + 2, 8, kv)
        h2o.h2o_pool_write(pool, 0, ints(range(n + 1)), prompt[0], prompt[1], lens=ints(lens + [70]))
        pools.append(pool)
    views = [h2o.h2o_pool_view(p, 0) for p in pools]
    r = h2o.h2o_rotary(D)
    made = []
    for _ in range(rounds):
        up = random_parents(rng, n, T)
        nodes = [T] * n
        made.append((randn(n, T, H * (GROUP + 2), D), torch.tensor(up, dtype=torch.int32, device="cuda"), ints(nodes),
                     torch.tensor(random_paths(rng, up, nodes, 6), dtype=torch.int32, device="cuda"), ints(range(n))))
    now = [x.clone() for x in made[0]]
    bufs = [(torch.full((n, T, H * GROUP, D), float("nan"), dtype=torch.bfloat16, device="cuda"),
             torch.zeros(n, T, H * GROUP, D, dtype=torch.bfloat16, device="cuda"),
             torch.full((n, T, H * GROUP), float("nan"), device="cuda")) for _ in range(2)]

    def step(pool, buf, x, up, lens, path, seqs):
        q, out, lse = buf
        h2o.h2o_pool_append(pool, 0, seqs, x[:, :, :H * GROUP], x[:, :, H * GROUP:H * (GROUP + 1)], x[:, :, H * (GROUP + 1):],
                            r, lens, up, out=q)
        h2o.h2o_pool_attend_tree(pool, 0, seqs, q, n, lens, up, out, lse)
        h2o.h2o_pool_accept(pool, 0, seqs, T, path, lens, q, lse, n)

    spare = h2o.h2o_pool_create(1, 30, PAGE, H, D, n + 2, 8, kv)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(spare, [x.clone() for x in bufs[0]], *now)  # what a first call sets up
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(pools[0], bufs[0], *now)
    refused = 0
    for x in made:
        free, have = int((views[1]["ref"] == 0).sum()), views[1]["meta"][:n, 0].tolist()
        listed, out_of = [], False
        for i in range(n):  # as the calls serve their entries: in order, until the pages run out
            need = -(-(have[i] + T) // PAGE) - -(-have[i] // PAGE)
            long = have[i] + T > 8 * PAGE
            out_of |= not long and need > free
            listed.append(-1 if long or out_of else i)
            free -= 0 if long or out_of else need
        refused += listed.count(-1)
        with torch.cuda.stream(side):
            for a, b in zip(now, x):
                a.copy_(b)
            graph.replay()
        step(pools[1], bufs[1], *x[:4], ints(listed))
        torch.cuda.synchronize()
        a, b = (state_bits(v) for v in views)
        for name in a:
            assert torch.equal(a[name], b[name]), name
        assert torch.equal(bufs[0][1], bufs[1][1])
    assert refused >= 3 and not torch.isnan(views[0]["score"]).any()
    with pytest.raises(h2o.H2OError, match="word 0x8 "):
        h2o.h2o_pool_sync_check(pools[0])
    h2o.h2o_pool_sync_check(pools[1])
    for p in (*pools, spare):
        p.close()


def test_an_entry_named_before_is_a_bad_list_alone():
    """Whatever its number of drafts: longer than the sequence, or out of range."""
    b = pool_of([20, 9], 9, 8, 16, "bf16")
    q64, q = torch.zeros(3, 12, H * GROUP, D).double().numpy(), torch.zeros(3, 12, H * GROUP, D, dtype=torch.bfloat16, device="cuda")
    b.tree([1, 0, 1], q64, q, lens=[4, 3, 12])
    b.check(errors=16)
    b.tree([1, 1, 7], q64, q, lens=[4, 13, -1])
    b.check(errors=16)
    b.accept([1, 1, 7], 12, [[0]] * 3, lens=[4, 13, -1])
    b.check(errors=16)
    b.close()
