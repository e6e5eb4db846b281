"""The paged cache against the oracle's: whole states after every call, on the sizes and lists
where page arithmetic, masks and the policy can go wrong."""
import numpy as np
import pytest
import torch

from pool_parity import Both, bf16, ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("page,d", [(16, 64), (32, 128), (64, 64), (128, 128)])
def test_write_lengths_around_pages(page, d, kv):
    b = Both(pages=24, page=page, heads=3, d=d, sequences=6, max_pages=4, kv=kv)
    lens = [0, 1, page - 1, page, page + 1, 2 * page]
    b.write(range(6), 2 * page, lens)
    b.check()
    b.write(range(6), 1)  # a step's token on every remainder
    b.check()
    b.write([3, -1, 0], page, [page, 5, 2], score=False)
    b.check()
    b.close()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_write_zero_tiny_and_large_values(kv):
    b = Both(pages=4, page=16, heads=1, d=64, sequences=1, max_pages=2, kv=kv)
    x = b.tokens(1, 6)
    x[0, 0, 0] = 0
    x[0, 0, 1] *= 2.0 ** -125
    x[0, 0, 2] *= 2.0 ** 100
    x[0, 0, 3, 1:] = 0
    b.write([0], 6, K=x, V=x[..., ::-1])
    b.check()
    b.close()


def test_a_full_pool_refuses_from_the_first_entry_that_does_not_fit():
    b = Both(pages=5, page=16, heads=2, d=64, sequences=5, max_pages=4)
    b.write([0, 1, 2, 3], 40, [20, 40, 1, 0])  # 2 + 3 pages, then none for 2; 3 needs none
    b.check(errors=8)
    b.write([0], 12)  # fills its last page
    b.check()
    b.write([0, 1], 40, [33, 9])  # beyond max_pages; no page
    b.check(errors=8)
    b.fork([1], [2])  # its last page is partial: a fresh one is needed
    b.check(errors=8)
    b.free([0])
    b.fork([1, 1], [2, 3])
    b.check()
    b.close()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("share", [True, False])
@pytest.mark.parametrize("page,d", [(16, 128), (128, 64)])
def test_fork_copy_and_free(share, page, d, kv):
    b = Both(pages=40, page=page, heads=3, d=d, sequences=9, max_pages=5, kv=kv)
    b.write([0, 1, 2], 4 * page, [3 * page + 1, 2 * page, 0])
    b.fork([0, 1, 0, 2, -1], [4, 5, 6, 7, 8], share)
    b.check()
    b.write([4, 0, 5], 3, [1, 3, 2])  # each goes on alone
    b.check()
    b.free([0, 1, 2])  # what the forks share stays
    b.check()
    b.fork([4, 6], [0, 1], share)
    b.free([4, 5, 6, 0, 1, 7, 3])
    b.check()
    assert int(b.view["ref"].sum()) == 0
    b.close()


def test_bad_lists_are_reported_and_skipped():
    b = Both(pages=12, page=16, heads=1, d=64, sequences=4, max_pages=4)
    b.write([0, 0, 1, 4, -2], 5)  # twice, outside, outside
    b.check(errors=16)
    b.write([2], 4, [9])  # longer than T: clamped
    b.check(errors=4)
    b.fork([0, 9, 1, 0], [1, 3, 3, 3])  # in use; no such source; named before
    b.check(errors=16)
    b.free([1, 1, 7])
    b.check(errors=16)
    b.compact([0, 0], 1, 1)
    b.check(errors=16)
    b.attend([0, 0, 5, 2, 3], 1, prefix=2)
    b.check(errors=16)
    b.close()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("page,d,h,r", [(16, 64, 5, 0), (16, 128, 0, 7), (32, 64, 16, 17), (64, 128, 1, 1),
                                        (128, 64, 100, 40)])
def test_compact_keeps_heavy_hitters_and_recent(page, d, h, r, kv):
    b = Both(pages=60, page=page, heads=3, d=d, sequences=7, max_pages=8, kv=kv, seed=h)
    k = h + r
    b.write(range(6), 8 * page, [8 * page, k, k + 1, 0, k - 1, 3 * page + 5])
    b.fork([0], [6])  # shares what the compaction moves
    b.compact([6, 1, 2, 3, -1, 5, 4], h, r)
    b.check()
    b.compact([6, 5], h, r)  # already within the budget
    b.check()
    b.write([6, 2, 0], 2, [2, 1, 0])
    b.attend([0, 6, 2, 3, 4], 6)
    b.compact([0, 6], h, r)
    b.check()
    b.close()


def test_compact_orders_equal_negative_infinite_and_nan_scores():
    b = Both(pages=12, page=16, heads=1, d=64, sequences=2, max_pages=4)
    b.write([0], 50)
    s = np.zeros(64, np.float32)
    s[:50] = np.resize([0.0, -0.0, -1.5, np.inf, 2.0, 2.0, -np.inf, 1e-40, 3e38], 50)
    s[[7, 30]] = np.nan
    b.view["score"][0, 0] = torch.from_numpy(s).cuda()
    b.oracle.score[0, 0] = s
    # the oracle's key of NaN and infinity: infinity below NaN, the zeros equal
    b.oracle.score[0, 0][np.isposinf(s)] = 1e300
    b.oracle.score[0, 0][np.isneginf(s)] = -1e300
    b.compact([0], 20, 3)
    got, want = (np.asarray(x)[0] for x in (b.view["pos"].cpu(), b.oracle.pos))
    assert np.array_equal(got, want)
    b.close()


@pytest.mark.parametrize("shortfall", [0, 1])
def test_compact_needs_fresh_pages(shortfall):
    b = Both(pages=6 - shortfall, page=16, heads=2, d=64, sequences=2, max_pages=4)
    b.write([0, 1], 33, [33, 17] if shortfall else [33, 16])
    b.compact([1, 0], 8, 9)
    b.check(errors=8 if shortfall else 0)
    b.close()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("page,d,heads,group", [(16, 64, 1, 1), (32, 128, 2, 3), (64, 64, 3, 8), (128, 128, 1, 32),
                                                (16, 128, 4, 5)])
def test_attend_lengths(page, d, heads, group, kv):
    cap = 640 // page
    b = Both(pages=4 * cap + 30, page=page, heads=heads, d=d, sequences=9, max_pages=cap, kv=kv, seed=page + d)
    lens = [1, 0, 127, 128, 129, 300, page, 640]
    b.write(range(8), 640, lens)
    seqs = [0, 1, 2, -1, 3, 4, 5, 6, 7]
    b.attend(seqs, heads * group)  # no prefix: sequence 1 has no token at all
    b.check()
    b.attend([7, 5, 8], heads * group, prefix=1)  # an empty prefix, an empty row
    b.check()
    b.attend([0, 1, 2, 8, 3, -1, 6], heads * group, prefix=7)
    b.check()
    b.attend([6], heads * group, prefix=4, accumulate=False)
    b.check()
    b.close()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("batch,heads,group,prefix", [(3, 2, 1, 257), (70, 1, 2, 130), (40, 2, 7, 300), (130, 1, 3, 511)])
def test_attend_many_rows_on_a_prefix(batch, heads, group, prefix, kv):
    b = Both(pages=batch * 2 + 20, page=32, heads=heads, d=64, sequences=batch + 1, max_pages=16, kv=kv, seed=batch)
    lens = [int(x) for x in b.rng.integers(0, 40, batch)] + [prefix]
    b.write(range(batch + 1), prefix, lens)
    b.attend(range(batch), heads * group, prefix=batch)
    b.check()
    b.attend(range(batch - 1, -1, -1), heads * group, prefix=batch)
    b.check()
    b.close()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("heads,group,d,page,batch,longest,prefix", [
    (24, 1, 64, 16, 6, 1500, 2200),   # many tiles per SM, units that begin and end inside a share
    (24, 2, 128, 64, 9, 700, 3000),
    (16, 5, 64, 32, 60, 130, 1700),   # three row tiles a head: a block of two and one of one
    (20, 8, 128, 128, 17, 260, 2500), # two row tiles, the second nearly empty
])
def test_attend_many_tiles(heads, group, d, page, batch, longest, prefix, kv):
    lens = [longest - (i * 331) % longest for i in range(batch)] + [prefix]
    pages = sum(-(-n // page) for n in lens) + 1
    b = Both(pages, page, heads, d, batch + 1, -(-max(lens) // page), kv, seed=batch)
    for i, n in enumerate(lens):
        b.write([i], n)
    b.check()
    b.attend(range(batch), heads * group, prefix=batch)
    b.check()
    b.attend(range(batch), heads * group, prefix=batch)
    b.attend([batch] + list(range(0, batch, 2)), heads * group)  # the prefix as a sequence
    b.check()
    b.close()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("heads,group,batch,prefix", [(700, 1, 36, 100), (330, 3, 47, 70)])
def test_attend_many_heads_to_a_share(heads, group, batch, prefix, kv):
    """More heads than SMs: a share of the prefix's tiles passes through several heads."""
    lens = [(7 * i) % 23 for i in range(batch)] + [prefix]
    b = Both(batch + 8, 32, heads, 64, batch + 1, 4, kv, seed=heads)
    b.write(range(batch + 1), prefix, lens)
    for _ in range(2):
        b.attend(range(batch), heads * group, prefix=batch)
        b.check()
    b.close()


def test_attend_ignores_what_lies_behind_a_sequence():
    """NaN and infinities in the slots behind the last token, of the prefix too."""
    b = Both(pages=12, page=32, heads=2, d=64, sequences=3, max_pages=4)
    b.write([0, 1], 50, [50, 33])
    for name in "KV":
        for seq, n in ((0, 50), (1, 33)):
            p = int(b.oracle.table[seq, n // 32])
            b.view[name][p, :, n % 32:] = float("nan") if name == "K" else float("inf")
    free = [p for p in range(12) if b.oracle.ref[p] == 0]
    b.view["V"][free] = float("nan")
    b.attend([1], 2, prefix=0)
    b.attend([0, 1], 4)
    b.close()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("what", ["key", "value", "query"])
def test_a_nan_reaches_the_rows_that_attend_to_it_and_no_others(kv, what):
    heads, d = 2, 64
    b = Both(pages=30, page=16, heads=heads, d=d, sequences=3, max_pages=12, kv=kv)
    K, V = b.tokens(3, 150), b.tokens(3, 150)
    q = b.queries(2, 4)
    if what == "query":
        q[0, 1, 5] = np.nan
    else:
        (K if what == "key" else V)[0, 1, 70, 3] = np.nan if kv == "bf16" else np.inf
    b.write([0, 1, 2], 150, [150, 140, 20], K=K, V=V)
    b.check()
    _, qt = bf16(q)
    out, lse = b.h2o.h2o_pool_attend(b.pool, 0, ints([0, 1]), qt, prefix=2)
    nan = out.isnan().cpu().numpy()  # [2, 4, d]
    if what == "query":
        assert nan[0, 1].all() and not nan[0, [0, 2, 3]].any() and not nan[1].any()
    else:  # key head 1 of sequence 0 serves the query heads 2 and 3
        assert not nan[1].any() and not nan[0, :2].any()
        assert nan[0, 2:].all() if what == "key" or kv == "fp8" else nan[0, 2:, 3].all()
    b.close()


def test_every_e4m3_value_is_attended_to_exactly():
    """A token that alone has weight returns its stored value: all 254 codes, both signs, as
    values; as keys, a logit of each."""
    d = 128
    b = Both(pages=40, page=16, heads=1, d=d, sequences=1, max_pages=40, kv="fp8")
    b.write([0], 600)
    from oracle import kv_fp8
    codes = np.array([c for c in range(256) if c & 0x7f != 0x7f], np.uint8)
    v = np.resize(codes, (2, d))
    v[1] = codes[-d:]
    slot = [(int(b.oracle.table[0, t // 16]), t % 16) for t in (300, 301)]
    for (p, o), row in zip(slot, v):
        b.view["V"][p, 0, o] = torch.from_numpy(row).cuda()
        b.view["vscale"][p, 0, o] = 0.5
        b.view["K"][p, 0, o] = 0
        b.view["kscale"][p, 0, o] = 1.0
    for (p, o), row in zip(slot, v):
        b.view["K"][p, 0, o, 0] = 0x7e  # 448 * 4 / sqrt(128): above every other logit by 100
        q = np.zeros((1, 1, d))
        q[..., 0] = 4.0
        out, lse = b.h2o.h2o_pool_attend(b.pool, 0, ints([0]), bf16(q)[1], accumulate=False)
        b.view["K"][p, 0, o, 0] = 0
        want = torch.from_numpy(kv_fp8.e4m3_decode(row) * 0.5).to(torch.bfloat16)
        assert torch.equal(out[0, 0].cpu(), want)
    # one code a key, the query a unit vector of each value: s = code / sqrt(d)
    b.view["K"].zero_()
    b.view["kscale"].fill_(1.0)
    for i, c in enumerate(codes):
        b.view["K"][int(b.oracle.table[0, i // 16]), 0, i % 16, 5] = int(c)
    b.view["score"].zero_()
    q = np.zeros((1, 1, d))
    q[..., 5] = 0.109375  # 7 / 64: two codes hold it
    out, lse = b.h2o.h2o_pool_attend(b.pool, 0, ints([0]), bf16(q)[1])
    x = np.zeros(600)
    x[:len(codes)] = kv_fp8.e4m3_decode(codes) * 0.109375 / np.sqrt(d)
    p = np.exp(x)
    np.testing.assert_allclose(b.view["score"][0, 0, :600].double().cpu().numpy(), p / p.sum(), rtol=1e-5)
    b.close()


@pytest.mark.parametrize("magnitude", [2.0 ** -130, 2.0 ** -40, 1.0, 2.0 ** 60])
def test_queries_of_any_magnitude_on_codes(magnitude):
    """An E4M3 pool splits a query into two codes a value: no magnitude loses bits."""
    d = 64
    b = Both(pages=64, page=16, heads=2, d=d, sequences=41, max_pages=40, kv="fp8")
    b.write([40], 333, K=b.tokens(1, 333) / magnitude if magnitude > 1 else None)
    for n in (3, 40):  # few and many rows
        q64, q = bf16(b.queries(n, 2) * magnitude * np.exp2(-np.arange(d) / 4))
        b.write(range(n), 1, score=False, K=b.tokens(n, 1) / max(1.0, magnitude))
        out, lse = b.h2o.h2o_pool_attend(b.pool, 0, ints(range(n)), q, prefix=40)
        want, want_lse = b.oracle.attend(range(n), q64, 40)
        # logits up to 32; a value is off by 2^-17 of the row's largest at most
        assert np.abs(lse.double().cpu().numpy() - want_lse).max() <= 2e-4
        assert np.abs(out.double().cpu().numpy() - want).max() <= 2.0 ** -7 * np.abs(b.oracle.V).max()
        b.check()
        b.free(range(n))
    b.close()


def test_attend_large_and_equal_logits():
    b = Both(pages=24, page=16, heads=1, d=64, sequences=2, max_pages=20)
    x = np.zeros((1, 1, 300, 64))
    x[..., 0] = 60.0
    x[0, 0, 150, 1] = 16.0
    b.write([0], 300, K=x)
    q = np.zeros((1, 1, 64))
    q[..., 0], q[..., 1] = 100.0, 1.0
    _, qt = bf16(q)
    out, lse = b.h2o.h2o_pool_attend(b.pool, 0, ints([0]), qt)
    p = np.ones(300)
    p[150] = np.exp(2.0)
    p /= p.sum()
    want = p @ b.oracle.V[b.oracle.table[0, np.arange(300) // 16], 0, np.arange(300) % 16]
    assert np.abs(out[0, 0].double().cpu().numpy() - want).max() <= 2.0 ** -7 * np.abs(b.oracle.V).max()
    # the logit 750 + ln 300..: fp32 holds it to 2^-15
    assert abs(float(lse[0, 0]) - (750 + np.log(299 + np.exp(2.0)))) <= 2e-4
    b.close()


def test_attend_repeats_bit_for_bit():
    b = Both(pages=80, page=32, heads=2, d=128, sequences=20, max_pages=30)
    b.write(range(17), 900, [int(x) for x in b.rng.integers(0, 90, 16)] + [900])
    _, q = bf16(b.queries(16, 8))
    before, runs = b.view["score"].clone(), []
    for _ in range(10):
        b.view["score"].copy_(before)
        out, lse = b.h2o.h2o_pool_attend(b.pool, 0, ints(range(16)), q, prefix=16)
        runs.append((out.clone(), lse.clone(), b.view["score"].clone()))
    for r in runs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(r, runs[0]))
    b.close()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_a_run_as_a_server_makes_it(kv):
    """Prompt attention and its scores, a shared prefix, sequences that come, fork, decode, are
    compacted and go, against the oracle after every step."""
    import h2o_heavy_hitter_gb300 as h2o
    heads, d, page = 2, 64, 16
    b = Both(pages=80, page=page, heads=heads, d=d, sequences=8, max_pages=12, kv=kv, layers=3, layer=1)
    T = 100
    k64, k = bf16(b.tokens(heads, T)[:, 0])
    _, q = bf16(b.queries(heads, T))
    v64, v = bf16(b.rng.standard_normal((heads, T, d)))
    _, col = h2o.h2o_prefill_attention(q, k, v)
    h2o.h2o_pool_write(b.pool, 1, ints([7]), k[None], v[None], score=col[None])
    b.oracle.write([7], k64[None], v64[None], score=col.double().cpu().numpy()[None])
    b.check()
    b.write([0, 1], 30, [30, 17])
    b.fork([0, 0, 1], [2, 3, 4])
    live = [0, 1, 2, 3, 4, -1]
    for step in range(12):
        b.write(live, 1, score=False)
        b.attend(live, 2 * heads, prefix=7)
        b.check()
        if step == 3:
            b.compact([7], 20, 12)  # the prefix, for all
            b.free([3])
            b.fork([2], [5])
            live = [5, 0, 1, -1, 2, 4]
        if step == 7:
            b.compact(live, 8, 8)
        b.check()
    for other in (0, 2):  # the other layers were never touched
        w = h2o.h2o_pool_view(b.pool, other)
        assert int(w["ref"].sum()) == 0 and int(w["meta"].abs().sum()) == 0 and int(w["table"].max()) == -1
    b.free(range(8))
    b.check()
    b.close()


def test_all_layers_at_once():
    import h2o_heavy_hitter_gb300 as h2o
    heads, d, page, L = 2, 64, 16, 3
    pools = [Both(30, page, heads, d, 6, 6, layers=L, layer=layer, seed=layer) for layer in range(L)]
    pool = pools[0].pool
    for b in pools[1:]:  # one pool, an oracle for each of its layers
        b.pool.close()
        b.pool, b.view = pool, h2o.h2o_pool_view(pool, b.layer)
    for layer, b in enumerate(pools):
        b.write([0, 1], 70, [70 - layer, 20 + layer])
    h2o.h2o_pool_fork(pool, -1, ints([0, 1]), ints([2, 3]))
    h2o.h2o_pool_copy(pool, -1, ints([0]), ints([4]))
    h2o.h2o_pool_compact(pool, -1, ints([2, 1]), 9, 8)
    h2o.h2o_pool_free(pool, -1, ints([0]))
    h2o.h2o_pool_sync_check(pool)
    for b in pools:
        b.oracle.fork([0, 1], [2, 3])
        b.oracle.fork([0], [4], share=False)
        b.oracle.compact([2, 1], 9, 8)
        b.oracle.free([0])
        b.check()
    whole = h2o.h2o_pool_view(pool)
    assert whole["K"].shape == (L, 30, heads, page, d)
    assert torch.equal(whole["table"][2], pools[2].view["table"])
    pool.close()


def test_calls_on_another_stream_and_in_a_graph():
    import h2o_heavy_hitter_gb300 as h2o
    b = Both(pages=60, page=16, heads=2, d=64, sequences=4, max_pages=16, seed=3)
    b.write([0, 1, 3], 60, [60, 21, 50])
    k64, k = bf16(b.tokens(2, 1))
    v64, v = bf16(b.tokens(2, 1))
    q64, q = bf16(b.queries(2, 4))
    seqs, sink = ints([0, 1]), ints([2])
    source = ints([0])

    def step():
        h2o.h2o_pool_write(b.pool, 0, seqs, k, v)
        out = h2o.h2o_pool_attend(b.pool, 0, seqs, q, prefix=3)
        h2o.h2o_pool_free(b.pool, 0, sink)
        h2o.h2o_pool_fork(b.pool, 0, source, sink)
        h2o.h2o_pool_compact(b.pool, 0, sink, 9, 9)
        return out

    def oracle_step():
        b.oracle.write([0, 1], k64, v64)
        want = b.oracle.attend([0, 1], q64, 3)
        b.oracle.free([2])
        b.oracle.fork([0], [2])
        b.oracle.compact([2], 9, 9)
        return want

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    oracle_step()
    b.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step()
    for _ in range(5):
        graph.replay()
        want, want_lse = oracle_step()
        assert np.abs(lse.double().cpu().numpy() - want_lse).max() <= 1e-4
    b.check()
    b.close()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("batch,heads,group", [(6, 32, 2), (64, 16, 1), (120, 8, 2), (70, 8, 5)])
def test_calls_back_to_back_equal_synchronised_ones(batch, heads, group, kv):
    """Launches that begin while the one before drains read nothing too early and overwrite nothing
    too early: the same calls with a synchronisation behind each give the same bits."""
    import h2o_heavy_hitter_gb300 as h2o
    rng = torch.Generator(device="cuda").manual_seed(batch)
    rand = lambda *shape: torch.randn(*shape, generator=rng, device="cuda").to(torch.bfloat16)
    prefix, steps = 2500, 6
    K, V = rand(batch + 1, heads, prefix, 128), rand(batch + 1, heads, prefix, 128)
    lens = ints([(37 * i) % 300 for i in range(batch)] + [prefix])
    k, v = rand(steps, batch, heads, 1, 128), rand(steps, batch, heads, 1, 128)
    q = rand(steps, 2, batch, heads * group, 128)
    everyone, seqs, one, sink = ints(range(batch + 1)), ints(range(batch)), ints([batch]), ints([batch + 1])

    def run(wait):
        pool = h2o.h2o_pool_create(1, 14 * batch + 100, 32, heads, 128, batch + 2, 80, kv)
        outs = torch.zeros(steps, 2, batch, heads * group, 128, dtype=torch.bfloat16, device="cuda")
        lses = torch.zeros(steps, 2, batch, heads * group, device="cuda")
        calls = [lambda: h2o.h2o_pool_write(pool, 0, everyone, K, V, lens=lens)]
        for t in range(steps):
            attend = lambda t, i: h2o.h2o_pool_attend(pool, 0, seqs, q[t, i], prefix=batch if i == 0 or t % 2 else -1,
                                                      out=outs[t, i], lse=lses[t, i], accumulate=t != 3)
            calls += [lambda t=t: h2o.h2o_pool_write(pool, 0, seqs, k[t], v[t]),
                      lambda t=t: attend(t, 0), lambda t=t: attend(t, 1),
                      lambda: h2o.h2o_pool_free(pool, 0, sink),
                      lambda: h2o.h2o_pool_fork(pool, 0, one, sink),
                      lambda: h2o.h2o_pool_compact(pool, 0, sink, 100, 60),
                      lambda: h2o.h2o_pool_compact(pool, 0, seqs, 150, 50)]
        torch.cuda.synchronize()
        for call in calls:
            call()
            if wait:
                torch.cuda.synchronize()
        h2o.h2o_pool_sync_check(pool)
        state = {name: x.clone() for name, x in h2o.h2o_pool_view(pool, 0).items()}
        torch.cuda.synchronize()
        pool.close()
        return state | {"out": outs, "lse": lses}

    want = run(True)
    for _ in range(3):
        got = run(False)
        for name, x in want.items():
            assert torch.equal(x.view(torch.uint8), got[name].view(torch.uint8)), name


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("batch", [3, 40, 90])  # narrow rows, one row tile of the prefix, three
def test_a_captured_step_behind_copies_and_joined_streams(kv, batch):
    """Every call of a captured graph behind a copy, a fill and a join of two streams."""
    import h2o_heavy_hitter_gb300 as h2o
    heads, group = 3, 3
    b = Both(pages=5 * batch + 30, page=16, heads=heads, d=128, sequences=batch + 2, max_pages=20, kv=kv, seed=batch)
    b.write(range(batch + 1), 290, [(13 * i) % 37 for i in range(batch)] + [290])
    k64, k = bf16(b.tokens(batch, 1))
    v64, v = bf16(b.tokens(batch, 1))
    q64, q = bf16(b.queries(batch, heads * group))
    k_in, v_in, q_in = torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(q)
    seqs, some, sink = ints(range(batch)), ints([batch]), ints([batch + 1])
    out = torch.zeros_like(q)
    lse = torch.zeros(q.shape[:2], device="cuda")
    side = torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        k_in.copy_(k)
        v_in.copy_(v)
        h2o.h2o_pool_write(b.pool, 0, seqs, k_in, v_in)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            q_in.copy_(q)
            lse.fill_(3.0)
        out.zero_()
        main.wait_stream(side)
        h2o.h2o_pool_attend(b.pool, 0, seqs, q_in, prefix=batch, out=out, lse=lse)
        h2o.h2o_pool_free(b.pool, 0, sink)
        h2o.h2o_pool_fork(b.pool, 0, some, sink)
        k_in.zero_()
        v_in.zero_()
        h2o.h2o_pool_compact(b.pool, 0, sink, 30, 9)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            q_in.zero_()
        main.wait_stream(side)

    def oracle_step():
        b.oracle.write(range(batch), k64, v64)
        want = b.oracle.attend(range(batch), q64, batch)
        b.oracle.free([batch + 1])
        b.oracle.fork([batch], [batch + 1])
        b.oracle.compact([batch + 1], 30, 9)
        return want

    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        step()
    torch.cuda.current_stream().wait_stream(warm)
    oracle_step()
    b.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        graph.replay()
        want, want_lse = oracle_step()
        size = np.abs(b.oracle.V).max()  # the tolerances of Both.attend
        assert np.all(np.abs(out.double().cpu().numpy() - want) <= 2.0 ** -8 * (size + np.abs(want)) + 1e-3 * size)
        assert np.all(np.abs(lse.double().cpu().numpy() - want_lse) <= 1e-4)
    b.check()
    b.close()


def test_two_graphs_and_eager_calls_on_streams_of_their_own():
    """Layers are independent: graphs of two layers and eager calls on a third run at once and
    leave what they leave one after the other."""
    import h2o_heavy_hitter_gb300 as h2o
    heads, d, page, L = 4, 64, 16, 3
    gen = torch.Generator("cuda").manual_seed(5)
    pool = h2o.h2o_pool_create(L, 120, page, heads, d, 12, 30)
    k = torch.randn(2, 12, heads, 400, d, generator=gen, device="cuda").to(torch.bfloat16)
    q = torch.randn(L, 11, 2 * heads, d, generator=gen, device="cuda").to(torch.bfloat16)
    one = torch.randn(11, heads, 1, d, generator=gen, device="cuda").to(torch.bfloat16)
    lens, all_, batch = ints([50 + 7 * i for i in range(11)] + [400]), ints(range(12)), ints(range(11))
    for layer in range(L):
        h2o.h2o_pool_write(pool, layer, all_, k[0], k[1], lens)
    view = h2o.h2o_pool_view(pool)
    start = {n: x.clone() for n, x in view.items()}

    def step(layer):
        h2o.h2o_pool_write(pool, layer, batch, one, one)
        return h2o.h2o_pool_attend(pool, layer, batch, q[layer], prefix=11)

    def reset():
        for n, x in start.items():
            view[n].copy_(x)

    want = []
    for layer in range(L):
        for _ in range(6):
            out = step(layer)
        want.append([x.clone() for x in out])
    scores = view["score"].clone()
    reset()
    streams = [torch.cuda.Stream() for _ in range(L)]
    graphs, outs = [], []
    for layer in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[layer]):
            outs.append(step(layer))
    reset()
    torch.cuda.synchronize()
    for _ in range(6):
        for layer in range(2):
            with torch.cuda.stream(streams[layer]):
                graphs[layer].replay()
        with torch.cuda.stream(streams[2]):
            eager = step(2)
    torch.cuda.synchronize()
    for got, ref in zip(outs + [eager], want):
        assert all(torch.equal(x, y) for x, y in zip(got, ref))
    assert torch.equal(view["score"], scores)
    h2o.h2o_pool_sync_check(pool)
    pool.close()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_the_longest_list(kv):
    """1024 entries, the most of one call: every operator."""
    n = 1024
    b = Both(pages=2 * n + 60, page=16, heads=1, d=64, sequences=2 * n + 1, max_pages=8, kv=kv)
    lens = [int(x) for x in b.rng.integers(0, 4, n)]
    b.write(range(n), 3, lens)
    b.write([2 * n], 100)
    b.attend(range(n), 2, prefix=2 * n)
    b.check()
    b.fork(range(n), range(n, 2 * n))
    b.compact(range(n, 2 * n), 1, 1)
    b.write(range(n), 1)
    b.free(range(n - 1, -1, -1))
    b.check()
    b.attend([-1, 0] * 2 + list(range(n + 4, 2 * n)), 1, prefix=2 * n)
    b.check(errors=16)  # sequence 0 twice
    b.close()


@pytest.mark.parametrize("kept_in_shared", [45056, 45057, 70000])
def test_compact_rows_around_what_shared_memory_holds(kept_in_shared):
    r, h = 40, 1000
    n = kept_in_shared + r
    b = Both(pages=1 + -(-n // 128) + 10, page=128, heads=1, d=64, sequences=1, max_pages=560, seed=1)
    b.write([0], n)
    b.compact([0], h, r)
    b.check()
    b.close()


def test_views_keep_their_pool():
    import gc
    import h2o_heavy_hitter_gb300 as h2o
    pool = h2o.h2o_pool_create(1, 8, 16, 2, 64, 3, 4)
    view = h2o.h2o_pool_view(pool)
    k = view["K"][0, 3]
    del view, pool
    gc.collect()
    others = [torch.full((8, 2, 16, 64), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(64)]
    assert not k.any() and len(others) == 64


def test_large_pool_offsets_pass_32_bits():
    """Slots of a layer beyond 2^31 bytes, and layers beyond that."""
    import h2o_heavy_hitter_gb300 as h2o
    heads, d, page, pages = 8, 128, 128, 10000  # 2.6 GB of keys a layer
    b = Both(2, page, heads, d, 3, 2, seed=5)
    pool = h2o.h2o_pool_create(2, pages, page, heads, d, 3, 2)
    b.pool.close()
    b.pool = pool
    b.layer = 1
    view = h2o.h2o_pool_view(pool, 1)
    view["ref"][:pages - 4] = 1  # only the last pages are free
    torch.cuda.synchronize()
    k64, k = bf16(b.tokens(2, 150))
    v64, v = bf16(b.tokens(2, 150))
    h2o.h2o_pool_write(pool, 1, ints([0, 1]), k, v, ints([150, 140]))
    assert view["table"].tolist() == [[pages - 4, pages - 3], [pages - 2, pages - 1], [-1, -1]]
    assert torch.equal(view["K"][pages - 1, :, :12], k[1, :, 128:140])
    q64, q = bf16(b.queries(1, heads))
    out, lse = h2o.h2o_pool_attend(pool, 1, ints([1]), q, prefix=0)
    kk, vv = (np.concatenate([x[0], x[1][:, :140]], 1) for x in (k64, v64))
    s = np.einsum("hd,hjd->hj", q64[0], kk) / np.sqrt(d)
    p = np.exp(s - s.max(1, keepdims=True))
    want = np.einsum("hj,hjd->hd", p / p.sum(1, keepdims=True), vv)
    assert np.abs(out[0].double().cpu().numpy() - want).max() <= 2.0 ** -7 * np.abs(vv).max()
    h2o.h2o_pool_sync_check(pool)
    pool.close()


def test_inconsistent_states_are_reported_not_followed():
    import h2o_heavy_hitter_gb300 as h2o
    b = Both(pages=12, page=16, heads=2, d=64, sequences=4, max_pages=4)
    b.write([0, 1], 40, [40, 20])
    v = b.view

    def word():
        with pytest.raises(h2o.H2OError) as e:
            h2o.h2o_pool_sync_check(b.pool)
        assert e.value.code == h2o.H2O_EDEVICE
        return int(str(e.value).split("word 0x")[1].split()[0], 16)

    _, q = bf16(b.queries(1, 2))
    v["meta"][0, 0] = 65  # longer than its table
    h2o.h2o_pool_fork(b.pool, 0, ints([0]), ints([2]))
    h2o.h2o_pool_compact(b.pool, 0, ints([0]), 2, 2)
    h2o.h2o_pool_free(b.pool, 0, ints([0]))
    h2o.h2o_pool_attend(b.pool, 0, ints([0]), q)
    assert word() == 2
    v["meta"][0, 0] = 40
    b.check()  # nothing was changed
    v["table"][0, 1] = 99  # no such page
    h2o.h2o_pool_attend(b.pool, 0, ints([0]), q, accumulate=False)
    assert word() == 2
    v["table"][0, 1] = -7
    h2o.h2o_pool_attend(b.pool, 0, ints([1]), q, prefix=0, accumulate=False)
    assert word() == 2
    v["table"][0, 1] = int(b.oracle.table[0, 1])
    b.check()
    v["ref"][int(b.oracle.table[1, 1])] = 2  # a partial page with two holders is not written
    _, k = bf16(b.tokens(1, 1))
    h2o.h2o_pool_write(b.pool, 0, ints([1]), k, k)
    assert word() == 2
    v["ref"][int(b.oracle.table[1, 1])] = 1
    b.check()
    b.close()


def test_refusals():
    import h2o_heavy_hitter_gb300 as h2o
    pool = h2o.h2o_pool_create(2, 8, 16, 2, 64, 3, 4)
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    one = ints([0])
    for bad in (lambda: h2o.h2o_pool_write(pool, 2, one, x, x),
                lambda: h2o.h2o_pool_write(pool, -1, one, x, x),
                lambda: h2o.h2o_pool_attend(pool, -1, one, q),
                lambda: h2o.h2o_pool_attend(pool, 0, one, q, prefix=3),
                lambda: h2o.h2o_pool_attend(pool, 0, one, q[:, :3].contiguous()),
                lambda: h2o.h2o_pool_compact(pool, 0, one, 0, 0),
                lambda: h2o.h2o_pool_compact(pool, 0, one, -1, 4),
                lambda: h2o.h2o_pool_compact(pool, 0, one, 2 ** 31 - 1, 1),
                lambda: h2o.h2o_pool_free(pool, -2, one),
                lambda: h2o.h2o_pool_free(pool, 0, ints([-1] * 1025)),
                lambda: h2o.h2o_pool_attend(pool, 0, one, q, out=q),
                lambda: h2o.h2o_pool_create(1, 8, 24, 2, 64, 3, 4),
                lambda: h2o.h2o_pool_create(1, 1 << 24, 128, 1, 64, 3, 4)):
        with pytest.raises(h2o.H2OError) as e:
            bad()
        assert e.value.code == h2o.H2O_EINVAL
    for bad in (lambda: h2o.h2o_pool_write(pool, 0, one, x.float(), x),
                lambda: h2o.h2o_pool_write(pool, 0, one, x, x[:, :, :3]),
                lambda: h2o.h2o_pool_write(pool, 0, one.long(), x, x),
                lambda: h2o.h2o_pool_write(pool, 0, one, x, x, lens=ints([1, 2])),
                lambda: h2o.h2o_pool_fork(pool, 0, one, ints([1, 2])),
                lambda: h2o.h2o_pool_free(pool, 0, one.cpu()),
                lambda: h2o.h2o_pool_free(pool, 0, [0]),
                lambda: h2o.h2o_pool_attend(pool, 0, one, q, out=q.float()),
                lambda: h2o.h2o_pool_attend(pool, 0, one, q.transpose(0, 1))):
        with pytest.raises((TypeError, ValueError)):
            bad()
    try:
        h2o.h2o_test_fail_allocations(1)
        with pytest.raises(h2o.H2OError) as e:
            h2o.h2o_pool_write(pool, 0, one, x, x)
        assert e.value.code == h2o.H2O_ENOMEM
        h2o.h2o_test_fail_allocations(1)
        with pytest.raises(h2o.H2OError) as e:
            h2o.h2o_pool_create(1, 8, 16, 2, 64, 3, 4)
        assert e.value.code == h2o.H2O_ENOMEM
    finally:
        h2o.h2o_test_fail_allocations(0)
    h2o.h2o_pool_sync_check(pool)
    empty = torch.empty(0, dtype=torch.int32, device="cuda")
    h2o.h2o_pool_free(pool, 0, empty)  # nothing to do
    h2o.h2o_pool_attend(pool, 0, empty, q[:0])
    h2o.h2o_pool_write(pool, 0, one, x[:, :, :0], x[:, :, :0])
    pool.close()
    with pytest.raises(h2o.H2OError):
        h2o.h2o_pool_free(pool, 0, one)
