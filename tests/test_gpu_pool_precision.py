"""How exact the paged cache's attention is: outputs and score increments against float64 with
bounds made of the roundings that the kernels document, on every path of the kernels (own tokens
with few and with many query heads a key head, prefixes with narrow, wide and tiled rows)."""
import numpy as np
import pytest
import torch

from pool_parity import Both, bf16, ints

pytestmark = pytest.mark.gpu

# (batch, heads, group, prefix tokens, own tokens): own tokens alone with rows in one half and in
# both halves of a narrow operand, a prefix with up to 16, up to 32 and more rows a head (one row
# tile, two, three)
PATHS = [(2, 3, 1, 0, 300), (3, 2, 5, 0, 270), (2, 1, 16, 0, 300), (2, 2, 17, 0, 300), (1, 1, 32, 0, 513),
         (3, 2, 3, 400, 70), (2, 2, 11, 400, 150), (1, 2, 32, 400, 90), (40, 2, 1, 400, 30),
         (30, 1, 8, 390, 20), (70, 2, 4, 300, 9)]


def filled(batch, heads, prefix, own, d, kv, K, V):
    """A pool whose sequences 0 .. batch - 1 hold `own` tokens and sequence `batch` the prefix; K, V
    (n, tokens) -> array of one entry's keys, values."""
    page = 32
    pages = -(-own // page) * batch + -(-prefix // page) + 2
    b = Both(pages, page, heads, d, batch + 1, -(-max(own, prefix) // page), kv)
    for seqs, T in ((range(batch), own), ([batch], prefix)):
        if T:
            b.write(seqs, T, score=False, K=K(len(seqs), T), V=V(len(seqs), T))
    return b


def probabilities(b, q64, seqs, prefix):
    """Per entry: (p [q_heads, tokens], values [q_heads, tokens, d], logit error), float64.

    A logit is a sum of d products that are exact in fp32 (bf16 by bf16, or codes by halves of a
    bf16 value); every addition is off by at most 2^-23 of the sum of magnitudes (round to nearest
    or towards zero), and an E4M3 pool's query by 2^-17 of the row's largest value in each product.
    Its scales and its difference to the normaliser are four more fp32 roundings, 2^-24 each, of
    values up to the largest logit and the logarithm of the number of tokens."""
    o, group = b.oracle, q64.shape[1] // b.heads
    for i, s in enumerate(seqs):
        at = [o._slots(s)] if prefix < 0 else [o._slots(prefix), o._slots(s)]
        pages, offs = (np.concatenate([x[j] for x in at]) for j in (0, 1))
        P, V, err = [], [], 0.0
        for hq in range(q64.shape[1]):
            k = o.K[pages, hq // group, offs]
            x = k @ q64[i, hq] / np.sqrt(b.d)
            e = np.exp(x - x.max())
            P.append(e / e.sum())
            V.append(o.V[pages, hq // group, offs])
            size = (np.abs(k) @ np.abs(q64[i, hq])).max()
            lost = 2.0 ** -17 * np.abs(q64[i, hq]).max() * np.abs(k).sum(1).max() if b.kv == "fp8" else 0.0
            err = max(err, (b.d * 2.0 ** -23 * size + lost) / np.sqrt(b.d)
                      + 2.0 ** -22 * (np.abs(x).max() + np.log(len(x))))
        yield np.array(P), np.array(V), err


def attend_and_compare(b, batch, heads, group, prefix, q64, q):
    """One accumulating call from scores of zero. Bounds:

    p: the logit's error twice (its own and the normaliser's), 2^-16 for the two bf16 terms that p
    is held in for its product with v (each off by half a step, 2^-8 relative), 2^-19 for the fp32
    exponentials, scales and joins. out: that of sum p |v|, the fp32 accumulator's (16 tokens a
    step, two steps of 2^-23 each), then its own rounding to bf16, half a step. scores: p's but
    for the two terms, and the fp32 sum over the rows."""
    seqs = list(range(batch))
    assert float(b.view["score"].abs().max()) == 0
    out, lse = b.h2o.h2o_pool_attend(b.pool, 0, ints(seqs), q, prefix=prefix)
    b.h2o.h2o_pool_sync_check(b.pool)
    got = out.double().cpu().numpy()
    score = b.view["score"].double().cpu().numpy()
    shared, worst, bound = 0.0, 0.0, 0.0
    P = 0 if prefix < 0 else int(b.oracle.meta[prefix, 0])
    for i, (p, v, err) in enumerate(probabilities(b, q64, seqs, prefix)):
        want, size = np.einsum("hj,hjd->hd", p, v), np.einsum("hj,hjd->hd", p, np.abs(v))
        rel = 2 * err + 2.0 ** -19
        tol = 2.0 ** -8 * np.abs(want) + (rel + 2.0 ** -16 + (p.shape[1] / 8 + 8) * 2.0 ** -23) * size
        diff = np.abs(got[i] - want)
        assert np.all(diff <= tol), (i, float((diff / tol).max()), np.argwhere(diff > tol)[:4])
        mass = p.reshape(heads, group, -1).sum(1)
        n = mass.shape[1] - P
        own = score[i, :, :n]
        assert np.all(np.abs(own - mass[:, P:]) <= (rel + group * 2.0 ** -24) * mass[:, P:] + 1e-37)
        assert not score[i, :, n:].any()
        shared = shared + mass[:, :P]
        worst, bound = max(worst, rel), bound + rel * mass[:, :P]
    if P:
        assert np.all(np.abs(score[prefix, :, :P] - shared) <= bound + batch * group * 2.0 ** -24 * shared + 1e-37)
        assert not score[prefix, :, P:].any()
    assert worst < 2.0 ** -9  # the bounds say something


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("batch,heads,group,prefix,own", PATHS)
def test_values_that_cancel(batch, heads, group, prefix, own, d, kv):
    """Tokens of probabilities p and p (1 - 0.8 2^-9) in turn, with values of 1 and -1: what is
    left of them is smaller than one rounding of a probability to bf16."""
    odd = lambda T: np.arange(T) % 2

    def K(n, T):
        k = np.zeros((n, heads, T, d))
        k[..., 0] = -0.8 * 2.0 ** -9 * np.sqrt(d) * odd(T)
        return k

    def V(n, T):
        v = np.ones((n, heads, T, d))
        v[:, :, odd(T) == 1] = -1
        return v

    b = filled(batch, heads, prefix, own, d, kv, K, V)
    q64 = np.zeros((batch, heads * group, d))
    q64[..., 0] = 1.0
    attend_and_compare(b, batch, heads, group, batch if prefix else -1, *bf16(q64))
    b.close()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("batch,heads,group,prefix,own", PATHS)
def test_outputs_and_scores_of_ordinary_values(batch, heads, group, prefix, own, d, kv):
    rng = np.random.default_rng(batch * 100 + group)
    K = lambda n, T: rng.standard_normal((n, heads, T, d)) + (rng.random((n, heads, T, 1)) < 0.05) * np.eye(d)[0] * 3
    V = lambda n, T: rng.standard_normal((n, heads, T, d))
    b = filled(batch, heads, prefix, own, d, kv, K, V)
    q64 = rng.standard_normal((batch, heads * group, d)) + 2 * np.eye(d)[0]
    attend_and_compare(b, batch, heads, group, batch if prefix else -1, *bf16(q64))
    b.close()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("batch,group", [(2, 2), (2, 12), (45, 1)])
def test_what_lies_behind_the_last_token_reaches_neither_outputs_nor_scores(batch, group, kv):
    """NaN and infinities in every slot behind a last token and in every free page: keys, values and
    (E4M3) scales."""
    heads, d, prefix, own = 2, 64, 150, 45
    rng = np.random.default_rng(group)
    make = lambda n, T: rng.standard_normal((n, heads, T, d))
    b = filled(batch, heads, prefix, own, d, kv, make, make)
    o, v = b.oracle, b.view
    behind = torch.ones(o.pos.shape[0], o.page, dtype=torch.bool)
    for s in range(batch + 1):
        pages, offs = o._slots(s)
        behind[pages, offs] = False
    behind = behind.cuda()[:, None, :].expand(-1, heads, -1)
    if kv == "fp8":
        for name in "KV":
            v[name][behind] = 0x7f  # the code of NaN
            v[name.lower() + "scale"][behind] = float("nan") if name == "K" else float("inf")
    else:
        v["K"][behind], v["V"][behind] = float("nan"), float("inf")
    q64, q = bf16(rng.standard_normal((batch, heads * group, d)))
    attend_and_compare(b, batch, heads, group, batch, q64, q)
    b.close()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("exponent", [-118, -100, 100])
@pytest.mark.parametrize("batch,heads,group,prefix,own", [PATHS[1], PATHS[4], PATHS[6], PATHS[8], PATHS[10]])
def test_queries_and_keys_of_opposite_magnitudes(batch, heads, group, prefix, own, exponent, kv):
    """Queries of 2^exponent and keys of 2^-exponent have ordinary logits, whichever product of
    theirs with a scale comes first."""
    d = 64
    rng = np.random.default_rng(group)
    K = lambda n, T: rng.standard_normal((n, heads, T, d)) * 2.0 ** -exponent
    V = lambda n, T: rng.standard_normal((n, heads, T, d))
    b = filled(batch, heads, prefix, own, d, kv, K, V)
    q64 = rng.standard_normal((batch, heads * group, d)) * 2.0 ** exponent
    attend_and_compare(b, batch, heads, group, batch if prefix else -1, *bf16(q64))
    b.close()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("batch,heads,group,prefix,own", PATHS)
def test_an_infinite_value_gives_an_infinite_output(batch, heads, group, prefix, own, d):
    """An infinity in a value that is attended to is one in its channel, of its sign, and nowhere
    else: no term of a probability makes a NaN of it."""
    rng = np.random.default_rng(group)
    K = lambda n, T: rng.standard_normal((n, heads, T, d)) * 0.3

    def V(n, T):
        v = rng.standard_normal((n, heads, T, d))
        if T == own:
            v[:, :, T // 2, 3] = np.inf
        if T == (prefix or own):
            v[:, :, T - 1, 5] = -np.inf
        return v

    b = filled(batch, heads, prefix, own, d, "bf16", K, V)
    _, q = bf16(rng.standard_normal((batch, heads * group, d)))
    out, lse = b.h2o.h2o_pool_attend(b.pool, 0, ints(range(batch)), q, prefix=batch if prefix else -1)
    b.h2o.h2o_pool_sync_check(b.pool)
    assert out[..., 3].eq(float("inf")).all() and out[..., 5].eq(float("-inf")).all()
    out[..., [3, 5]] = 0
    assert out.isfinite().all() and lse.isfinite().all()
    b.close()
