"""Lock-step driver of the paged cache: every call goes to the library's pool (one layer of it)
and to the oracle's, and the whole states are compared."""
import numpy as np
import torch

from oracle import kv_pool


def bf16(x):
    """x (array or tensor) rounded to bf16, as (float64 array, CUDA bf16 tensor)."""
    t = torch.as_tensor(np.asarray(x, np.float32)).to(torch.bfloat16)
    return t.double().numpy(), t.cuda().contiguous()


def ints(values):
    return torch.tensor(list(values), dtype=torch.int32, device="cuda")


class Both:
    def __init__(self, pages, page, heads, d, sequences, max_pages, kv="bf16", layers=1, layer=0,
                 seed=0):
        import h2o_heavy_hitter_gb300 as h2o
        self.h2o, self.kv, self.layer = h2o, kv, layer
        self.pool = h2o.h2o_pool_create(layers, pages, page, heads, d, sequences, max_pages, kv)
        self.view = h2o.h2o_pool_view(self.pool, layer)
        self.oracle = kv_pool.Pool(pages, page, heads, d, sequences, max_pages, kv == "fp8")
        self.rng = np.random.default_rng(seed)
        self.heads, self.d = heads, d

    # values that a kernel can be wrong on: peaked attention, equal scores
    def tokens(self, n, T):
        x = self.rng.standard_normal((n, self.heads, T, self.d))
        x[..., 0] += np.where(self.rng.random((n, self.heads, T)) < 0.1, 6.0, 0.0)
        return x

    def queries(self, n, q_heads):
        x = self.rng.standard_normal((n, q_heads, self.d))
        x[..., 0] += 2.0
        return x

    def scores(self, n, T):
        return np.round(self.rng.random((n, self.heads, T)) * 20) / 4

    def write(self, seqs, T, lens=None, score=True, K=None, V=None):
        n = len(seqs)
        k64, k = bf16(self.tokens(n, T) if K is None else K)
        v64, v = bf16(self.rng.standard_normal((n, self.heads, T, self.d)) if V is None else V)
        sc = self.scores(n, T).astype(np.float32) if score else None
        self.h2o.h2o_pool_write(self.pool, self.layer, ints(seqs), k, v,
                                None if lens is None else ints(lens),
                                None if sc is None else torch.from_numpy(sc).cuda())
        self.oracle.write(seqs, k64, v64, lens, sc)

    def fork(self, src, dst, share=True):
        f = self.h2o.h2o_pool_fork if share else self.h2o.h2o_pool_copy
        f(self.pool, self.layer, ints(src), ints(dst))
        self.oracle.fork(src, dst, share)

    def free(self, seqs):
        self.h2o.h2o_pool_free(self.pool, self.layer, ints(seqs))
        self.oracle.free(seqs)

    def compact(self, seqs, h, r):
        self.h2o.h2o_pool_compact(self.pool, self.layer, ints(seqs), h, r)
        self.oracle.compact(seqs, h, r)

    def attend(self, seqs, q_heads, prefix=-1, accumulate=True):
        """Compares outputs; the scores are left to `check`.

        out: p is rounded to bf16 before the product with v (half a step, 2^-9 relative to
        values in [1, 2) and so at most 2^-8 of any value), and so is the result: an error of at
        most 2^-8 (sum_j p_j |v_j| + |out|), plus fp32 sums, exponentials and logits far
        below that: logits of magnitude up to 64 carry at most d 2^-24 64 / 8 ~ 2^-14 each.
        lse: the same logit error, and fp32's rounding of values up to 64."""
        n = len(seqs)
        q64, q = bf16(self.queries(n, q_heads))
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full(q.shape[:2], 7.0, device="cuda")
        self.h2o.h2o_pool_attend(self.pool, self.layer, ints(seqs), q, prefix, out, lse, accumulate)
        want, want_lse = self.oracle.attend(seqs, q64, prefix, accumulate)
        got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        skipped = np.isnan(want_lse)
        assert np.all(got[skipped] == 7) and np.all(got_lse[skipped] == 7), "a skipped row was written"
        size = np.abs(self.oracle.V).max()
        tol = 2.0 ** -8 * (size + np.abs(want)) + 1e-3 * size
        bad = ~(np.abs(got - want) <= tol) & ~skipped[..., None]
        assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])
        empty = np.isneginf(want_lse)
        assert np.array_equal(np.isneginf(got_lse), empty)
        live = ~skipped & ~empty
        assert np.all(np.abs(got_lse[live] - want_lse[live]) <= 1e-4)
        return out, lse

    def check(self, errors=0):
        """The whole state: whole numbers and stored values equal, scores to fp32. The error word
        holds exactly `errors`."""
        word = 0
        try:
            self.h2o.h2o_pool_sync_check(self.pool)
        except self.h2o.H2OError as e:
            assert e.code == self.h2o.H2O_EDEVICE
            word = int(str(e).split("word 0x")[1].split()[0], 16)
        o, v = self.oracle, {k: x.cpu() for k, x in self.view.items()}
        assert word == o.errors == errors, (word, o.errors, errors)
        o.errors = 0
        for name, want in (("table", o.table), ("meta", o.meta), ("ref", o.ref), ("pos", o.pos)):
            assert np.array_equal(v[name].numpy(), want), name
        for name in "KV":
            if self.kv == "fp8":
                assert np.array_equal(v[name].numpy(), o.codes[name]), name
                assert np.array_equal(v[name.lower() + "scale"].numpy(), o.scale[name], equal_nan=True), name
            else:
                assert np.array_equal(v[name].double().numpy(), getattr(o, name), equal_nan=True), name
        # a probability's error is that of its logit (up to 2^-14, see attend); the sums add fp32
        # roundings of values up to the score itself
        np.testing.assert_allclose(v["score"].double().numpy(), o.score, rtol=2e-4, atol=1e-6)
        # the accumulated scores decide later compactions: both sides go on from the same ones
        o.score = v["score"].double().numpy()

    def close(self):
        self.pool.close()
