"""The paged cache without a GPU: the C entry points' argument checks, and the oracle's own
properties (the CUDA path is compared with it in test_gpu_pool.py)."""
import ctypes

import numpy as np
import pytest

import oracle
from oracle import kv_pool

P, I = ctypes.c_void_p, ctypes.c_int


@pytest.fixture(scope="module")
def lib():
    from h2o_heavy_hitter_gb300 import _build
    lib = ctypes.CDLL(str(_build.build()))
    lib.h2o_last_error.restype = ctypes.c_char_p
    lib.h2o_pool_create.argtypes = [I] * 8 + [ctypes.POINTER(P)]
    return lib


@pytest.mark.parametrize("args,word", [
    ((1, 8, 16, 2, 96, 3, 4, 0), b"head_dim"),
    ((1, 8, 48, 2, 64, 3, 4, 0), b"page_size"),
    ((0, 8, 16, 2, 64, 3, 4, 0), b"layers"),
    ((1, 0, 16, 2, 64, 3, 4, 0), b"pages"),
    ((1, 8, 16, 0, 64, 3, 4, 0), b"heads"),
    ((1, 8, 16, 1025, 64, 3, 4, 0), b"heads"),
    ((1, 8, 16, 2, 64, 0, 4, 0), b"sequences"),
    ((1, 8, 16, 2, 64, 3, 0, 0), b"max_pages"),
    ((1, 8, 16, 2, 64, 3, 65537, 0), b"H2O_MAX_T"),
    ((1, 1 << 23, 128, 2, 64, 3, 4, 0), b"2^31"),
    ((1, 8, 16, 2, 64, 3, 4, 2), b"kv_format"),
    ((1, 8, 16, 2, 64, 3, 4, 0x100), b"kv_format"),
])
def test_create_checks_its_arguments(lib, args, word):
    out = P(1)
    assert lib.h2o_pool_create(*args, ctypes.byref(out)) == -1
    assert word in lib.h2o_last_error() and out.value is None


def test_a_pool_beyond_any_device_is_refused(lib):
    """Sizes whose product passes 64 bits must not wrap to a small allocation."""
    out = P(1)
    assert lib.h2o_pool_create(65535, 8, 16, 1024, 64, 1 << 20, 65536, 0, ctypes.byref(out)) == -3
    assert b"too large" in lib.h2o_last_error() and out.value is None


def test_null_pools_are_refused(lib):
    fake = 0x10000  # never dereferenced
    for name, types, args in (
            ("h2o_pool_write", [P, I, I, P, P, P, I, P, P], (None, 0, 1, fake, fake, fake, 1, None, None)),
            ("h2o_pool_fork", [P, I, I, P, P], (None, 0, 1, fake, fake)),
            ("h2o_pool_copy", [P, I, I, P, P], (None, 0, 1, fake, fake)),
            ("h2o_pool_free", [P, I, I, P], (None, 0, 1, fake)),
            ("h2o_pool_compact", [P, I, I, P, I, I], (None, 0, 1, fake, 1, 1)),
            ("h2o_pool_attend", [P, I, I, P, I, P, I, P, P, I], (None, 0, 1, fake, -1, fake, 1, fake, None, 1)),
            ("h2o_pool_view", [P, I] + [P] * 9, (None, 0) + (None,) * 9),
            ("h2o_pool_sync_check", [P], (None,))):
        fn = getattr(lib, name)
        fn.argtypes = types
        assert fn(*args) == -1 and b"null pool" in lib.h2o_last_error(), name
    lib.h2o_pool_destroy.argtypes, lib.h2o_pool_destroy.restype = [P], None
    lib.h2o_pool_destroy(None)
    assert lib.h2o_pool_create(1, 8, 16, 2, 64, 3, 4, 0, None) == -1


def _filled(rng, fp8=False):
    p = kv_pool.Pool(40, 16, 2, 8, 6, 8, fp8)
    for s, n in enumerate((50, 33, 16)):
        x = rng.standard_normal((2, 1, 2, n, 8)).astype(np.float32).astype(np.float64)
        p.write([s], x[0], x[1], score=rng.random((1, 2, n)))
    return p


def test_oracle_pages_have_the_holders_that_the_tables_say():
    rng = np.random.default_rng(0)
    p = _filled(rng)
    p.fork([0, 1], [3, 4])
    p.compact([3], 9, 9)
    p.free([1])
    p.fork([0], [1], share=False)
    held = np.bincount(p.table[p.table >= 0], minlength=len(p.ref))
    assert np.array_equal(held, p.ref) and p.errors == 0
    assert np.all((p.table >= 0).sum(1) == -(-p.meta[:, 0] // 16))


def test_oracle_attention_is_that_of_the_tokens_in_one_list():
    rng = np.random.default_rng(1)
    p = _filled(rng)
    q = rng.standard_normal((2, 4, 8))
    before = p.score.copy()
    out, lse = p.attend([1, 2], q, prefix=0)
    mass = p.score - before
    assert mass.sum() == pytest.approx(2 * 4)  # each row's probabilities sum to 1
    for i, s in enumerate((1, 2)):
        for hq in range(4):
            h = hq // 2
            k, v = (np.concatenate([x[p._slots(t)[0], h, p._slots(t)[1]] for t in (0, s)]) for x in (p.K, p.V))
            x = k @ q[i, hq] / np.sqrt(8)
            w = np.exp(x)
            np.testing.assert_allclose(out[i, hq], w @ v / w.sum(), rtol=1e-12)
            assert lse[i, hq] == pytest.approx(np.log(w.sum()))


def test_oracle_compaction_selects_as_the_prompt_selection_does():
    rng = np.random.default_rng(2)
    p = _filled(rng)
    scores = np.round(rng.random((2, 50)) * 6) / 6  # many equal
    p.score[0, :, :50] = scores
    p.compact([0], 12, 5)
    for head in range(2):
        kept, _ = oracle.prefill_select(scores[head], 12, 5)
        pages, offs = p._slots(0)
        assert np.array_equal(p.pos[pages, head, offs], np.sort(kept))


def test_oracle_quantises_every_vector_as_the_fp8_oracle_does():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((5, 3, 16)).astype(np.float32).astype(np.float64)
    x[0, 0] = 0
    x[1] *= 1e30
    x[2] *= 1e-30
    c, s = kv_pool.quantise(x)
    for i in np.ndindex(5, 3):
        want = oracle.kv_fp8.quantize_vector(x[i])
        assert np.array_equal(c[i], want[0]) and s[i] == want[1]
