"""Rotations at the borders of the launch: a warp of the grid takes a token's rounds (of 512 / head_dim heads),
several warps share a token where the tokens are few, and warps go on to further tokens where they are many."""
import numpy as np
import pytest
import torch

from draft_parity import Drafts, Rotation, assert_rounded, random_parents
from pool_parity import bf16
from test_gpu_rotary import rotate

pytestmark = pytest.mark.gpu


def warps():
    return torch.cuda.get_device_properties(0).multi_processor_count * 2 * 8  # two blocks an SM, eight warps a block


# tokens as (share of the warps, more): one warp a token, one more token than warps, two warps a token, one token
# too many for that; and few tokens, whose rounds are dealt to warps that get the queries, the keys and the values in
# part, or all that there are
TOKENS = [(1, 0), (1, 1), (2, 0), (2, 1), (3, 0), (4, -1), (0, 7), (0, 1)]
HEADS = [(9, 3, 128), (9, 5, 128), (3, 1, 128), (17, 9, 64), (1, 20, 64)]


def tokens(share):
    return (warps() // share[0] if share[0] else 0) + share[1]


@pytest.mark.parametrize("share", TOKENS)
@pytest.mark.parametrize("hq,h,d", HEADS)
def test_rows(share, hq, h, d):
    n = tokens(share)
    rng = np.random.default_rng(n + hq)
    r = Rotation(d, d // 2, "half" if h % 2 else "interleaved", norm=True)
    q, k, v = (bf16(rng.standard_normal((1, n, x, d)))[0] for x in (hq, h, h))
    positions = rng.integers(0, 1 << 20, (1, n))
    got = rotate(r, q, k, v, positions, rng)
    assert_rounded(got[0], *r(q, positions, 0), "q")
    assert_rounded(got[1], *r(k, positions, 1), "k")
    assert np.array_equal(got[2], v)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("share", TOKENS)
@pytest.mark.parametrize("hq,h,d", HEADS[:2] + HEADS[3:4])
def test_pages(share, hq, h, d, kv):
    """The same into pages: in two entries, of which one has fewer tokens than the call allows; then drafts."""
    n = tokens(share)
    T = max(1, n // 2)
    lens = [T, max(0, T - 3)]
    b = Drafts(pages=2 * (-(-(T + 40) // 128)) + 2, page=128, heads=h, d=d, sequences=3, max_pages=-(-(T + 40) // 128), kv=kv, seed=n)
    r = Rotation(d, d // 2, norm=True)
    b.append([2, 0], T, hq // h * h, r, lens=lens)
    b.check()
    t = min(T, 31)
    b.append([0, 2], t, hq // h * h, r, lens=[t, t // 2], parent=random_parents(b.rng, 2, t))
    b.check()
    b.close()
