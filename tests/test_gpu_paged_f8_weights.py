"""Small softmax weights of the attention over the 8-bit cache: one token far above the rest whose value is zero (an
attention sink), so that the output is what the small weights make of it, and values without a mean, so that their errors
show.

Tolerance.  A weight that is off by at most 2^-8 of itself, as a bf16 weight is, moves the output by at most that: by 2^-8
of its norm where the errors are alike, by 2^-8 of the root of the sum of the squared terms where they are not, which the
norm of 512 such outputs is within 15 % of (5 deviations).  Rounding the output to bf16 adds 2^-8 of its norm.  Errors of the
scores (576 products in fp32, twice: 2^-13 of magnitudes below 1) are part of the 15 %.
"""
import numpy as np
import pytest
import torch

from oracle import paged as O
from tests.paged_harness import F8, SCALE, Cache, attend, dev, forest, random_tree
from top_cache_gb300 import kvo as K

pytestmark = pytest.mark.gpu
LIMIT = 2.15 * 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _built():
    from top_cache_gb300 import build
    build.build()
    yield


def _sink_cache(lens, at, size, seed, block=64):
    """Rows whose rope key is 0 but for a sink's at place `at` of every request: its latent is 0, one element of its rope key
    `size`."""
    c = Cache(lens, block, F8, seed)
    g = np.random.default_rng(seed)
    for r, n in enumerate(lens):
        rows = np.concatenate([g.standard_normal((n, 512)), np.zeros((n, 64))], 1)
        rows[at] = 0.0
        rows[at, 512] = size
        t = np.arange(n)
        K.kvo_paged_write(dev(O.bf16_bits(rows).view(np.int16), torch.int16), dev(c.table[r, t // block] * block + t % block),
                          c.pool, c.n_blocks, block, F8)
    torch.cuda.synchronize()
    c.refresh()
    return c


def _queries(tokens, heads, spread, above, size, seed):
    """Scores of the rows with a deviation of `spread`, the sink's log2 weight `above` that of a score of 0, by head."""
    q = np.zeros((tokens, heads, 576))
    q[:, :, :512] = np.random.default_rng(seed).standard_normal((tokens, heads, 512)) * spread / (SCALE * 512 ** 0.5)
    q[:, :, 512] = np.asarray(above)[None, :] * np.log(2.0) / (SCALE * size)
    return O.bf16_bits(q)


def _check(c, q_bits, cu, kv, out, lse, trees=None):
    q = O.bf16_values(q_bits)
    for r, n in enumerate(np.diff(cu)):
        t, i = np.arange(kv[r]), np.arange(n)
        seen = (t[None, :] <= kv[r] - n + i[:, None] if trees is None else
                O.tree_seen(kv[r], n, trees[r][0], trees[r][1], t, 0, 0))
        k, ok = c.rows_of(r)(t)
        assert ok.all()
        ref, ref_lse = O.attend_seen(k, q[cu[r]:cu[r + 1]], seen, SCALE)[:2]
        got = O.bf16_values(out[cu[r]:cu[r + 1]])
        off = np.linalg.norm(got - ref, axis=-1) / np.linalg.norm(ref, axis=-1)
        assert off.max() <= LIMIT, "request %d: %s" % (r, np.array2string(off.max(0) / 2.0 ** -8, precision=2))
        assert np.abs(lse[cu[r]:cu[r + 1]] - ref_lse).max() < 2.0 ** -12 * (1 + np.abs(ref_lse).max())


# 16, 32 and 64 rows; one request, over every CTA; nearly as many as there are CTAs, each whole
@pytest.mark.parametrize("H", [16, 32, 64])
@pytest.mark.parametrize("lens,at", [([40000], 0), ([40000], 17000), ([1000] * 150, 5)])
def test_a_sink_above_many_rows(H, lens, at):
    c = _sink_cache(lens, at, 4.0, H + at)
    cu = np.arange(len(lens) + 1).astype(np.int32)
    for spread in (0.0, 0.3):  # equal weights: equal errors
        q = _queries(len(lens), H, spread, np.linspace(6.3, 20.7, H), 4.0, H)
        out, lse = attend(c, q, cu, lens)
        _check(c, q, cu, lens, out, lse)


@pytest.mark.parametrize("H", [16, 64])
def test_a_sink_of_large_magnitude(H):
    # its row's scale is 2^5 times the others': what its weight adds is held 2^5 times larger
    c = _sink_cache([30000], 0, 128.0, 3)
    q = _queries(1, H, 0.3, np.linspace(4.0, 16.0, H), 128.0, 4)
    out, lse = attend(c, q, [0, 1], [30000])
    _check(c, q, [0, 1], [30000], out, lse)


@pytest.mark.parametrize("H", [4, 32])
def test_a_sink_under_trees(H):
    g = np.random.default_rng(7)
    lens, new = [9000, 700], [16, 5]
    c = _sink_cache(lens, 0, 4.0, 8)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    trees, masks, depths = forest([random_tree(g, n) for n in new])
    q = _queries(int(cu[-1]), H, 0.3, np.linspace(8.0, 18.0, H), 4.0, 9)
    out, lse = attend(c, q, cu, lens, masks=masks, depths=depths)
    _check(c, q, cu, lens, out, lse, trees)


@pytest.mark.parametrize("H", [16, 64])
def test_a_sink_that_comes_last(H):
    # the running maximum moves by far when most of the sums are there
    c = _sink_cache([20000], 19990, 4.0, 11)
    q = _queries(2, H, 0.3, np.linspace(6.0, 18.0, H), 4.0, 12)
    out, lse = attend(c, q, [0, 2], [20000])
    _check(c, q, [0, 2], [20000], out, lse)


def test_the_check_sees_weights_of_eight_bits():
    # what it is for: the same outputs from weights rounded to E5M2 and E4M3 codes of the rest pass the limit
    g = np.random.default_rng(13)
    v = g.standard_normal((20000, 512))
    w = np.exp(0.3 * g.standard_normal(20000)) * 2.0 ** (7 - 14)

    def code(x, bits, low, top):  # to nearest, `bits` behind the leading one, steps of 2^low at least
        step = 2.0 ** np.maximum(np.floor(np.log2(np.maximum(np.abs(x), 1e-300))) - bits, low)
        return np.clip(np.round(x / step) * step, -top, top)

    hi = code(w, 2, -16, 57344.0)
    for held, fine in ((code(w, 7, -133, 3e38), True), (hi + code(w - hi, 3, -9, 448.0), False)):
        ref, got = w @ v, held @ v
        assert (np.linalg.norm(got - ref) / np.linalg.norm(ref) <= LIMIT) == fine


@pytest.mark.parametrize("H", [16, 32, 64])
def test_scores_whose_steps_pass_the_weights_range(H):
    # log2 scores of 2^22 to 2^36: steps of 1 to 2^13 between fp32 numbers, so the running maximum and what is added to it
    # round to each other.  Scores are off by at most 2^-22 of 576 products: where the largest is ahead by more, the output
    # is its row, rounded to bf16.
    lens = [600, 129]
    c = Cache(lens, 16, F8, 21)
    x = np.random.default_rng(22).standard_normal((2, H, 576))
    for power in range(20, 34):
        q_bits = O.bf16_bits(x * 2.0 ** power)
        out, lse = attend(c, q_bits, [0, 1, 2], lens)
        got, q = O.bf16_values(out), O.bf16_values(q_bits)
        assert np.isfinite(got).all() and np.isfinite(lse).all(), "scores of 2^%d" % (power + 2)
        sure = 0
        for r, n in enumerate(lens):
            k, _ = c.rows_of(r)(np.arange(n))
            z = SCALE * (q[r] @ k.T)
            off = 2.0 ** -22 * 576 * SCALE * (np.abs(q[r]) @ np.abs(k).T).max(-1)
            two = np.sort(z, -1)[:, -2:]
            ahead = two[:, 1] - two[:, 0] > 2 * off + 30
            top = k[z.argmax(-1)][:, :512]
            assert (np.abs(got[r] - top) <= 2.0 ** -8 * np.abs(top))[ahead].all(), "scores of 2^%d" % (power + 2)
            sure += ahead.sum()
        assert sure > H
