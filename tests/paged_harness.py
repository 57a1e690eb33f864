"""What the GPU tests of the 8-bit cache and of draft trees share: caches of random rows, calls, and the check of an
attention against its definition in 64 bits.

Tolerances, from the arithmetic of the kernels (a rounding is off by at most half a step of its type):
16 bits: a weight is rounded to bf16, 2^-8 of it; 4 bits: to fp16, 2^-11, and at least 2^-32 of the running maximum's.
8 bits: a weight W_t = w_t 2^x_t (x_t the row scale's exponent) is rounded to fp16, 2^-11, then split in two: what an E5M2
code leaves is at most an eighth of the power of two below W, and its E4M3 code is off by at most 2^-8 of that power; below
2^-6 codes of the rest are 2^-9 apart, off by 2^-10, where the largest weight is at least 2^7: 2^-17 of it; E5M2 codes end at
2^-16, so weights below 2^-24 of the largest may vanish.  Queries of 8 bits are off by at most 2^-14 of a code's unit, where the row's largest is at least 224.
Sums of n products in fp32 that may truncate are off by n 2^-23 of the sum of magnitudes: 576 for a score (8 bits: 1152, in
two columns, and 2^-18 for adding exponents up to 32 to a score and a maximum), the seen tokens for the weighted values and
the sum of the weights; 2^x adds 2^-21; the output is rounded to bf16.
"""
import numpy as np
import torch

from oracle import paged as O
from tests import test_gpu_paged as P
from top_cache_gb300 import kvo as K

BF16, Q4, F8 = K.KVO_CACHE_BF16, K.KVO_CACHE_Q4, K.KVO_CACHE_F8
SCALE = P.SCALE
dev = P._dev


class Cache(P.Cache):
    def refresh(self):
        self.rows, self.exps = pool_rows(self.pool, self.block, self.fmt)

    def set_rows(self, r, tokens, bits):
        slots = self.table[r, np.asarray(tokens) // self.block] * self.block + np.asarray(tokens) % self.block
        K.kvo_paged_write(dev(bits.view(np.int16), torch.int16), dev(slots), self.pool, self.n_blocks, self.block, self.fmt)
        torch.cuda.synchronize()
        self.refresh()


def pool_rows(pool, block, fmt):
    """float64 rows of a whole pool, from its bytes, and the exponents of its rows' scales."""
    if fmt != F8:
        return P._pool_rows(pool, block, fmt), None
    p = pool.cpu().numpy()
    bits = p[:, 576 * block:].copy().view(np.uint32).reshape(-1)
    return O.dequantize8(p[:, :576 * block].reshape(-1, 576), bits), (bits >> 23).astype(np.int64) - 127


def attend(c, q_bits, cu, kv, scale=SCALE, window=0, sinks=0, masks=None, depths=None, workspace=None, stream=None, want=0):
    T, H = q_bits.shape[:2]
    out = torch.full((T, H, 512), 0x1234, dtype=torch.int16, device="cuda")
    lse = torch.full((T, H), 77.0, dtype=torch.float32, device="cuda")
    status = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    a = (c.pool, c.n_blocks, c.block, c.fmt, dev(c.table), dev(kv), dev(cu))
    q, kw = dev(q_bits.view(np.int16), torch.int16), dict(window=window, sinks=sinks, workspace=workspace, status=status, stream=stream)
    if masks is None:
        K.kvo_paged_attend(*a, q, scale, out, lse, **kw)
    else:
        K.kvo_paged_attend_tree(*a, dev(masks), q, scale, out, lse, depths=None if depths is None else dev(depths), **kw)
    torch.cuda.synchronize()
    assert status.item() == want
    return out.cpu().numpy().view(np.uint16), lse.cpu().numpy()


def causal(kv, n, window, sinks):
    """bool [n][kv]: the tokens that each position sees."""
    p, t = kv - n + np.arange(n)[:, None], np.arange(max(kv, 0))[None, :]
    return (t <= p) & ((window == 0) | (t > p - window) | (t < sinks))


def check(c, q_bits, cu, kv, out, lse, scale=SCALE, window=0, sinks=0, trees=None, tokens=None):
    """Every token (or the listed ones) of every request; trees: (ancestor masks bool [n][n], depths [n]) of each request."""
    q = O.bf16_values(q_bits)
    for r in range(len(kv)):
        n = cu[r + 1] - cu[r]
        mine = [i for i in range(n) if tokens is None or cu[r] + i in tokens]
        if not mine:
            continue
        ids = [cu[r] + i for i in mine]
        t = np.arange(max(kv[r], 0))
        seen = (causal(kv[r], n, window, sinks) if trees is None else
                O.tree_seen(kv[r], n, trees[r][0], trees[r][1], t, window, sinks))[mine]
        some = np.flatnonzero(seen.any(0))  # (a window leaves few)
        k, ok = c.rows_of(r)(some) if len(some) else (np.zeros((0, 576)), np.zeros(0, bool))
        seen = seen[:, some] & ok
        with np.errstate(invalid="ignore"):
            ref, ref_lse, mag, dot, count, w = O.attend_seen(k, q[ids], seen, scale)
            es = 576 * 2.0 ** -23 * dot + 2.0 ** -21
            extra = 0.0
            if c.fmt == F8:
                x = c.exps[np.where(ok, c.table[r, some // c.block].astype(np.int64) * c.block + some % c.block, 0)]
                x = np.where(np.abs(x) > 32, 0, x)
                lost = abs(scale) * 2.0 ** -14 / 224 * np.abs(q[ids]).max(-1) * np.abs(np.where(np.isfinite(k), k, 0)).sum(-1).max(initial=0)
                es = 2 * es + 2.0 ** -18 + lost
                big = w * 2.0 ** x
                most = big.max(-1, keepdims=True, initial=0)
                err = np.minimum(big / 8, most * 2.0 ** -17) + np.minimum(big, most * 2.0 ** -24)
                extra = (err * 2.0 ** -x) @ np.abs(np.where(np.isfinite(k[:, :512]), k[:, :512], 0))
            eps = {BF16: 2.0 ** -8, Q4: 2.0 ** -11, F8: 2.0 ** -8 + 2.0 ** -11}[c.fmt]
            ew = 2 * es + (count[:, None] + 8) * 2.0 ** -23
            if c.fmt == Q4:
                extra = count[:, None, None] * 2.0 ** -32 * np.abs(k[np.isfinite(k)]).max(initial=0)
            tol = (eps + ew[..., None]) * mag + extra + 2.0 ** -8 * 1.01 * np.abs(ref) + 1e-30
            got, got_lse = O.bf16_values(out[ids]), lse[ids].astype(np.float64)
            nan = np.isnan(ref)
            assert np.array_equal(np.isnan(got).any(-1), nan.any(-1)), "request %d: NaN at other places" % r
            bad = np.where(nan, 0.0, np.abs(got - ref)) > np.where(nan, 1.0, tol)
            assert not bad.any(), "request %d: %d of %d off, worst %.3g (tol %.3g)" % (
                r, bad.sum(), bad.size, np.abs(got - ref)[bad].max(), tol[bad][np.argmax(np.abs(got - ref)[bad])])
            none = np.isneginf(ref_lse)
            assert np.array_equal(np.isneginf(got_lse), none) and not got[none].any()
            fine = np.isfinite(ref_lse)
            tl = ew + 2.0 ** -21 * (1 + np.abs(np.where(fine, ref_lse, 0)))
            assert np.all(np.abs(got_lse - ref_lse)[fine] <= np.broadcast_to(tl, fine.shape)[fine])


def run(fmt, lens, new, H, block, window=0, sinks=0, seed=1, scale=SCALE, spread=1.0, pad=0, q_scale=1.0, tokens=None, parents=None,
        words=None):
    """parents: a function of (request, nodes) for trees."""
    c = Cache(lens, block, fmt, seed, spread)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(cu[-1])
    q = O.bf16_bits(q_scale * np.random.default_rng(seed + 1).standard_normal((T + pad, H, 576)))
    trees = masks = depths = None
    if parents:
        trees, masks, depths = forest([parents(r, n) for r, n in enumerate(new)], words, pad)
    out, lse = attend(c, q, cu, lens, scale, window, sinks, masks, depths)
    check(c, q, cu, lens, out, lse, scale, window, sinks, trees, tokens)
    assert (out[T:] == 0x1234).all() and (lse[T:] == 77.0).all()  # rows behind the last sequence stay
    return c, q, cu, out, lse


def forest(all_parents, words=None, pad=0):
    """([(masks, depths)] of each request, mask words [T + pad][words], depths [T + pad])."""
    words = words or max(1, max(-(-len(p) // 32) for p in all_parents))
    trees = [(O.ancestors(p), O.ancestors(p).sum(1) - 1) for p in all_parents]
    masks = [O.mask_words(m, words) for m, _ in trees if len(m)]
    filler = np.full((pad, words), -1, np.int32)
    return trees, np.concatenate(masks + [filler]), np.concatenate([d for _, d in trees] + [np.full(pad, 5)]).astype(np.int32)


def random_tree(g, n):
    """Parents: the root, then nodes below any earlier one, recent ones more often."""
    return [-1] + [int(max(0, i - 1 - g.geometric(0.3) + 1)) for i in range(1, n)] if n else []
