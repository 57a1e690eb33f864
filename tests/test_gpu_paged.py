"""Paged device cache (kvo_paged_*) against its plain definitions in 64 bits (oracle/paged.py).

Plans, codes and read-back rows have to be equal.  Attention tolerances, from the arithmetic
of the kernel: each softmax weight is rounded to bf16 (relative error at most 2^-8) or, over
the 4-bit cache, to fp16 (2^-11; below 2^-14 of 2^7 times the running maximum's weight 2^-25
of that, absolute), the output to bf16 (2^-8 |out|).  Sums of n products in fp32 that may
truncate are off by n 2^-23 of the sum of magnitudes: 576 for a score, which moves a weight
by as much (and the sum of the weights by as much again), and the seen tokens for the
weighted values and for the sum; 2^x adds 2^-21.
"""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from oracle import paged as O
from top_cache_gb300 import kvo as K

pytestmark = pytest.mark.gpu

SCALE = 1.0 / np.sqrt(192.0)
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16, Q4 = K.KVO_CACHE_BF16, K.KVO_CACHE_Q4


@pytest.fixture(scope="module", autouse=True)
def _built():
    from top_cache_gb300 import build
    build.build()
    yield


def _dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


# ---- plan -----------------------------------------------------------------------------------

def _run_plan(lengths, new, block, table, ring, bounds, n_slots, window, sinks, in_place=False):
    R = len(lengths)
    old, b_in = _dev(lengths), _dev(bounds, torch.int64)
    e = lambda n: torch.full((n,), 77, dtype=torch.int32, device="cuda")  # noqa: E731
    lo = old if in_place else e(R)
    bo = b_in if in_place else torch.full((2,), 77, dtype=torch.int64, device="cuda")
    o = dict(table=_dev(table), ring=_dev(ring), bounds=bo, lengths=lo, kv_lens=e(R), cu=e(R + 1), slots=e(n_slots),
             status=e(R))
    K.kvo_paged_plan(old, _dev(new), block, o["table"], o["ring"], b_in, bo, lo, o["kv_lens"], o["cu"], o["slots"],
                     o["status"], window=window, sinks=sinks)
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in o.items()}


def _same(got, want):
    for k in ("status", "cu", "lengths", "kv_lens", "bounds", "table", "slots", "ring"):
        assert np.array_equal(got[k], want[k]), k


@pytest.mark.parametrize("R,block,M,window,sinks,spare", [
    (1, 8, 1, 0, 0, 0), (1, 64, 40, 0, 0, 100), (5, 16, 9, 20, 4, 30), (31, 24, 12, 50, 0, 8), (64, 64, 30, 700, 64, 400),
    (1023, 8, 5, 0, 0, 300), (1025, 16, 6, 33, 17, 5000), (2500, 8, 7, 9, 3, 1500), (4096, 128, 4, 130, 1, 3000)])
def test_plan_steps(R, block, M, window, sinks, spare):
    g = np.random.default_rng(R)
    n_blocks = R + spare + 1
    ring = np.concatenate([g.permutation(n_blocks), np.full(3, -1)]).astype(np.int32)
    state = dict(lengths=np.zeros(R, np.int32), table=np.full((R, M), -1, np.int32), ring=ring,
                 bounds=np.array([0, n_blocks], np.int64))
    refused = 0
    for step in range(6):
        # prompts, single tokens, idle requests, some that end, some past the table
        new = g.choice([0, 1, 1, 1, 4, block, 3 * block + 1, -1, M * block + 1], R)
        n_slots = int(np.maximum(new, 0).sum()) - (3 if step == 4 else 0)
        n_slots = max(0, n_slots) + (5 if step == 1 else 0)
        args = (state["lengths"], new, block, state["table"], state["ring"], state["bounds"], n_slots)
        want = O.plan(*args, window=window, sinks=sinks)
        _same(_run_plan(*args, window, sinks, in_place=step % 2 == 1), want)
        refused += int((want["status"] != O.OK).sum())
        live = set(want["ring"][i % len(ring)] for i in range(want["bounds"][0], want["bounds"][1]))
        assert len(live) == want["bounds"][1] - want["bounds"][0]  # no id is free twice
        state = {k: want[k] for k in state}
    assert refused > 0


def test_plan_far_ring_positions():
    # the counters only grow: positions past 2^32 and a wrapped ring
    ring = np.arange(7, dtype=np.int32)
    args = (np.array([3, 8], np.int32), np.array([9, 20]), 8, np.array([[100, -1, -1, -1], [101, -1, -1, -1]], np.int32),
            ring, np.array([(1 << 33) + 5, (1 << 33) + 11], np.int64), 29)
    _same(_run_plan(*args, 0, 0), O.plan(*args))


# ---- rows -----------------------------------------------------------------------------------

def _pool(n_blocks, block, fmt, byte=0xA5):
    return torch.full((n_blocks, K.kvo_paged_block_bytes(fmt, block)), byte, dtype=torch.uint8, device="cuda")


def _pool_rows(pool, block, fmt):
    """float64 rows of a whole pool (from its bytes, by the oracle)."""
    p = pool.cpu().numpy()
    if fmt == BF16:
        return O.bf16_values(p.view(np.uint16).reshape(-1, 576))
    c = p[:, :288 * block].reshape(-1, 288)
    codes = np.stack([c & 15, c >> 4], -1).reshape(-1, 576)
    scales = p[:, 288 * block:].reshape(-1, 36)
    return O.dequantize(codes, np.minimum(scales, 127))


def _special_rows(n, seed):
    g = np.random.default_rng(seed)
    x = g.standard_normal((n, 576)) * np.exp(3 * g.standard_normal((n, 36))).repeat(16, 1)
    x[g.random((n, 576)) < 0.05] = 0.0
    bits = O.bf16_bits(x)
    if n > 4:
        bits[0] = 0                      # a zero row
        bits[1, :16] = 0x0001            # subnormals
        bits[1, 16:32] = 0x7F7F          # the largest value: saturates
        bits[2, 3], bits[2, 40], bits[2, 70] = 0x7F80, 0xFF80, 0x7FC1  # infinities and NaN, one group each
        bits[3] = g.integers(0, 0x7F80, 576).astype(np.uint16)         # every magnitude
        # ties of both roundings: scale 2^k, elements on the midpoints of the codes
        bits[4, :16] = O.bf16_bits(np.array([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, 0]))
        bits[4, 16:32] = O.bf16_bits(np.full(16, 6 * 1.0625))
        bits[4, 32:48] = O.bf16_bits(np.full(16, 6 * 1.1875))
    return bits


@pytest.mark.parametrize("fmt", [BF16, Q4])
@pytest.mark.parametrize("n,block", [(1, 8), (7, 24), (8, 16), (129, 64), (1000, 128), (4097, 8)])
def test_rows_written_and_read(n, block, fmt):
    g = np.random.default_rng(n)
    n_blocks = -(-n // block) + 2
    bits = _special_rows(n, n)
    slots = g.permutation(n_blocks * block)[:n].astype(np.int32)
    skip = g.random(n) < 0.1
    slots[skip] = g.choice([-1, -7, n_blocks * block, 2 ** 31 - 1], int(skip.sum()))
    pool = _pool(n_blocks, block, fmt)
    before = pool.cpu().numpy().copy()
    K.kvo_paged_write(_dev(bits.view(np.int16), torch.int16), _dev(slots), pool, n_blocks, block, fmt)
    back = torch.full((n, 576), 0x1234, dtype=torch.int16, device="cuda")
    K.kvo_paged_read(pool, n_blocks, block, fmt, _dev(slots), back)
    torch.cuda.synchronize()
    got = back.cpu().numpy().view(np.uint16)
    assert (got[skip] == 0x1234).all()
    after = pool.cpu().numpy()
    if fmt == BF16:
        assert np.array_equal(got[~skip], bits[~skip])
        want = before.view(np.uint16).reshape(-1, 576).copy()
        want[slots[~skip]] = bits[~skip]
        assert np.array_equal(after.view(np.uint16).reshape(-1, 576), want)
        return
    codes, scales = O.quantize(bits)
    v = O.dequantize(codes, scales)[~skip]
    assert np.array_equal(O.bf16_values(got[~skip]), v, equal_nan=True)
    # the bytes: other rows untouched, written ones as the definition gives them (a zero may have either sign)
    want_c, want_s = before[:, :288 * block].reshape(-1, 288).copy(), before[:, 288 * block:].reshape(-1, 36).copy()
    got_c, got_s = after[:, :288 * block].reshape(-1, 288), after[:, 288 * block:].reshape(-1, 36)
    at = slots[~skip]
    want_s[at] = scales[~skip]
    assert np.array_equal(got_s, want_s)
    keep = np.ones(len(want_c), bool)
    keep[at] = False
    assert np.array_equal(got_c[keep], want_c[keep])
    assert not (v[0] if n > 4 and not skip[0] else np.zeros(1)).any()


# ---- attention ------------------------------------------------------------------------------

class Cache:
    """A cache of random rows for requests of the given lengths, blocks in random order."""

    def __init__(self, lens, block, fmt, seed, spread=1.0, extra=3):
        g = np.random.default_rng(seed)
        self.block, self.fmt, self.lens = block, fmt, list(lens)
        used = [-(-n // block) for n in lens]
        self.M = max(max(used), 1) + extra
        self.n_blocks = sum(used) + 2
        ids = g.permutation(self.n_blocks)
        self.table = np.full((len(lens), self.M), -1, np.int32)
        k = 0
        for r, n in enumerate(used):
            self.table[r, :n] = ids[k:k + n]
            k += n
        self.pool = _pool(self.n_blocks, block, fmt, 0xFF)  # rows that are not written read as NaN
        for r, n in enumerate(lens):
            t = np.arange(n)
            if n == 0:
                continue
            slots = self.table[r, t // block] * block + t % block
            bits = O.bf16_bits(spread * g.standard_normal((n, 576)))
            K.kvo_paged_write(_dev(bits.view(np.int16), torch.int16), _dev(slots), self.pool, self.n_blocks, block, fmt)
        torch.cuda.synchronize()
        self.refresh()

    def refresh(self):
        self.rows = _pool_rows(self.pool, self.block, self.fmt)

    def rows_of(self, r):
        def f(t):
            b = self.table[r, t // self.block].astype(np.int64)
            ok = (b >= 0) & (b < self.n_blocks)
            return self.rows[np.where(ok, b * self.block + t % self.block, 0)], ok
        return f


def _attend(c, q_bits, cu, kv, scale, window=0, sinks=0, workspace=None, stream=None):
    T, H = q_bits.shape[:2]
    out = torch.full((T, H, 512), 0x1234, dtype=torch.int16, device="cuda")
    lse = torch.full((T, H), 77.0, dtype=torch.float32, device="cuda")
    status = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    K.kvo_paged_attend(c.pool, c.n_blocks, c.block, c.fmt, _dev(c.table), _dev(kv), _dev(cu),
                       _dev(q_bits.view(np.int16), torch.int16), scale, out, lse, window=window, sinks=sinks,
                       workspace=workspace, status=status, stream=stream)
    torch.cuda.synchronize()
    assert status.item() == 0
    return out.cpu().numpy().view(np.uint16), lse.cpu().numpy()


def _check(c, q_bits, cu, kv, scale, window, sinks, out, lse, tokens=None):
    """Every token (or the listed ones) of every request."""
    q = O.bf16_values(q_bits)
    eps_w = 2.0 ** -8 if c.fmt == BF16 else 2.0 ** -11
    for r in range(len(kv)):
        ids = [i for i in range(cu[r], cu[r + 1]) if tokens is None or i in tokens]
        if not ids:
            continue
        pos = [kv[r] - (cu[r + 1] - cu[r]) + (i - cu[r]) for i in ids]
        ref, ref_lse, mag, dot, n = O.attend(c.rows_of(r), q[ids], pos, scale, window, sinks)
        got, got_lse = O.bf16_values(out[ids]), lse[ids].astype(np.float64)
        with np.errstate(invalid="ignore"):
            es = (576 * 2.0 ** -23) * dot + 2.0 ** -21                       # a score, a weight
            ew = 2 * es + (n[:, None] + 8) * 2.0 ** -23
            flush = 0.0 if c.fmt == BF16 else n[:, None, None] * 2.0 ** -32 * np.abs(c.rows[np.isfinite(c.rows)]).max(initial=0)
            tol = (eps_w + ew[..., None]) * mag + flush + 2.0 ** -8 * 1.01 * np.abs(ref) + 1e-30
            nan = np.isnan(ref)
            assert np.array_equal(np.isnan(got).any(-1), nan.any(-1)), "request %d: NaN at other places" % r
            err = np.where(nan, 0.0, np.abs(got - ref))
            bad = err > np.where(nan, 1.0, tol)
            assert not bad.any(), "request %d: %d of %d off, worst %.3g (tol %.3g)" % (
                r, bad.sum(), bad.size, err[bad].max(), tol[bad][np.argmax(err[bad])])
            none = np.isneginf(ref_lse)
            assert np.array_equal(np.isneginf(got_lse), none)
            ok = np.isfinite(ref_lse)
            tl = ew + 2.0 ** -21 * (1 + np.abs(np.where(ok, ref_lse, 0)))
            assert np.all(np.abs(got_lse - ref_lse)[ok] <= np.broadcast_to(tl, ok.shape)[ok])
            assert not got[none].any()


def _run(lens, new, H, block, fmt, window=0, sinks=0, seed=1, scale=SCALE, spread=1.0, pad=0, q_scale=1.0, tokens=None):
    c = Cache(lens, block, fmt, seed, spread)
    g = np.random.default_rng(seed + 1)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = O.bf16_bits(q_scale * g.standard_normal((int(cu[-1]) + pad, H, 576)))
    out, lse = _attend(c, q, cu, lens, scale, window, sinks)
    _check(c, q, cu, lens, scale, window, sinks, out, lse, tokens)
    T = int(cu[-1])
    assert (out[T:] == 0x1234).all() and (lse[T:] == 77.0).all()  # rows behind the last sequence stay
    return c, q, cu, out, lse


FORMATS = [pytest.param(BF16, id="bf16"), pytest.param(Q4, id="q4")]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("H", [1, 16, 17, 32, 40, 64, 128])
def test_one_token(fmt, H):
    _run([1], [1], H, 8, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("H,lens", [(16, [127]), (16, [128]), (16, [129]), (5, [300, 1, 77]), (32, [1000]), (24, [257, 640, 3]),
                                    (64, [500, 128]), (128, [700]), (100, [390])])
def test_decode(fmt, H, lens):
    _run(lens, [1] * len(lens), H, 16, fmt, seed=H)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("block", [8, 24, 40, 64, 128, 192])
def test_block_sizes(fmt, block):
    _run([block - 1, block, 3 * block + 5], [1, 2, 1], 8, block, fmt, seed=block)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("H,new,lens", [(16, [4, 4], [260, 131]), (3, [5, 1, 7], [300, 9, 7]), (20, [33], [161]), (128, [4], [260]),
                                        (1, [200], [450]), (7, [64, 3], [64, 130]), (16, [0, 2, 0], [50, 200, 0])])
def test_several_positions(fmt, H, new, lens):
    _run(lens, new, H, 16, fmt, seed=len(lens) + H, pad=3)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("H,new,lens,window,sinks", [
    (16, [1], [1000], 1, 0), (16, [1], [1000], 128, 0), (16, [1, 1], [1000, 90], 100, 4), (8, [9, 4], [900, 300], 40, 1),
    (3, [150], [700], 130, 70), (64, [3], [2000], 129, 128), (128, [2], [800], 300, 200), (16, [5], [400], 4000, 4),
    (16, [3], [1500], 64, 5000), (2, [300], [300], 17, 2)])
def test_window_and_sinks(fmt, H, new, lens, window, sinks):
    _run(lens, new, H, 24, fmt, window, sinks, seed=window)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("scale,q_scale", [(0.0, 1.0), (-0.1, 1.0), (3.0, 1.0), (SCALE, 1e4), (1e-6, 1e20), (SCALE, 1e-30)])
def test_scales(fmt, scale, q_scale):
    # a large scale moves the running maximum by far more than 2^8 from block to block (O^T is rescaled in TMEM)
    _run([600, 129], [1, 3], 16, 16, fmt, seed=5, scale=scale, q_scale=q_scale)


@pytest.mark.parametrize("fmt", FORMATS)
def test_growing_scores(fmt):
    # each block's rows larger than the last one's: a new maximum in every block
    c = Cache([900], 16, fmt, 3)
    g = np.random.default_rng(4)
    bits = O.bf16_bits(g.standard_normal((900, 576)) * (1 + np.arange(900) / 30.0)[:, None])
    slots = c.table[0, np.arange(900) // 16] * 16 + np.arange(900) % 16
    K.kvo_paged_write(_dev(bits.view(np.int16), torch.int16), _dev(slots), c.pool, c.n_blocks, 16, fmt)
    c.refresh()
    for H in (16, 32, 64):
        q = O.bf16_bits(g.standard_normal((2, H, 576)))
        out, lse = _attend(c, q, [0, 2], [900], SCALE)
        _check(c, q, [0, 2], [900], SCALE, 0, 0, out, lse)


@pytest.mark.parametrize("fmt", FORMATS)
def test_positions_that_see_nothing(fmt):
    # more query tokens than cached ones (the first positions are negative), an empty cache, a request without queries
    c = Cache([3, 0, 40], 8, fmt, 6)
    q = O.bf16_bits(np.random.default_rng(7).standard_normal((7, 16, 576)))
    cu = [0, 5, 7, 7]
    out, lse = _attend(c, q, cu, [3, 0, 40], SCALE)
    _check(c, q, cu, [3, 0, 40], SCALE, 0, 0, out, lse)
    assert np.isneginf(lse[[0, 1, 5, 6]]).all() and np.isfinite(lse[2:5]).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_unmapped_blocks_are_not_seen(fmt):
    c = Cache([500, 200], 16, fmt, 8)
    c.table[0, [0, 7, 8, 31]] = [-1, -5, c.n_blocks, 2 ** 31 - 1]
    c.table[1, :] = -1
    q = O.bf16_bits(np.random.default_rng(9).standard_normal((4, 20, 576)))
    out, lse = _attend(c, q, [0, 2, 4], [500, 200], SCALE)
    _check(c, q, [0, 2, 4], [500, 200], SCALE, 0, 0, out, lse)
    assert np.isneginf(lse[2:]).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("H", [4, 16, 128])
def test_what_is_not_finite_stays_with_those_that_see_it(fmt, H):
    # NaN and infinities in rows that only some positions of a tile see: the last token, and one that leaves the window
    c = Cache([400], 16, fmt, 10)
    rows = O.bf16_bits(np.random.default_rng(11).standard_normal((3, 576)))
    rows[0, 5], rows[1, 511], rows[2, 100] = 0x7FC0, 0x7F80, 0xFF80
    slots = [c.table[0, t // 16] * 16 + t % 16 for t in (399, 397, 299)]
    K.kvo_paged_write(_dev(rows.view(np.int16), torch.int16), _dev(slots), c.pool, c.n_blocks, 16, fmt)
    c.refresh()
    q = O.bf16_bits(np.abs(np.random.default_rng(12).standard_normal((6, H, 576))) + 0.1)
    for window in (0, 100):
        out, lse = _attend(c, q, [0, 6], [400], SCALE, window=window)
        got = np.isnan(O.bf16_values(out)).any((1, 2))
        # positions 394..399: token 299 is seen by all without a window, by 394..398 with one of 100
        want = np.ones(6, bool) if window == 0 else np.array([True] * 6)
        if window == 100:
            want[:] = [p - 100 < 299 or p >= 397 for p in range(394, 400)]
        if fmt == BF16:
            # -inf where the query is positive: a weight of 0, and 0 times infinity in that column alone
            fine = [p for p in range(6) if 394 + p < 397]
            assert not np.isnan(O.bf16_values(out[fine])[..., :100]).any()
            assert got[[p for p in range(6) if 394 + p >= 397]].all()
        else:
            assert np.array_equal(got, want)
    out, lse = _attend(c, q, [0, 6], [400], SCALE, window=20)  # 299 is out of every window
    got = np.isnan(O.bf16_values(out)).any((1, 2))
    assert not got[:3].any() and got[3:].all()
    ref, *_ = O.attend(c.rows_of(0), O.bf16_values(q[:3]), [394, 395, 396], SCALE, 20)
    assert np.abs(O.bf16_values(out[:3]) - ref).max() < 2.0 ** -6 * np.abs(ref).max()


@pytest.mark.parametrize("fmt", FORMATS)
def test_split_and_joined(fmt):
    # one request over every CTA, and tiles of other requests between: partial results of many CTAs are joined
    _run([30011], [1], 16, 64, fmt, seed=13)
    _run([9000, 5, 3001, 0, 700], [1, 1, 2, 0, 1], 64, 64, fmt, seed=14)
    _run([5000], [2], 128, 64, fmt, seed=15)


@pytest.mark.parametrize("fmt", FORMATS)
def test_many_tiles(fmt):
    # more tiles than are listed: whole tiles per CTA; sampled tokens
    new = [700, 0, 1, 900, 17]
    lens = [700, 5, 200, 1300, 17]
    _run(lens, new, 90, 64, fmt, 100, 3, seed=16, tokens={0, 1, 350, 699, 700, 701, 1100, 1600, 1601, 1617})


def test_many_requests():
    g = np.random.default_rng(17)
    lens = g.integers(0, 40, 1500).tolist()
    new = [min(n, 1) for n in lens]
    _run(lens, new, 2, 8, BF16, seed=17, tokens=set(range(0, 1500, 37)))
    _run([9] * 4096, [1] * 4096, 1, 16, Q4, seed=18, tokens=set(range(0, 4096, 111)))


def test_same_bits_again_and_on_another_stream():
    c = Cache([7000, 300], 64, Q4, 19)
    q = O.bf16_bits(np.random.default_rng(20).standard_normal((3, 16, 576)))
    a = _attend(c, q, [0, 1, 3], [7000, 300], SCALE)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, s):
        b = _attend(c, q, [0, 1, 3], [7000, 300], SCALE, stream=stream)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1].view(np.uint32), b[1].view(np.uint32))
    # two calls in flight, each with its own workspace
    dev = [torch.full((3, 16, 512), 0, dtype=torch.int16, device="cuda") for _ in range(2)]
    args = (c.pool, c.n_blocks, 64, Q4, _dev(c.table), _dev([7000, 300]), _dev([0, 1, 3]), _dev(q.view(np.int16), torch.int16), SCALE)
    torch.cuda.synchronize()
    for o, st in zip(dev, (s, torch.cuda.Stream())):
        K.kvo_paged_attend(*args, o, stream=st)
    torch.cuda.synchronize()
    assert all(np.array_equal(o.cpu().numpy().view(np.uint16), a[0]) for o in dev)


# ---- together ---------------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", FORMATS)
def test_a_serving_loop_in_one_graph(fmt):
    """Plan, write and attend of a decode step captured once and replayed: requests grow, pass block borders, give
    blocks back and end, with nothing read on the host."""
    R, B, M, H, W, S = 5, 8, 12, 16, 21, 3
    g = np.random.default_rng(21)
    T = 2 * R
    n_blocks = 26
    i32 = lambda a: _dev(a)  # noqa: E731
    ring = i32(np.concatenate([g.permutation(n_blocks), [-1, -1]]))
    bounds = _dev([0, n_blocks], torch.int64)
    lengths, table = i32(np.zeros(R)), i32(np.full((R, M), -1))
    new, kv, cu, slots, status = i32(np.zeros(R)), i32(np.zeros(R)), i32(np.zeros(R + 1)), i32(np.zeros(T)), i32(np.zeros(R))
    pool = _pool(n_blocks, B, fmt, 0xFF)
    rows = torch.zeros(T, 576, dtype=torch.int16, device="cuda")
    q = torch.zeros(T, H, 576, dtype=torch.int16, device="cuda")
    out = torch.zeros(T, H, 512, dtype=torch.int16, device="cuda")
    lse = torch.zeros(T, H, dtype=torch.float32, device="cuda")
    ws = torch.empty(K.kvo_paged_attend_workspace_size(R, T, H, 0), dtype=torch.uint8, device="cuda")

    def step():
        K.kvo_paged_plan(lengths, new, B, table, ring, bounds, bounds, lengths, kv, cu, slots, status, window=W, sinks=S)
        K.kvo_paged_write(rows, slots, pool, n_blocks, B, fmt)
        K.kvo_paged_attend(pool, n_blocks, B, fmt, table, kv, cu, q, SCALE, out, lse, window=W, sinks=S, workspace=ws)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()  # nothing new: loads the modules
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    torch.cuda.synchronize()
    plan = dict(lengths=np.zeros(R, np.int32), table=np.full((R, M), -1, np.int32), ring=ring.cpu().numpy(),
                bounds=np.array([0, n_blocks], np.int64))
    history = [np.zeros((0, 576), np.uint16) for _ in range(R)]
    for it in range(60):
        n = g.choice([0, 1, 1, 2, 2], R)
        n[(plan["lengths"] > 80) | (g.random(R) < 0.02)] = -1
        bits = O.bf16_bits(g.standard_normal((T, 576)))
        qb = O.bf16_bits(g.standard_normal((T, H, 576)))
        new.copy_(_dev(n)); rows.copy_(_dev(bits.view(np.int16), torch.int16)); q.copy_(_dev(qb.view(np.int16), torch.int16))
        graph.replay()
        torch.cuda.synchronize()
        want = O.plan(plan["lengths"], n, B, plan["table"], plan["ring"], plan["bounds"], T, window=W, sinks=S)
        assert np.array_equal(slots.cpu().numpy(), want["slots"]) and np.array_equal(status.cpu().numpy(), want["status"])
        assert np.array_equal(table.cpu().numpy(), want["table"]) and np.array_equal(ring.cpu().numpy(), want["ring"])
        assert np.array_equal(bounds.cpu().numpy(), want["bounds"])
        got, gl = O.bf16_values(out.cpu().numpy().view(np.uint16)), lse.cpu().numpy()
        for r in range(R):
            a, b = want["cu"][r], want["cu"][r + 1]
            if n[r] < 0:
                history[r] = history[r][:0]
            if want["status"][r] != O.OK:
                assert np.isneginf(gl[a:b]).all() and not got[a:b].any()
                continue
            x = bits[a:b]
            if fmt == Q4 and b > a:
                x = O.bf16_bits(O.dequantize(*O.quantize(x)))
            history[r] = np.concatenate([history[r], x])
            if b > a:
                h = O.bf16_values(history[r])
                L = len(h)
                ref, rl, mag, dot, _ = O.attend(lambda t: (h[t], np.ones(len(t), bool)), O.bf16_values(qb[a:b]), range(L - (b - a), L), SCALE, W, S)
                es = (576 * 2.0 ** -23) * dot + 2.0 ** -20
                tol = (2.0 ** -8 + 4 * es[..., None]) * mag + 2.0 ** -8 * 1.01 * np.abs(ref) + 1e-30
                assert np.all(np.abs(got[a:b] - ref) <= tol), (it, r)
                assert np.all(np.abs(gl[a:b] - rl) <= 4 * es + 2.0 ** -20 * (1 + np.abs(rl)))
        plan = {k: want[k] for k in plan}
    assert int(plan["bounds"][1]) > 2 * n_blocks  # blocks were given back and taken again


def test_plan_bad_block_ids_give_no_slot():
    ring = np.array([-3, 2 ** 31 - 1, 1 << 28, 5], np.int32)
    args = (np.array([0, 0, 0, 0], np.int32), np.array([2, 2, 2, 2]), 8, np.full((4, 1), -1, np.int32), ring,
            np.array([0, 4], np.int64), 9)
    got = _run_plan(*args, 0, 0)
    _same(got, O.plan(*args))
    assert got["slots"].tolist() == [-1] * 6 + [40, 41, -1]


@pytest.mark.parametrize("fmt", FORMATS)
def test_rows_past_32_bit_offsets(fmt):
    # a pool of more than 4 GB: blocks at its far end
    B = 4096
    n_blocks = (5 << 30) // K.kvo_paged_block_bytes(fmt, B)
    pool = torch.empty(n_blocks, K.kvo_paged_block_bytes(fmt, B), dtype=torch.uint8, device="cuda")
    L = 300
    bits = O.bf16_bits(np.random.default_rng(23).standard_normal((L, 576)))
    slots = (n_blocks - 1) * B + np.arange(L)
    K.kvo_paged_write(_dev(bits.view(np.int16), torch.int16), _dev(slots), pool, n_blocks, B, fmt)
    back = torch.zeros(L, 576, dtype=torch.int16, device="cuda")
    K.kvo_paged_read(pool, n_blocks, B, fmt, _dev(slots), back)
    torch.cuda.synchronize()
    rows = O.bf16_values(back.cpu().numpy().view(np.uint16))
    assert np.array_equal(rows, O.bf16_values(bits) if fmt == BF16 else O.dequantize(*O.quantize(bits)))

    class C:
        pass
    c = C()
    c.pool, c.n_blocks, c.block, c.fmt, c.table, c.rows = pool, n_blocks, B, fmt, np.array([[n_blocks - 1, 7]], np.int32), rows
    c.rows_of = lambda r: lambda t: (rows[t], np.ones(len(t), bool))
    q = O.bf16_bits(np.random.default_rng(24).standard_normal((1, 40, 576)))
    out, lse = _attend(c, q, [0, 1], [L], SCALE)
    _check(c, q, [0, 1], [L], SCALE, 0, 0, out, lse)


@pytest.mark.parametrize("fmt", FORMATS)
def test_not_finite_beside_a_half_empty_tile(fmt):
    # tiles of 64 rows, the last request's only 16 of them filled: the other half's rows lie past the queries
    c = Cache([200, 90], 16, fmt, 25)
    rows = O.bf16_bits(np.random.default_rng(26).standard_normal((2, 576)))
    rows[0, 7], rows[1, 300] = 0x7FC0, 0x7F80
    slots = [c.table[1, 89 // 16] * 16 + 89 % 16, c.table[0, 199 // 16] * 16 + 199 % 16]
    K.kvo_paged_write(_dev(rows.view(np.int16), torch.int16), _dev(slots), c.pool, c.n_blocks, 16, fmt)
    c.refresh()
    q = O.bf16_bits(np.abs(np.random.default_rng(27).standard_normal((12, 8, 576))) + 0.1)
    out, lse = _attend(c, q, [0, 10, 12], [200, 90], SCALE)
    _check(c, q, [0, 10, 12], [200, 90], SCALE, 0, 0, out, lse, tokens=set(range(9)) | {10})
    got = O.bf16_values(out)
    assert np.isfinite(got[:9]).all() and np.isfinite(got[10]).all() and np.isnan(got[[9, 11]]).any((1, 2)).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lens,new,H", [([300, 900], [1, 2], 64), ([600] * 20, [20] * 20, 64)])
def test_captured_call_replayed_on_new_data(fmt, lens, new, H):
    """One call in a graph (short and long lists of tiles), replayed after lengths, table, queries and rows changed."""
    c = Cache(lens, 32, fmt, 28)
    g = np.random.default_rng(29)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(cu[-1])
    q, kv, table = torch.zeros(T, H, 576, dtype=torch.int16, device="cuda"), _dev(lens), _dev(c.table)
    out, lse = torch.zeros(T, H, 512, dtype=torch.int16, device="cuda"), torch.zeros(T, H, device="cuda")
    cud = _dev(cu)

    def call():
        K.kvo_paged_attend(c.pool, c.n_blocks, 32, fmt, table, kv, cud, q, SCALE, out, lse)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in range(3):
        bits = O.bf16_bits(g.standard_normal((T, H, 576)))
        kv_h = [max(1, n - 31 * k) for n in lens]
        q.copy_(_dev(bits.view(np.int16), torch.int16))
        kv.copy_(_dev(kv_h))
        graph.replay()
        torch.cuda.synchronize()
        _check(c, bits, cu, kv_h, SCALE, 0, 0, out.cpu().numpy().view(np.uint16), lse.cpu().numpy(),
               tokens={0, 1, T // 2, T - 1})


def test_empty_calls_and_streams():
    c = Cache([9], 8, Q4, 30)
    e = torch.empty(0, 576, dtype=torch.bfloat16, device="cuda")
    s = torch.empty(0, dtype=torch.int32, device="cuda")
    K.kvo_paged_write(e, s, c.pool, c.n_blocks, 8, Q4)
    K.kvo_paged_read(c.pool, c.n_blocks, 8, Q4, s, e)
    status = torch.full((1,), 5, dtype=torch.int32, device="cuda")
    K.kvo_paged_attend(c.pool, c.n_blocks, 8, Q4, _dev(c.table), _dev([9]), _dev([0, 0]),
                       torch.empty(0, 4, 576, dtype=torch.bfloat16, device="cuda"), SCALE,
                       torch.empty(0, 4, 512, dtype=torch.bfloat16, device="cuda"), status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    other = torch.cuda.Stream()
    q = torch.zeros(1, 4, 576, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(1, 4, 512, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(K.KvoError):  # a raw stream whose memory the allocator cannot order
        K.kvo_paged_attend(c.pool, c.n_blocks, 8, Q4, _dev(c.table), _dev([9]), _dev([0, 1]), q, SCALE, out,
                           stream=other.cuda_stream)
    for bad in (dict(out=out[:, :2].expand(1, 2, 512)), dict(queries=q.float()), dict(kv_lens=_dev([9]).long())):
        a = dict(block_table=_dev(c.table), kv_lens=_dev([9]), cu_tokens=_dev([0, 1]), queries=q, scale=SCALE, out=out)
        with pytest.raises(K.KvoError) as x:
            K.kvo_paged_attend(c.pool, c.n_blocks, 8, Q4, **{**a, **bad})
        assert x.value.code == K.KVO_EINVAL
    with pytest.raises(K.KvoError):
        K.kvo_paged_write(q[0], _dev([0, 1, 2, 3]), c.pool, c.n_blocks + 1, 8, Q4)  # the pool is smaller


def test_tokens_that_decrease_are_reported():
    # cu_tokens 0, 3, 0, 3 lists six tokens of three: nothing is computed, and the status says so
    c = Cache([9, 9, 9], 8, BF16, 22)
    q = torch.zeros(3, 4, 576, dtype=torch.int16, device="cuda")
    out = torch.full((3, 4, 512), 0x1234, dtype=torch.int16, device="cuda")
    for R, cu in ((3, [0, 3, 0, 3]), (3, [0, 0, 3, 2]), (300, [0, 3] * 150 + [0])):
        n = torch.full((R,), 9, dtype=torch.int32, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        table = _dev(np.resize(c.table, (R, c.M)))
        K.kvo_paged_attend(c.pool, c.n_blocks, 8, BF16, table, n, _dev(cu), q, SCALE, out, status=status)
        torch.cuda.synchronize()
        assert status.item() == 2 and bool((out == 0x1234).all())


_FIRST_PLAN = """
import torch
from top_cache_gb300 import kvo as K
R = %d
z = lambda n, t=torch.int32: torch.zeros(n, dtype=t, device="cuda")
ring, ends, slots, status = torch.arange(R, dtype=torch.int32, device="cuda"), z(2, torch.int64), z(R), z(R) + 5
ends[1] = R
K.kvo_paged_plan(z(R), z(R) + 1, 8, z(R).view(R, 1), ring, ends, ends, z(R), z(R), z(R + 1), slots, status)
torch.cuda.synchronize()
assert not status.any() and torch.equal(slots, 8 * ring), slots
"""


@pytest.mark.parametrize("R", [2443, 2444, 2457])
def test_plan_as_the_first_call_of_a_process(R):
    # the shared memory that a plan needs is asked for whatever its size is and whatever was called before
    subprocess.run([sys.executable, "-c", _FIRST_PLAN % R], cwd=ROOT, check=True, timeout=300)


def test_plans_of_two_threads():
    # both need more shared memory than a launch has by default, one of them more than the other
    failed = []

    def plans(R):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                z = lambda n, t=torch.int32: torch.zeros(n, dtype=t, device="cuda")  # noqa: E731
                a = (z(R), z(R), 8, z(R).view(R, 1), z(R), z(2, torch.int64), z(2, torch.int64), z(R), z(R), z(R + 1), z(1), z(R))
                for _ in range(300):
                    K.kvo_paged_plan(*a)
                torch.cuda.synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=plans, args=(R,)) for R in (4096, 2600)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


def test_plan_of_the_longest_slot_list():
    # 2^31 - 1 slots, 8 GB of them: the entries behind the new tokens are -1 to the last
    n = 2 ** 31 - 1
    z = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    slots = torch.full((n,), 7, dtype=torch.int32, device="cuda")
    ends = torch.tensor([0, 2], dtype=torch.int64, device="cuda")
    status = z(5, 5)
    K.kvo_paged_plan(z(0, 3), z(9, -1), 16, z(-1, 4).view(2, 1), z(3, 2, -1), ends, ends, z(0, 0), z(0, 0), z(0, 0, 0), slots, status)
    torch.cuda.synchronize()
    assert status.tolist() == [0, 0] and slots[:9].tolist() == list(range(48, 57)) and ends.tolist() == [1, 3]
    assert all(bool((part == -1).all()) for part in slots[9:].split(1 << 28))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("H", [4, 64])
def test_lengths_that_do_not_fit_are_reported(fmt, H):
    # a length past the block table, tokens past the queries or before them: nothing is computed, and the status says so
    c = Cache([40, 9, 17], 8, fmt, 33)
    full = c.M * 8
    n = 6
    q = torch.zeros(n, H, 576, dtype=torch.int16, device="cuda")
    for many in (1, 100):
        table = _dev(np.tile(c.table, (many, 1)))
        rest = 3 * (many - 1)
        for kv, cu, want in (([40, 9, 17], [0, 2, 4, 6], 0), ([full, 9, 17], [0, 2, 4, 6], 0), ([0, -1, 17], [0, 2, 2, 6], 0),
                             ([full + 1, 9, 17], [0, 2, 4, 6], 2), ([40, 9, 2 ** 31 - 1], [0, 2, 4, 6], 2),
                             ([40, 2 * full, 17], [0, 2, 2, 6], 2), ([40, 9, 17], [0, 2, 4, 7], 2),
                             ([40, 9, 17], [-1, 2, 4, 6], 2), ([40, 9, 17], [0, 9, 9, 9], 2)):
            out = torch.full((n, H, 512), 0x1234, dtype=torch.int16, device="cuda")
            status = torch.full((1,), 9, dtype=torch.int32, device="cuda")
            # (requests without tokens behind the three)
            K.kvo_paged_attend(c.pool, c.n_blocks, 8, fmt, table, _dev(kv + [0] * rest), _dev(cu + [cu[-1]] * rest), q, SCALE, out,
                               status=status)
            torch.cuda.synchronize()
            assert status.item() == want, (kv, cu)
            assert bool((out == 0x1234).all()) == (want != 0)


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_workspace_serves_smaller_calls(fmt):
    # fewer requests, tokens or heads: taller tiles of fewer requests need no more than the size says
    R, T, H = 40, 40, 16
    size = K.kvo_paged_attend_workspace_size(R, T, H)
    for r, t, h in ((1, 40, 16), (1, 1, 16), (40, 2, 16), (39, 40, 15), (7, 31, 3), (2, 5, 1), (40, 40, 16), (1, 0, 1)):
        assert 0 < K.kvo_paged_attend_workspace_size(r, t, h) <= size
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    for lens, new, h in (([3000], [40], 16), ([700, 20], [4, 1], 16), ([5000], [1], 16), ([90] * 40, [1] * 40, 16),
                         ([60] * 39, [1] * 39, 15), ([2000], [1], 1)):
        c = Cache(lens, 16, fmt, 31)
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        q = O.bf16_bits(np.random.default_rng(32).standard_normal((int(cu[-1]), h, 576)))
        out, lse = _attend(c, q, cu, lens, SCALE, workspace=ws)
        _check(c, q, cu, lens, SCALE, 0, 0, out, lse, tokens={0, 1, int(cu[-1]) - 1})


@pytest.mark.parametrize("block", [8, 40])
def test_bytes_of_the_4_bit_cache(block):
    """The written bytes are the definition's, and what the definition packs is read: neither call is the other's check."""
    n_blocks, n = 3, 2 * block
    bits = _special_rows(n, 34)
    codes, scales = O.quantize(bits)
    blocks = np.stack([O.pack_block(codes[i:i + block], scales[i:i + block]) for i in (0, block)])
    order = np.array([2, 0])  # block of the first and of the second half of the rows
    slots = (order[:, None] * block + np.arange(block)).reshape(-1)
    pool = _pool(n_blocks, block, Q4)
    K.kvo_paged_write(_dev(bits.view(np.int16), torch.int16), _dev(slots), pool, n_blocks, block, Q4)
    torch.cuda.synchronize()
    got = pool.cpu().numpy()
    assert (got[1] == 0xA5).all()
    nibbles = lambda b: np.stack([b & 15, b >> 4], -1)  # noqa: E731
    a, b = nibbles(got[order, :288 * block]), nibbles(blocks[:, :288 * block])
    assert np.array_equal(np.where(a == 8, 0, a), np.where(b == 8, 0, b))  # (a zero may have either sign)
    assert np.array_equal(got[order, 288 * block:], blocks[:, 288 * block:])
    # read back: bytes of every code and every scale, not only those that a write makes
    g = np.random.default_rng(35)
    codes, scales = g.integers(0, 16, (n, 576)).astype(np.uint8), g.integers(0, 128, (n, 36)).astype(np.uint8)
    pool = torch.full_like(pool, 0xA5)
    pool[torch.from_numpy(order).cuda()] = torch.from_numpy(
        np.stack([O.pack_block(codes[i:i + block], scales[i:i + block]) for i in (0, block)])).cuda()
    back = torch.full((n, 576), 0x1234, dtype=torch.int16, device="cuda")
    K.kvo_paged_read(pool, n_blocks, block, Q4, _dev(slots), back)
    torch.cuda.synchronize()
    got = O.bf16_values(back.cpu().numpy().view(np.uint16))
    assert np.array_equal(got, O.dequantize(codes, scales), equal_nan=True)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("H", [8, 64])
def test_a_step_whose_tokens_pass_the_slots(fmt, H):
    # the plan refuses the requests whose tokens pass the slots and counts their tokens all the same; the attention over
    # as many query tokens computes the others, and gives nothing to those tokens of refused ones that it has
    B, lens, new, T = 8, [30, 5, 20, 17], np.array([2, 9, 0, 3], np.int32), 4
    c = Cache(lens, B, fmt, 36)
    got = _run_plan(lens, new, B, c.table, np.array([-1], np.int32), np.array([0, 0]), T, 0, 0)  # (no block is needed)
    assert got["status"].tolist() == [0, -3, 0, -3] and got["cu"].tolist() == [0, 2, 11, 11, 14]
    last = int(c.table[0, 3]) * B
    assert got["kv_lens"].tolist() == [32, 0, 20, 0] and got["slots"].tolist() == [last + 6, last + 7, -1, -1]
    rows = O.bf16_bits(np.random.default_rng(37).standard_normal((T, 576)))
    K.kvo_paged_write(_dev(rows.view(np.int16), torch.int16), _dev(got["slots"]), c.pool, c.n_blocks, B, fmt)
    torch.cuda.synchronize()
    c.refresh()
    q = O.bf16_bits(np.random.default_rng(38).standard_normal((T, H, 576)))
    out, lse = _attend(c, q, got["cu"], got["kv_lens"], SCALE)
    _check(c, q, [0, 2], [32], SCALE, 0, 0, out, lse)
    assert np.isneginf(lse[2:]).all() and not out[2:].any()
