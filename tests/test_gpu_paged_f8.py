"""The 8-bit paged cache against its plain definitions in 64 bits: rows (equal), attention (tolerances: paged_harness)."""
import numpy as np
import pytest
import torch

from oracle import paged as O
from tests import test_gpu_paged as P
from tests.paged_harness import F8, SCALE, Cache, attend, check, dev, run
from top_cache_gb300 import kvo as K

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from top_cache_gb300 import build
    build.build()
    yield


# ---- rows -----------------------------------------------------------------------------------

def _rows(n, seed):
    bits = P._special_rows(n, seed)
    if n > 8:
        bits[5] = O.bf16_bits(np.resize([448, 17, 19, 2.0 ** -10, -3 * 2.0 ** -10, 5 * 2.0 ** -10, 2.0 ** -9, -0.0], 576))  # ties
        bits[6] = O.bf16_bits(np.resize([450.0, -2.0 ** -30], 576))    # just past 448
        bits[7] = O.bf16_bits(np.resize([2.0 ** -40, -2.0 ** -41, 2.0 ** -42], 576))  # the least scale
        bits[8] = O.bf16_bits(np.resize([448 * 2.0 ** 32, 450 * 2.0 ** 32, -3e38], 576))  # the greatest
    return bits


@pytest.mark.parametrize("n,block", [(1, 8), (7, 24), (16, 16), (129, 64), (1000, 128), (4097, 8)])
def test_rows_written_and_read(n, block):
    g = np.random.default_rng(n)
    n_blocks = -(-n // block) + 2
    bits = _rows(n, n)
    slots = g.permutation(n_blocks * block)[:n].astype(np.int32)
    skip = g.random(n) < 0.1
    slots[skip] = g.choice([-1, -7, n_blocks * block, 2 ** 31 - 1], int(skip.sum()))
    pool = P._pool(n_blocks, block, F8)
    want = pool.cpu().numpy()
    K.kvo_paged_write(dev(bits.view(np.int16), torch.int16), dev(slots), pool, n_blocks, block, F8)
    back = torch.full((n, 576), 0x1234, dtype=torch.int16, device="cuda")
    K.kvo_paged_read(pool, n_blocks, block, F8, dev(slots), back)
    torch.cuda.synchronize()
    got = back.cpu().numpy().view(np.uint16)
    assert (got[skip] == 0x1234).all()
    codes, scales = O.quantize8(bits)
    at = slots[~skip]
    want_c, want_s = want[:, :576 * block].reshape(-1, 576).copy(), want[:, 576 * block:].copy().view(np.uint32).reshape(-1)
    want_c[at], want_s[at] = codes[~skip], scales[~skip]
    after = pool.cpu().numpy()
    got_s = after[:, 576 * block:].copy().view(np.uint32).reshape(-1)
    nan = lambda s: np.isnan(s.view(np.float32))  # noqa: E731  (any NaN serves)
    assert np.array_equal(after[:, :576 * block].reshape(-1, 576), want_c)
    assert np.array_equal(nan(got_s), nan(want_s)) and np.array_equal(got_s[~nan(got_s)], want_s[~nan(want_s)])
    assert np.array_equal(O.bf16_values(got[~skip]), O.dequantize8(codes, scales)[~skip], equal_nan=True)


@pytest.mark.parametrize("block", [8, 40])
def test_every_byte_is_read(block):
    # what the definition packs, not only what a write makes: any code, and scales that are none
    g = np.random.default_rng(block)
    n = 2 * block
    codes = g.integers(0, 256, (n, 576)).astype(np.uint8)
    scales = (2.0 ** g.integers(-32, 33, n)).astype(np.float32).view(np.uint32)
    scales[1:9] = [0, 0x3F800001, 0xBF800000, 0x7F800000, 0xFFFFFFFF, 0x50000000, 0x2F000000, 0x2F800000]
    pool = P._pool(3, block, F8)
    order = [2, 0]
    pool[order] = torch.from_numpy(np.stack([O.pack_block8(codes[i:i + block], scales[i:i + block]) for i in (0, block)])).cuda()
    slots = (np.array(order)[:, None] * block + np.arange(block)).reshape(-1)
    back = torch.full((n, 576), 0x1234, dtype=torch.int16, device="cuda")
    K.kvo_paged_read(pool, 3, block, F8, dev(slots), back)
    torch.cuda.synchronize()
    assert np.array_equal(O.bf16_values(back.cpu().numpy().view(np.uint16)), O.dequantize8(codes, scales), equal_nan=True)


# ---- attention ------------------------------------------------------------------------------

@pytest.mark.parametrize("H", [1, 16, 17, 32, 40, 64, 128])
def test_one_token(H):
    run(F8, [1], [1], H, 8)


@pytest.mark.parametrize("H,lens", [(16, [127]), (16, [128]), (16, [129]), (5, [300, 1, 77]), (32, [1000]), (24, [257, 640, 3]),
                                    (64, [500, 128]), (128, [700]), (100, [390])])
def test_decode(H, lens):
    run(F8, lens, [1] * len(lens), H, 16, seed=H)


@pytest.mark.parametrize("block", [8, 24, 40, 64, 128, 192])
def test_block_sizes(block):
    for H in (8, 24, 64):
        run(F8, [block - 1, block, 3 * block + 5], [1, 2, 1], H, block, seed=block)


@pytest.mark.parametrize("H,new,lens", [(16, [4, 4], [260, 131]), (3, [5, 1, 7], [300, 9, 7]), (20, [33], [161]), (128, [4], [260]),
                                        (1, [200], [450]), (7, [64, 3], [64, 130]), (16, [0, 2, 0], [50, 200, 0])])
def test_several_positions(H, new, lens):
    run(F8, lens, new, H, 16, seed=len(lens) + H, pad=3)


@pytest.mark.parametrize("H,new,lens,window,sinks", [
    (16, [1], [1000], 1, 0), (16, [1], [1000], 128, 0), (16, [1, 1], [1000, 90], 100, 4), (8, [9, 4], [900, 300], 40, 1),
    (3, [150], [700], 130, 70), (64, [3], [2000], 129, 128), (128, [2], [800], 300, 200), (16, [5], [400], 4000, 4),
    (16, [3], [1500], 64, 5000), (2, [300], [300], 17, 2)])
def test_window_and_sinks(H, new, lens, window, sinks):
    run(F8, lens, new, H, 24, window, sinks, seed=window)


@pytest.mark.parametrize("scale,q_scale", [(0.0, 1.0), (-0.1, 1.0), (3.0, 1.0), (SCALE, 1e4), (1e-6, 1e20), (SCALE, 1e-30)])
@pytest.mark.parametrize("H", [16, 30, 64])
def test_scales(H, scale, q_scale):
    # a large scale moves the running maximum by far more than 2^2 from block to block (O^T is rescaled in TMEM)
    run(F8, [600, 129], [1, 3], H, 16, seed=5, scale=scale, q_scale=q_scale)


@pytest.mark.parametrize("H", [8, 16, 32])
def test_growing_scores(H):
    # each block's rows larger than the last one's: a new maximum in every block
    c = Cache([900], 16, F8, 3)
    g = np.random.default_rng(4)
    c.set_rows(0, np.arange(900), O.bf16_bits(g.standard_normal((900, 576)) * (1 + np.arange(900) / 30.0)[:, None]))
    q = O.bf16_bits(g.standard_normal((2, H, 576)))
    out, lse = attend(c, q, [0, 2], [900])
    check(c, q, [0, 2], [900], out, lse)


@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("low,high", [(-6, 6), (-31, 20), (-45, -25)])
def test_rows_of_different_size(H, low, high):
    # row scales over many powers of two: what a row adds to the output is its weight times its scale
    c = Cache([700, 40], 16, F8, 41)
    g = np.random.default_rng(42)
    size = 2.0 ** g.integers(low, high + 1, 700)
    size[[3, 400]] = 0.0
    c.set_rows(0, np.arange(700), O.bf16_bits(g.standard_normal((700, 576)) * size[:, None]))
    q = O.bf16_bits(g.standard_normal((2, H, 576)))
    # (scores stay of the order of one)
    scale = SCALE * 2.0 ** -min(max(high, 0), 31)
    out, lse = attend(c, q, [0, 1, 2], [700, 40], scale)
    check(c, q, [0, 1, 2], [700, 40], out, lse, scale)


@pytest.mark.parametrize("H", [16, 64])
def test_one_token_has_nearly_all_the_weight(H):
    # and 20,000 others share what is left: they may not vanish
    c = Cache([20001], 64, F8, 43)
    g = np.random.default_rng(44)
    bits = O.bf16_bits(0.01 * g.standard_normal((20001, 576)) + 1.0)
    bits[7] = O.bf16_bits(np.full(576, 3.0))
    c.set_rows(0, np.arange(20001), bits)
    q = O.bf16_bits(np.full((1, H, 576), 0.05))
    for scale in (0.1, 0.2):  # the others 2^-8 to 2^-17 of the largest
        out, lse = attend(c, q, [0, 1], [20001], scale)
        check(c, q, [0, 1], [20001], out, lse, scale)


def test_queries_with_a_large_element():
    c = Cache([500], 16, F8, 45)
    g = np.random.default_rng(46)
    x = g.standard_normal((4, 16, 576))
    x[0, :, 5], x[1, :, 570], x[2, :, :300] = 500.0, -2000.0, 2.0 ** -12
    x[3] = 0.0
    q = O.bf16_bits(x)
    out, lse = attend(c, q, [0, 4], [500], SCALE / 8)
    check(c, q, [0, 4], [500], out, lse, SCALE / 8)


def test_queries_that_are_not_finite():
    c = Cache([300], 16, F8, 47)
    x = np.random.default_rng(48).standard_normal((1, 20, 576))
    q = O.bf16_bits(x)
    q[0, 3, 9], q[0, 7, 575] = 0x7FC0, 0xFF80
    out, lse = attend(c, q, [0, 1], [300])
    bad = np.isnan(O.bf16_values(out)).all(-1)[0]
    assert np.flatnonzero(bad).tolist() == [3, 7] and np.isnan(lse[0, [3, 7]]).all()
    keep = [h for h in range(20) if h not in (3, 7)]
    check(c, q[:, keep], [0, 1], [300], out[:, keep], lse[:, keep])


def test_positions_that_see_nothing():
    # more query tokens than cached ones (the first positions are negative), an empty cache, a request without queries
    c = Cache([3, 0, 40], 8, F8, 6)
    q = O.bf16_bits(np.random.default_rng(7).standard_normal((7, 16, 576)))
    cu = [0, 5, 7, 7]
    out, lse = attend(c, q, cu, [3, 0, 40])
    check(c, q, cu, [3, 0, 40], out, lse)
    assert np.isneginf(lse[[0, 1, 5, 6]]).all() and np.isfinite(lse[2:5]).all()


def test_unmapped_blocks_are_not_seen():
    c = Cache([500, 200], 16, F8, 8)
    c.table[0, [0, 7, 8, 31]] = [-1, -5, c.n_blocks, 2 ** 31 - 1]
    c.table[1, :] = -1
    q = O.bf16_bits(np.random.default_rng(9).standard_normal((4, 20, 576)))
    out, lse = attend(c, q, [0, 2, 4], [500, 200])
    check(c, q, [0, 2, 4], [500, 200], out, lse)
    assert np.isneginf(lse[2:]).all()


@pytest.mark.parametrize("H", [4, 16, 128])
def test_what_is_not_finite_stays_with_those_that_see_it(H):
    # rows that are not finite (their scale is NaN), and codes that are NaN under a scale that is none or a good one
    c = Cache([400], 16, F8, 10)
    rows = O.bf16_bits(np.random.default_rng(11).standard_normal((2, 576)))
    rows[0, 5], rows[1, 511] = 0x7FC0, 0x7F80
    c.set_rows(0, [399, 397], rows)
    blk, at = int(c.table[0, 299 // 16]), 299 % 16
    c.pool[blk, 576 * at + 100] = 0xFF  # a code alone, in the value part
    blk = int(c.table[0, 298 // 16])
    c.pool[blk, 576 * 16 + 4 * (298 % 16):576 * 16 + 4 * (298 % 16) + 4] = 0xFF
    c.refresh()
    q = O.bf16_bits(np.abs(np.random.default_rng(12).standard_normal((6, H, 576))) + 0.1)
    for window in (0, 100, 20):
        out, lse = attend(c, q, [0, 6], [400], window=window)
        check_nan = np.isnan(O.bf16_values(out)).any((1, 2))
        # positions 394..399; 298 and 299 are in a window of 100 of 394..397 and 394..398, in none of 20
        want = [p >= 397 or window == 0 or p - window < 299 for p in range(394, 400)]
        assert check_nan.tolist() == want
        fine = [i for i in range(6) if not want[i]]
        check(c, q, [0, 6], [400], out, lse, window=window, tokens=set(fine))


def test_not_finite_beside_a_half_empty_tile():
    # tiles of 64 rows, the last request's only 16 of them filled: the other half's rows lie past the queries
    c = Cache([200, 90], 16, F8, 25)
    rows = O.bf16_bits(np.random.default_rng(26).standard_normal((2, 576)))
    rows[0, 7], rows[1, 300] = 0x7FC0, 0x7F80
    c.set_rows(1, [89], rows[:1])
    c.set_rows(0, [199], rows[1:])
    q = O.bf16_bits(np.abs(np.random.default_rng(27).standard_normal((12, 8, 576))) + 0.1)
    out, lse = attend(c, q, [0, 10, 12], [200, 90])
    check(c, q, [0, 10, 12], [200, 90], out, lse, tokens=set(range(9)) | {10})
    got = O.bf16_values(out)
    assert np.isfinite(got[:9]).all() and np.isfinite(got[10]).all() and np.isnan(got[[9, 11]]).any((1, 2)).all()


def test_split_and_joined():
    # one request over every CTA, and tiles of other requests between: partial results of many CTAs are joined
    run(F8, [30011], [1], 16, 64, seed=13)
    run(F8, [9000, 5, 3001, 0, 700], [1, 1, 2, 0, 1], 64, 64, seed=14)
    run(F8, [5000], [2], 128, 64, seed=15)


def test_many_tiles():
    # more tiles than are listed: whole tiles per CTA; sampled tokens
    run(F8, [700, 5, 200, 1300, 17], [700, 0, 1, 900, 17], 90, 64, 100, 3, seed=16,
        tokens={0, 1, 350, 699, 700, 701, 1100, 1600, 1601, 1617})


def test_many_requests():
    g = np.random.default_rng(17)
    lens = g.integers(0, 40, 1500).tolist()
    run(F8, lens, [min(n, 1) for n in lens], 2, 8, seed=17, tokens=set(range(0, 1500, 37)))
    run(F8, [9] * 4096, [1] * 4096, 1, 16, seed=18, tokens=set(range(0, 4096, 111)))


@pytest.mark.parametrize("H", [16, 64])
def test_same_bits_again_and_on_another_stream(H):
    c = Cache([7000, 300], 64, F8, 19)
    q = O.bf16_bits(np.random.default_rng(20).standard_normal((3, H, 576)))
    a = attend(c, q, [0, 1, 3], [7000, 300])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, s):
        b = attend(c, q, [0, 1, 3], [7000, 300], stream=stream)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1].view(np.uint32), b[1].view(np.uint32))
    # two calls in flight, each with its own workspace
    outs = [torch.zeros(3, H, 512, dtype=torch.int16, device="cuda") for _ in range(2)]
    args = (c.pool, c.n_blocks, 64, F8, dev(c.table), dev([7000, 300]), dev([0, 1, 3]), dev(q.view(np.int16), torch.int16), SCALE)
    torch.cuda.synchronize()
    for o, st in zip(outs, (s, torch.cuda.Stream())):
        K.kvo_paged_attend(*args, o, stream=st)
    torch.cuda.synchronize()
    assert all(np.array_equal(o.cpu().numpy().view(np.uint16), a[0]) for o in outs)


@pytest.mark.parametrize("lens,new,H", [([300, 900], [1, 2], 64), ([600] * 20, [20] * 20, 64), ([900, 77], [1, 1], 16)])
def test_captured_call_replayed_on_new_data(lens, new, H):
    """One call in a graph (short and long lists of tiles), replayed after lengths and queries changed."""
    c = Cache(lens, 32, F8, 28)
    g = np.random.default_rng(29)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(cu[-1])
    q, kv, table, cud = torch.zeros(T, H, 576, dtype=torch.int16, device="cuda"), dev(lens), dev(c.table), dev(cu)
    out, lse = torch.zeros(T, H, 512, dtype=torch.int16, device="cuda"), torch.zeros(T, H, device="cuda")

    def call():
        K.kvo_paged_attend(c.pool, c.n_blocks, 32, F8, table, kv, cud, q, SCALE, out, lse)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in range(3):
        bits = O.bf16_bits(g.standard_normal((T, H, 576)))
        kv_h = [max(1, n - 31 * k) for n in lens]
        q.copy_(dev(bits.view(np.int16), torch.int16))
        kv.copy_(dev(kv_h))
        graph.replay()
        torch.cuda.synchronize()
        check(c, bits, cu, kv_h, out.cpu().numpy().view(np.uint16), lse.cpu().numpy(), tokens={0, 1, T // 2, T - 1})


def test_rows_past_32_bit_offsets():
    # a pool of more than 4 GB: blocks at its far end
    B = 4096
    n_blocks = (5 << 30) // K.kvo_paged_block_bytes(F8, B)
    pool = torch.empty(n_blocks, K.kvo_paged_block_bytes(F8, B), dtype=torch.uint8, device="cuda")
    L = 300
    bits = O.bf16_bits(np.random.default_rng(23).standard_normal((L, 576)))
    slots = (n_blocks - 1) * B + np.arange(L)
    K.kvo_paged_write(dev(bits.view(np.int16), torch.int16), dev(slots), pool, n_blocks, B, F8)
    back = torch.zeros(L, 576, dtype=torch.int16, device="cuda")
    K.kvo_paged_read(pool, n_blocks, B, F8, dev(slots), back)
    torch.cuda.synchronize()
    codes, scales = O.quantize8(bits)
    rows = O.dequantize8(codes, scales)
    assert np.array_equal(O.bf16_values(back.cpu().numpy().view(np.uint16)), rows)

    class C:  # as a Cache whose one request begins at the far block; the check sees its rows alone
        def __init__(self, block0):
            self.pool, self.n_blocks, self.block, self.fmt = pool, n_blocks, B, F8
            self.table, self.exps = np.array([[block0, 7]], np.int32), (scales >> 23).astype(np.int64) - 127
            self.rows_of = lambda r: lambda t: (rows[t], np.ones(len(t), bool))

    for H in (16, 40):
        q = O.bf16_bits(np.random.default_rng(24).standard_normal((1, H, 576)))
        out, lse = attend(C(n_blocks - 1), q, [0, 1], [L])
        check(C(0), q, [0, 1], [L], out, lse)


@pytest.mark.parametrize("H", [4, 64])
def test_lengths_that_do_not_fit_are_reported(H):
    c = Cache([40, 9, 17], 8, F8, 33)
    full = c.M * 8
    q = np.zeros((6, H, 576), np.uint16)
    for kv, cu in (([full + 1, 9, 17], [0, 2, 4, 6]), ([40, 9, 17], [0, 2, 4, 7]), ([40, 9, 17], [0, 9, 9, 9])):
        out, _ = attend(c, q, cu, kv, want=2)
        assert (out == 0x1234).all()


def test_a_workspace_serves_smaller_calls():
    size = K.kvo_paged_attend_workspace_size(40, 40, 16)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    for lens, new, h in (([3000], [40], 16), ([700, 20], [4, 1], 16), ([5000], [1], 16), ([90] * 40, [1] * 40, 16), ([2000], [1], 1)):
        c = Cache(lens, 16, F8, 31)
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        q = O.bf16_bits(np.random.default_rng(32).standard_normal((int(cu[-1]), h, 576)))
        out, lse = attend(c, q, cu, lens, workspace=ws)
        check(c, q, cu, lens, out, lse, tokens={0, 1, int(cu[-1]) - 1})


def test_empty_calls():
    c = Cache([9], 8, F8, 30)
    e, s = torch.empty(0, 576, dtype=torch.bfloat16, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    K.kvo_paged_write(e, s, c.pool, c.n_blocks, 8, F8)
    K.kvo_paged_read(c.pool, c.n_blocks, 8, F8, s, e)
    out, lse = attend(c, np.zeros((0, 4, 576), np.uint16), [0, 0], [9])
    assert out.shape == (0, 4, 512)
