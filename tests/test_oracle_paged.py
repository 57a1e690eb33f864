"""Pins of the paged cache's oracle: hand-made plans, exhaustive 4-bit values, small attentions."""
import numpy as np
import pytest

from oracle import paged as O


def test_plan_takes_blocks_in_request_order():
    table = np.full((3, 4), -1, np.int32)
    table[0, 0], table[2, :2] = 9, (7, 8)
    ring = np.array([5, 4, 3, 2, 1, 0, -1, -1], np.int32)
    r = O.plan([6, 0, 16], [3, 0, 1], 8, table, ring, [0, 6], 6)
    assert r["table"].tolist() == [[9, 5, -1, -1], [-1] * 4, [7, 8, 4, -1]]
    assert r["slots"].tolist() == [9 * 8 + 6, 9 * 8 + 7, 5 * 8, 4 * 8, -1, -1]
    assert r["cu"].tolist() == [0, 3, 3, 4] and r["bounds"].tolist() == [2, 6]
    assert r["lengths"].tolist() == [9, 0, 17] and r["status"].tolist() == [0, 0, 0]


def test_plan_refusals_change_nothing():
    table = np.full((4, 2), -1, np.int32)
    ring = np.array([3, 2], np.int32)
    # 16 tokens need both blocks; the next has none left, but one that needs none is served; 17 pass the table
    r = O.plan([0, 0, 4, 0], [16, 1, 1, 17], 8, table, ring, [0, 2], 64)
    assert r["status"].tolist() == [O.OK, O.ECAPACITY, O.OK, O.ERANGE]
    assert r["lengths"].tolist() == [16, 0, 5, 0] and r["kv_lens"].tolist() == [16, 0, 5, 0]
    assert r["slots"][16:19].tolist() == [-1, -1, -1]  # refused, a table without the entry, refused
    # the slot list is too short for the second request only
    r = O.plan([0, 0, 0], [3, 9, 0], 8, np.full((3, 2), -1, np.int32), np.arange(6, dtype=np.int32), [0, 6], 8)
    assert r["status"].tolist() == [O.OK, O.ERANGE, O.OK]


def test_plan_gives_back_what_no_position_sees():
    # blocks of 8, window 10, 3 sinks: at length 30 the next position sees tokens 21.. and 0..2
    table = np.arange(8, dtype=np.int32)[None, :]
    r = O.plan([20], [10], 8, np.where(np.arange(8) < 3, table, -1), np.array([50, 51, 52, -1], np.int32), [0, 3], 16,
               window=10, sinks=3)
    assert r["table"][0, :5].tolist() == [0, 1, 2, 50, -1]
    # length 20 saw 11..: block 1 (8..15) was still needed; length 30 sees 21..: block 1 goes, block 2 (16..23) stays
    assert r["ring"][3] == 1 and r["bounds"].tolist() == [1, 4]
    # ending gives back the sinks' block and the live ones, not the block that went before
    r = O.plan([30], [-1], 8, r["table"], r["ring"], r["bounds"], 16, window=10, sinks=3)
    assert [int(r["ring"][i % 4]) for i in range(4, 7)] == [0, 2, 50] and r["lengths"][0] == 0


def test_e2m1_and_e4m3_values():
    assert O._E4M3[1] == 2.0 ** -9 and O._E4M3[126] == 448.0 and O._E4M3[8] == 2.0 ** -6
    x = np.array([0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.1, 7.0])
    assert O._E2M1[O._nearest(x, O._E2M1)].tolist() == [0, 0.5, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0, 6.0]


def test_quantize_round_trip():
    x = np.zeros((2, 576), np.float32)
    x[0, :16] = [6, -6, 3, 0.5, 0, -0.5, 4, 2, 1.5, 1, -1, -4, -3, -2, -1.5, 0.2]  # scale 1: values of the grid, and 0.2 -> 0
    x[1, 20] = 3e38                                                             # saturates at 448 * 6
    c, s = O.quantize(O.bf16_bits(x))
    v = O.dequantize(c, s)
    want = x[0, :16].copy()
    want[15] = 0.0
    assert np.array_equal(v[0, :16], want) and s[0, 0] == 56  # 56: 1.0
    assert v[1, 20] == 2688.0 and not v[1, :16].any()
    x[1, 575] = np.inf
    assert np.isnan(O.dequantize(*O.quantize(O.bf16_bits(x)))[1, 560:]).all()


@pytest.mark.parametrize("p,window,sinks,want", [(-1, 0, 0, []), (3, 0, 0, [0, 1, 2, 3]), (5, 2, 0, [4, 5]),
                                                 (5, 2, 1, [0, 4, 5]), (1, 4, 9, [0, 1]), (0, 1, 0, [0])])
def test_visible(p, window, sinks, want):
    assert O.visible(p, window, sinks).tolist() == want


def test_attend_is_the_weighted_mean():
    rows = np.zeros((2, 576))
    rows[0, 0], rows[1, 1] = 1.0, 2.0
    q = np.zeros((1, 1, 576))
    q[0, 0, 0] = np.log(3.0)
    out, lse, *_ = O.attend(lambda t: (rows[t], np.ones(len(t), bool)), q, [1], 1.0)
    assert np.allclose(out[0, 0, :2], [0.75, 0.5]) and np.allclose(lse, np.log(4.0))
