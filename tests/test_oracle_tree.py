"""Pins of the oracle of 8-bit rows and draft trees: hand-made rows, trees, paths and commits (no GPU)."""
import numpy as np
import pytest

from oracle import paged as O


def test_8_bit_rows():
    x = np.zeros((6, 576), np.float32)
    x[0, :5] = [448, -448, 1, 0.0156, 2.0 ** -9]     # scale 1: 0.0156 is below the least normal code, 2^-6
    x[1, :2] = [450, 18]                             # 2: 225 lies between 224 and 240
    x[2, 0] = 3e38                                   # saturates at 448 2^32
    x[3, 0] = 2.0 ** -50                             # below the least code of the least scale
    x[5, 7] = np.inf
    c, s = O.quantize8(O.bf16_bits(x))
    v = O.dequantize8(c, s)
    assert s[:5].view(np.float32).tolist() == [1.0, 2.0, 2.0 ** 32, 2.0 ** -32, 2.0 ** -32]
    assert v[0, :5].tolist() == [448, -448, 1, 0.015625, 2.0 ** -9]
    assert v[1, :2].tolist() == [448.0, 18.0] and v[2, 0] == 448 * 2.0 ** 32 and v[3, 0] == 0 and not v[4].any()
    assert np.isnan(v[5]).all()


def test_8_bit_ties_go_to_the_even_code():
    x = np.zeros((1, 576), np.float32)
    x[0, :6] = [448, 17, 19, 2.0 ** -10, 3 * 2.0 ** -10, 5 * 2.0 ** -10]  # steps of 2 and of 2^-9
    v = O.dequantize8(*O.quantize8(O.bf16_bits(x)))
    assert v[0, :6].tolist() == [448, 16, 20, 0, 2.0 ** -8, 2.0 ** -8]


@pytest.mark.parametrize("bits,fine", [(0x3F800000, True), (0x2F800000, True), (0x4F800000, True), (0x2F000000, False),
                                       (0x50000000, False), (0x3F800001, False), (0xBF800000, False), (0, False),
                                       (0x7F800000, False), (0xFFFFFFFF, False)])
def test_scales_that_are_none(bits, fine):
    assert np.isfinite(O.dequantize8(np.full((1, 576), 56, np.uint8), np.array([bits], np.uint32))).all() == fine


def test_pack_block8():
    b = O.pack_block8(np.arange(16 * 576).astype(np.uint8).reshape(16, 576), np.arange(16, dtype=np.uint32))
    assert len(b) == 16 * 580 and b[577] == 577 % 256 and b[16 * 576:].view(np.uint32).tolist() == list(range(16))


def test_ancestors_and_words():
    a = O.ancestors([-1, 0, 0, 1, 9, 3, -5])
    assert [np.flatnonzero(r).tolist() for r in a] == [[0], [0, 1], [0, 2], [0, 1, 3], [4], [0, 1, 3, 5], [6]]
    assert O.mask_words(a, 2).tolist() == [[1, 0], [3, 0], [5, 0], [11, 0], [16, 0], [43, 0], [64, 0]]
    chain = O.mask_words(O.ancestors(list(range(-1, 33))), 2)
    assert chain[31].tolist() == [-1, 0] and chain[33].tolist() == [-1, 3]


def test_accept():
    parents, drafted = [-1, 0, 0, 1, 2, 4], [7, 10, 11, 12, 13, 14]
    assert O.accept(parents, drafted, [11, 0, 13, 0, 99, 0]) == [0, 2, 4]
    assert O.accept(parents, drafted, [10, 12, 13, 0, 99, 0]) == [0, 1, 3]
    assert O.accept(parents, drafted, [5, 12, 13, 0, 14, 0]) == [0]
    # two children with the same token: the deeper path; as deep: the first
    assert O.accept([-1, 0, 0, 2], [0, 3, 3, 4], [3, 9, 4, 9]) == [0, 2, 3]
    assert O.accept([-1, 0, 0], [0, 3, 3], [3, 9, 9]) == [0, 1]
    assert O.accept([], [], []) == [] and O.accept([-1, 1, 5], [0, 0, 0], [0, 0, 0]) == [0]


def test_commit_gives_blocks_back():
    table = np.arange(24, dtype=np.int32).reshape(3, 8)
    ring = np.full(9, -1, np.int32)
    # 21 of 30 tokens stay: block 3 (of 8 rows: 24..31) goes
    L, ring2, b = O.commit([30, 5, 40], [30, 0, 40], [10, 3, 0], [1, 0, 0], 8, table, ring, [0, 7])
    assert L.tolist() == [21, 5, 40] and b.tolist() == [0, 8] and ring2[7] == 3
    L, ring2, b = O.commit([30], [30], [10], [1], 8, table, ring, [0, 7], window=5)
    # at length 20 block 1 (8..15) was the last hidden one (16 and later are seen); at 21 none more
    assert b.tolist() == [0, 8] and ring2[7] == 3
    L, ring2, b = O.commit([30], [30], [10], [9], 8, table, ring, [0, 7], window=5)
    assert L[0] == 29 and b.tolist() == [0, 8] and ring2[7] == 2  # 29 sees 25..: block 2 (16..23) goes, none behind
    L, ring2, b = O.commit([30], [30], [10], [9], 8, table, ring, [0, 7], window=5, sinks=17)
    assert b.tolist() == [0, 7]


def test_tree_seen():
    m = O.ancestors([-1, 0, 0, 1])
    s = O.tree_seen(7, 4, m, [0, 1, 1, 2], range(7))
    assert [np.flatnonzero(r).tolist() for r in s] == [[0, 1, 2, 3], [0, 1, 2, 3, 4], [0, 1, 2, 3, 5], [0, 1, 2, 3, 4, 6]]
    # a window of 2: nodes at positions 3, 4, 4, 5; the last sees itself and its parent (4), not the root (3)
    s = O.tree_seen(7, 4, m, [0, 1, 1, 2], range(7), window=2, sinks=1)
    assert [np.flatnonzero(r).tolist() for r in s] == [[0, 2, 3], [0, 3, 4], [0, 3, 5], [0, 4, 6]]
    assert not O.tree_seen(3, 4, m, [0, 1, 1, 2], range(3)).any()


def test_attend_seen_is_the_weighted_mean():
    rows = np.zeros((3, 576))
    rows[0, 0], rows[1, 1], rows[2, 0] = 1.0, 2.0, 50.0
    q = np.zeros((1, 1, 576))
    q[0, 0, 0] = np.log(3.0)
    out, lse, mag, dot, n, w = O.attend_seen(rows, q, np.array([[True, True, False]]), 1.0)
    assert np.allclose(out[0, 0, :2], [0.75, 0.5]) and np.allclose(lse, np.log(4.0)) and np.allclose(w, [0.75, 0.25, 0])
