"""Draft trees over the paged cache against their plain definitions: masks, paths, commits and moves (equal), attention in
every format (tolerances: paged_harness), and a loop of draft steps in one graph."""
import numpy as np
import pytest
import torch

from oracle import paged as O
from tests import test_gpu_paged as P
from tests.paged_harness import BF16, F8, Q4, SCALE, Cache, attend, check, dev, forest, pool_rows, random_tree, run
from top_cache_gb300 import kvo as K

pytestmark = pytest.mark.gpu
FORMATS = [pytest.param(BF16, id="bf16"), pytest.param(F8, id="f8"), pytest.param(Q4, id="q4")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from top_cache_gb300 import build
    build.build()
    yield


def _cu(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


# ---- masks, paths -------------------------------------------------------------------------------

def _trees(seed):
    g = np.random.default_rng(seed)
    out = [[], [-1], [-1, 0], list(range(-1, 70)), [-1] + [0] * 99, random_tree(g, 33), random_tree(g, 257), [-1, 5, -7, 2, 4, 1, 0, 2]]
    out += [random_tree(g, int(n)) for n in g.integers(0, 90, 6)]
    return out


@pytest.mark.parametrize("words", [9, 32])
def test_masks(words):
    trees = _trees(1) + ([list(range(-1, 1023)), random_tree(np.random.default_rng(2), 1024), [-1] + [0] * 1000] if words == 32 else [])
    cu = _cu([len(t) for t in trees])
    T, pad = int(cu[-1]), 3
    parents = np.concatenate([np.array(t, np.int64) for t in trees] + [np.full(pad, -1)])
    masks = torch.full((T + pad, words), 0x1234, dtype=torch.int32, device="cuda")
    depths, status = torch.full((T + pad,), 77, dtype=torch.int32, device="cuda"), dev([9])
    K.kvo_tree_masks(dev(parents), dev(cu), masks, depths, status)
    again = torch.zeros_like(masks)
    K.kvo_tree_masks(dev(parents), dev(cu), again)
    torch.cuda.synchronize()
    want, words_want, depths_want = forest([t for t in trees], words)
    assert status.item() == 0
    assert np.array_equal(masks.cpu().numpy()[:T], words_want) and np.array_equal(depths.cpu().numpy()[:T], depths_want)
    assert bool((masks[T:] == 0x1234).all()) and bool((depths[T:] == 77).all()) and torch.equal(again[:T], masks[:T])


def test_masks_that_do_not_fit():
    # 33 nodes in one word: reported, and none of its nodes sees one; the others are right.  Tokens outside: none written
    parents = list(range(-1, 32)) + [-1, 0]
    masks, depths, status = torch.full((35, 1), 7, dtype=torch.int32, device="cuda"), dev(np.full(35, 7)), dev([9])
    K.kvo_tree_masks(dev(parents), dev([0, 33, 35]), masks, depths, status)
    torch.cuda.synchronize()
    assert status.item() == 2 and masks[:, 0].tolist() == [0] * 33 + [1, 3] and depths.tolist() == [0] * 34 + [1]
    for cu in ([-4, 2, 2 ** 31 - 1], [5, 3, 0], [-9, -5, -1], [40, 50, 60]):
        K.kvo_tree_masks(dev(parents), dev(cu), masks, depths, status)
        torch.cuda.synchronize()


def _drafts(g, trees, tokens):
    """Drafted and chosen tokens out of few, so that paths are accepted and siblings repeat."""
    n = sum(len(t) for t in trees)
    return g.integers(0, tokens, n), g.integers(0, tokens, n)


@pytest.mark.parametrize("tokens", [1, 2, 3, 1000])
def test_accept(tokens):
    g = np.random.default_rng(tokens)
    trees = _trees(tokens) + [list(range(-1, 1023)), random_tree(g, 1024), list(range(-1, 1024))]
    cu = _cu([len(t) for t in trees])
    drafted, chosen = _drafts(g, trees, tokens)
    kv = np.array([len(t) + int(g.integers(0, 50)) for t in trees])
    kv[6], kv[9] = len(trees[6]) - 1, 0  # refused
    T = int(cu[-1])
    path, accepted, nxt = dev(np.full(T + 2, 77)), dev(np.full(len(trees), 77)), dev(np.full(len(trees), 77))
    two = lambda x: dev(np.concatenate([x, [5, 5]]))  # noqa: E731
    K.kvo_tree_accept(two(np.concatenate([np.array(t, np.int64) for t in trees])), two(drafted), two(chosen), dev(cu), dev(kv), path,
                      accepted, nxt)
    torch.cuda.synchronize()
    path, accepted, nxt = path.cpu().numpy(), accepted.cpu().numpy(), nxt.cpu().numpy()
    for r, t in enumerate(trees):
        a, b = cu[r], cu[r + 1]
        want = O.accept(t, drafted[a:b], chosen[a:b]) if kv[r] >= len(t) and len(t) <= 1024 else []
        assert accepted[r] == len(want), r
        assert path[a:b].tolist() == want + [-1] * (b - a - len(want)), r
        assert nxt[r] == (chosen[a + want[-1]] if want else -1)
    assert (path[T:] == 77).all()


# ---- commit, move ---------------------------------------------------------------------------------

@pytest.mark.parametrize("R,block,M,window,sinks", [(1, 8, 6, 0, 0), (7, 16, 9, 20, 4), (64, 8, 12, 33, 17), (1030, 8, 7, 9, 3),
                                                    (4096, 16, 5, 0, 0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_commit(R, block, M, window, sinks, in_place):
    g = np.random.default_rng(R)
    n = g.choice([0, 1, 2, 5, 17, 30], R)
    kv = np.array([int(g.integers(min(k, M * block), M * block + 1)) for k in n])
    n = np.minimum(n, kv)
    accepted = np.array([int(g.integers(0, k + 1)) for k in n])
    lengths = kv.copy()
    refused = g.random(R) < 0.1
    kv[refused & (n > 0)] = 0
    accepted[g.random(R) < 0.02] = 10 ** 6   # taken as all
    accepted[g.random(R) < 0.02] = -3        # as none
    n_blocks = R * M
    table = g.permutation(n_blocks).reshape(R, M).astype(np.int32)
    ring = np.full(n_blocks + 3, -1, np.int32)
    bounds = np.array([2, n_blocks + 1], np.int64)
    want = O.commit(lengths, kv, n, accepted, block, table, ring, bounds, window, sinks)
    lo, b_in, r_dev = dev(lengths), dev(bounds, torch.int64), dev(ring)
    out = lo if in_place else dev(np.full(R, 77))
    b_out = b_in if in_place else dev([77, 77], torch.int64)
    K.kvo_paged_commit(lo, dev(kv), dev(_cu(n)), dev(accepted), block, dev(table), r_dev, b_in, b_out, out, window=window, sinks=sinks)
    torch.cuda.synchronize()
    for x, y in zip((out, r_dev, b_out), want):
        assert np.array_equal(x.cpu().numpy(), y)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("block,pools", [(8, 1), (24, 3), (64, 2)])
def test_move(fmt, block, pools):
    g = np.random.default_rng(block)
    n = np.array([5, 1, 40, 0, 33, 100, 9, 6])
    kv = n + g.integers(0, 70, len(n))
    kv[6] = 3  # refused
    R, T = len(n), int(n.sum())
    M = -(-int(kv.max()) // block) + 1
    n_blocks = R * M + 2
    table = g.permutation(R * M).reshape(R, M).astype(np.int32)
    accepted, path = np.zeros(R, np.int64), np.full(T, -1)
    cu = _cu(n)
    for r in range(R):
        a = {0: 3, 2: 40, 4: 9, 5: 61, 7: 6}.get(r, min(1, n[r]))
        p = np.concatenate([[0], np.sort(g.choice(np.arange(1, n[r]), a - 1, replace=False))]) if a else np.zeros(0)
        accepted[r] = a
        path[cu[r]:cu[r] + a] = p
    path[cu[7]:cu[7] + 6] = [0, 2, 1, 99, 5, 3]  # a node before its place, one that is none: skipped
    table[5, 1] = -1
    table[4, 0] = n_blocks
    bytes_of = K.kvo_paged_block_bytes(fmt, block)
    before = g.integers(0, 256, (pools, n_blocks, bytes_of)).astype(np.uint8)
    pool = torch.from_numpy(before.copy()).cuda()
    K.kvo_paged_move(pool, n_blocks, block, fmt, dev(table), dev(kv), dev(cu), dev(path), dev(accepted), n_pools=pools)
    torch.cuda.synchronize()
    parts = {BF16: [(1152, 0)], F8: [(576, 0), (4, 576 * block)], Q4: [(288, 0), (36, 288 * block)]}[fmt]
    want = before.copy()
    for r in range(R):
        if kv[r] < n[r]:
            continue
        first = kv[r] - n[r]
        for k in range(accepted[r]):
            p = path[cu[r] + k]
            if not k <= p < n[r]:
                continue
            b0, b1 = table[r, (first + p) // block], table[r, (first + k) // block]
            if not (0 <= b0 < n_blocks and 0 <= b1 < n_blocks):
                continue
            for width, at in parts:
                s, d = at + width * ((first + p) % block), at + width * ((first + k) % block)
                want[:, b1, d:d + width] = before[:, b0, s:s + width]
    assert np.array_equal(pool.cpu().numpy(), want)


# ---- attention ------------------------------------------------------------------------------------

def _random(seed):
    g = np.random.default_rng(seed)
    return lambda r, n: random_tree(g, n)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("H,new,lens", [(16, [1], [1]), (16, [16], [300]), (1, [7], [7]), (5, [40, 1, 8], [300, 1, 140]),
                                        (128, [5], [260]), (20, [61, 33], [700, 33]), (2, [200], [333]), (16, [0, 9, 0], [50, 137, 0])])
def test_trees(fmt, H, new, lens):
    run(fmt, lens, new, H, 16, seed=H, pad=3, parents=_random(H + len(new)))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("H,new,lens,window,sinks", [(16, [16], [300], 5, 0), (3, [40, 12], [500, 12], 9, 2), (64, [30], [700], 130, 70),
                                                     (8, [25], [25], 3, 20), (20, [61], [900], 400, 4), (16, [9], [2000], 4000, 1)])
def test_windows_go_by_depth(fmt, H, new, lens, window, sinks):
    run(fmt, lens, new, H, 24, window, sinks, seed=window, parents=_random(window))


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_chain_is_the_causal_order(fmt):
    for H, new, lens, window in ((16, [70], [400], 0), (64, [3, 9], [200, 9], 50)):
        c = Cache(lens, 16, fmt, 51)
        cu = _cu(new)
        q = O.bf16_bits(np.random.default_rng(52).standard_normal((int(cu[-1]), H, 576)))
        _, masks, depths = forest([list(range(-1, n - 1)) for n in new])
        a = attend(c, q, cu, lens, window=window)
        b = attend(c, q, cu, lens, window=window, masks=masks, depths=depths)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("H", [4, 16, 64])
def test_masks_of_any_kind(fmt, H):
    # bits that are no tree's, none at all (the context alone), bits behind a node, nodes past the mask's words, no context
    g = np.random.default_rng(53)
    new, lens = [40, 6, 70, 5], [300, 6, 200, 4]
    cu = _cu(new)
    T = int(cu[-1])
    words = 2
    masks = g.integers(-2 ** 31, 2 ** 31, (T, words)).astype(np.int64).astype(np.int32)
    masks[cu[0] + 3] = 0
    masks[cu[1]:cu[2]] = 0           # nothing visible at all: 0 and -inf
    masks[cu[1] + 5] = [1 << 2, 0]
    trees = []
    for r, n in enumerate(new):
        b = np.unpackbits(masks[cu[r]:cu[r + 1]].view(np.uint8), axis=1, bitorder="little").astype(bool)
        trees.append((np.pad(b, ((0, 0), (0, max(0, n - 64))))[:, :n], np.zeros(n, int)))
    c = Cache(lens, 16, fmt, 54)
    q = O.bf16_bits(g.standard_normal((T, H, 576)))
    out, lse = attend(c, q, cu, lens, masks=masks)
    check(c, q, cu, lens, out, lse, trees=trees)
    assert np.isneginf(lse[cu[1]:cu[1] + 5]).all() and np.isfinite(lse[cu[1] + 5]).all()
    assert np.isneginf(lse[cu[3]:]).all()  # fewer rows than nodes
    # depths out of range are taken as 0 or as the node's index
    depths = g.integers(-5, 200, T)
    trees = [(m, np.clip(depths[cu[r]:cu[r + 1]], 0, np.arange(new[r]))) for r, (m, _) in enumerate(trees)]
    out, lse = attend(c, q, cu, lens, window=30, sinks=3, masks=masks, depths=depths)
    check(c, q, cu, lens, out, lse, window=30, sinks=3, trees=trees)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("H", [2, 16, 64])
def test_what_is_not_finite_stays_with_those_that_see_it(fmt, H):
    # a node's row with NaN: its descendants get NaN, its siblings do not
    parents = [-1, 0, 0, 1, 2, 3, 4, 0]
    c = Cache([150], 16, fmt, 55)
    row = O.bf16_bits(np.random.default_rng(56).standard_normal((1, 576)))
    row[0, 9] = 0x7FC0
    c.set_rows(0, [150 - 8 + 1], row)
    trees, masks, depths = forest([parents])
    q = O.bf16_bits(np.random.default_rng(57).standard_normal((8, H, 576)))
    out, lse = attend(c, q, [0, 8], [150], masks=masks, depths=depths)
    bad = np.isnan(O.bf16_values(out)).any((1, 2)).tolist()
    assert bad == [bool(m[1]) for m in trees[0][0]]
    check(c, q, [0, 8], [150], out, lse, trees=trees, tokens={i for i in range(8) if not bad[i]})


@pytest.mark.parametrize("fmt", FORMATS)
def test_split_joined_and_many_tiles(fmt):
    run(fmt, [20011], [3], 16, 64, seed=61, parents=_random(62))
    run(fmt, [9000, 5, 3001, 0, 700], [7, 1, 2, 0, 1], 64, 64, seed=63, parents=_random(64))
    new = [1000, 600, 1, 700, 1024]  # more tiles than are listed, as many nodes as masks hold
    run(fmt, [1000, 800, 1, 1300, 1100], new, 50, 64, 100, 3, seed=65, parents=_random(66), tokens={0, 999, 1000, 1300, 1599, 1600, 2000, 3324})


def test_more_nodes_than_masks_hold():
    # causal order beyond: nodes without a bit see the context and those before them that have one
    n = 1100
    c = Cache([1200], 64, BF16, 67)
    q = O.bf16_bits(np.random.default_rng(68).standard_normal((n, 1, 576)))
    masks = np.full((n, 32), -1, np.int32)
    seen = np.ones((n, n), bool)
    seen[:, 1024:] = False
    out, lse = attend(c, q, [0, n], [1200], masks=masks)
    check(c, q, [0, n], [1200], out, lse, trees=[(seen, np.zeros(n, int))], tokens={0, 5, 1023, 1024, 1099})


# ---- together -------------------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("W,S", [(0, 0), (40, 3)])
def test_a_loop_of_draft_steps_in_one_graph(fmt, W, S):
    """Plan, masks, write, attend, accept, commit and move of a draft step captured once and replayed: trees change, paths
    are accepted, blocks come back, and the cache holds what a sequence without drafts would hold."""
    R, B, M, H, n_most, layers = 4, 8, 16, 16, 12, 2
    g = np.random.default_rng(71)
    T, words = R * n_most, 1
    n_blocks = 48
    ring = dev(np.concatenate([g.permutation(n_blocks), [-1, -1]]))
    bounds = dev([0, n_blocks], torch.int64)
    z = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    lengths, table, new, kv, cu, slots, status = z(R), z(R, M) - 1, z(R), z(R), z(R + 1), z(T), z(R)
    parents, drafted, chosen, masks, depths, path, accepted, nxt = z(T), z(T), z(T), z(T, words), z(T), z(T), z(R), z(R)
    pools = torch.full((layers, n_blocks, K.kvo_paged_block_bytes(fmt, B)), 0xFF, dtype=torch.uint8, device="cuda")
    rows = torch.zeros(layers, T, 576, dtype=torch.int16, device="cuda")
    q = torch.zeros(layers, T, H, 576, dtype=torch.int16, device="cuda")
    out = torch.zeros(layers, T, H, 512, dtype=torch.int16, device="cuda")
    lse = torch.zeros(layers, T, H, device="cuda")
    ws = torch.empty(K.kvo_paged_attend_workspace_size(R, T, H, 0), dtype=torch.uint8, device="cuda")

    def step():
        K.kvo_paged_plan(lengths, new, B, table, ring, bounds, bounds, lengths, kv, cu, slots, status)
        K.kvo_tree_masks(parents, cu, masks, depths)
        for layer in range(layers):
            K.kvo_paged_write(rows[layer], slots, pools[layer], n_blocks, B, fmt)
            K.kvo_paged_attend_tree(pools[layer], n_blocks, B, fmt, table, kv, cu, masks, q[layer], SCALE, out[layer], lse[layer],
                                    depths=depths, window=W, sinks=S, workspace=ws)
        K.kvo_tree_accept(parents, drafted, chosen, cu, kv, path, accepted, nxt)
        K.kvo_paged_commit(lengths, kv, cu, accepted, B, table, ring, bounds, bounds, lengths, window=W, sinks=S)
        K.kvo_paged_move(pools, n_blocks, B, fmt, table, kv, cu, path, accepted, n_pools=layers)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()  # nothing new: loads the modules
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    torch.cuda.synchronize()
    state = dict(lengths=np.zeros(R, np.int32), table=np.full((R, M), -1, np.int32), ring=ring.cpu().numpy(),
                 bounds=np.array([0, n_blocks], np.int64))
    history = [[np.zeros((0, 576), np.uint16) for _ in range(R)] for _ in range(layers)]
    moved = refused = 0
    for it in range(40):
        if it in (15, 28):  # a request ends, in a plan of its own with the window
            n = np.array([-1 if r == it % R else 0 for r in range(R)])
            want = O.plan(state["lengths"], n, B, state["table"], state["ring"], state["bounds"], T, window=W, sinks=S)
            new.copy_(dev(n))
            K.kvo_paged_plan(lengths, new, B, table, ring, bounds, bounds, lengths, kv, cu, slots, status, window=W, sinks=S)
            state = {k: want[k] for k in state}
            for h in history:
                h[it % R] = h[it % R][:0]
        n = g.integers(0, n_most + 1, R)
        n[state["lengths"] > M * B - 30] = 0
        if it == 20:
            n[1] = n_most
        trees = [random_tree(g, int(k)) for k in n]
        par = np.concatenate([np.array(t, np.int64) for t in trees] + [np.full(T - int(n.sum()), -1)])
        dr, ch = g.integers(0, 2, T), g.integers(0, 2, T)
        bits = O.bf16_bits(g.standard_normal((layers, T, 576)))
        qb = O.bf16_bits(g.standard_normal((layers, T, H, 576)))
        for d, x in ((new, n), (parents, par), (drafted, dr), (chosen, ch)):
            d.copy_(dev(x))
        rows.copy_(dev(bits.view(np.int16), torch.int16))
        q.copy_(dev(qb.view(np.int16), torch.int16))
        graph.replay()
        torch.cuda.synchronize()
        plan = O.plan(state["lengths"], n, B, state["table"], state["ring"], state["bounds"], T)
        c0 = plan["cu"]
        paths = []
        for r in range(R):
            a, b = c0[r], c0[r + 1]
            ok = plan["status"][r] == O.OK
            refused += not ok
            paths.append(O.accept(trees[r], dr[a:b], ch[a:b]) if ok and b > a else [])
        acc = [len(p) for p in paths]
        L, ring_w, bounds_w = O.commit(plan["lengths"], plan["kv_lens"], n, acc, B, plan["table"], plan["ring"], plan["bounds"], W, S)
        assert accepted.tolist() == acc and lengths.tolist() == L.tolist() and bounds.tolist() == bounds_w.tolist()
        assert np.array_equal(ring.cpu().numpy(), ring_w) and np.array_equal(table.cpu().numpy(), plan["table"])
        live = [int(ring_w[i % len(ring_w)]) for i in range(bounds_w[0], bounds_w[1])]
        assert len(set(live)) == len(live)
        for layer in range(layers):
            x = bits[layer]
            if fmt != BF16:
                x = O.bf16_bits(O.dequantize(*O.quantize(x)) if fmt == Q4 else O.dequantize8(*O.quantize8(x)))
            now, _ = pool_rows(pools[layer], B, fmt)
            got, gl = O.bf16_values(out[layer].cpu().numpy().view(np.uint16)), lse[layer].cpu().numpy()
            for r in range(R):
                a, b = c0[r], c0[r + 1]
                if plan["status"][r] != O.OK:
                    assert np.isneginf(gl[a:b]).all()
                    continue
                old = history[layer][r]
                if b > a:
                    k = O.bf16_values(np.concatenate([old, x[a:b]]))
                    m = O.ancestors(trees[r])
                    seen = O.tree_seen(len(k), b - a, m, m.sum(1) - 1, np.arange(len(k)), W, S)
                    ref, rl, mag, dot, cnt, _ = O.attend_seen(k, O.bf16_values(qb[layer][a:b]), seen, SCALE)
                    es = 2 * 576 * 2.0 ** -23 * dot + 2.0 ** -17
                    tol = (2.0 ** -8 + 2.0 ** -11 + 4 * es[..., None]) * mag + 1e-4 * np.abs(k).max() + 2.0 ** -8 * 1.01 * np.abs(ref)
                    assert np.all(np.abs(got[a:b] - ref) <= tol), (it, r)
                    assert np.all(np.abs(gl[a:b] - rl) <= 4 * es + 2.0 ** -20 * (1 + np.abs(rl)))
                history[layer][r] = np.concatenate([old, x[a:b][paths[r]]]) if paths[r] else old
                moved += any(p != k for k, p in enumerate(paths[r]))
                h = history[layer][r]
                assert len(h) == L[r]
                # the cache's rows, as far as they are kept
                t = np.array([t for t in range(len(h)) if W == 0 or t > len(h) - W or t < S], np.int64)
                if len(t):
                    at = plan["table"][r, t // B].astype(np.int64) * B + t % B
                    assert np.array_equal(now[at], O.bf16_values(h[t])), (it, r)
        state = dict(lengths=L, table=plan["table"], ring=ring_w, bounds=bounds_w)
    assert moved > 20 and int(state["bounds"][0]) > n_blocks // 2  # paths were moved, blocks taken again


@pytest.mark.parametrize("fmt", FORMATS)
def test_other_streams_and_raw_ones(fmt):
    c = Cache([200], 16, fmt, 81)
    parents = random_tree(np.random.default_rng(82), 9)
    trees, masks, depths = forest([parents])
    q = O.bf16_bits(np.random.default_rng(83).standard_normal((9, 16, 576)))
    a = attend(c, q, [0, 9], [200], masks=masks, depths=depths)
    s = torch.cuda.Stream()
    b = attend(c, q, [0, 9], [200], masks=masks, depths=depths, stream=s)
    assert np.array_equal(a[0], b[0])
    ws = torch.empty(K.kvo_paged_attend_workspace_size(1, 9, 16), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    b = attend(c, q, [0, 9], [200], masks=masks, depths=depths, stream=s.cuda_stream, workspace=ws)
    assert np.array_equal(a[0], b[0])
    with pytest.raises(K.KvoError):
        attend(c, q, [0, 9], [200], masks=masks, depths=depths, stream=s.cuda_stream)


def test_empty_calls():
    e, c1 = torch.empty(0, dtype=torch.int32, device="cuda"), dev([0, 0])
    one = dev([7])
    K.kvo_tree_masks(e, c1, e.view(0, 1), e)
    K.kvo_tree_accept(e, e, e, c1, dev([5]), e, one, one.clone())
    torch.cuda.synchronize()
    assert one.item() == 0
    pool = P._pool(2, 8, F8)
    K.kvo_paged_move(pool, 2, 8, F8, dev([[0, 1]]), dev([5]), c1, e, dev([3]))
    out, lse = attend(Cache([9], 8, F8, 84), np.zeros((0, 4, 576), np.uint16), [0, 0], [9], masks=np.zeros((0, 1), np.int32))
    assert out.shape == (0, 4, 512)
    torch.cuda.synchronize()
