"""Cases of the 8-bit paged cache and of steps that verify a tree of drafted tokens over the paged cache.

A cached row is 576 elements (latent 512, which is also the value, and rope key 64).  The 8-bit
cache holds E4M3 codes and one power of two a row.  A draft step writes the rows of a tree's
nodes behind the context, attends with every node seeing the context and its ancestors, accepts
the longest path that the model agrees with, and moves that path's rows together.  `run`
computes an operator in elementary torch operations, or, with `own`, through the library's entry
points.
"""
import math

import numpy as np
import torch

own = False

ROW, VAL, GROUP = 576, 512, 16
SCALE = 1.0 / math.sqrt(192.0)
FORMATS = {"bf16": 0, "q4": 1, "f8": 8}
ROW_BYTES = {"bf16": 1152, "q4": 324, "f8": 580}
LOW, HIGH = -32, 32  # exponents of the 8-bit cache's row scales


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def listed():
    return [
        # a decode step's new rows (32 requests of 4 positions) into the 8-bit cache, and read back
        dict(name="rows_f8_128", op="rows", rows=128, block=64),
        # a prompt chunk's rows with padding behind it, odd count
        dict(name="rows_f8_65531", op="rows", rows=65531, block=64),
        # one short request over the 8-bit cache, 16 heads: latency
        dict(name="f8_one_4k_h16", op="attend", requests=1, context=4096, new=1, ragged=False, heads=16, window=0,
             sinks=0, block=64),
        # the 64k decode batch on the 8-bit cache with a tensor-parallel share of the heads, whole context
        dict(name="f8_32x64k_h16", op="attend", requests=32, context=65536, new=1, ragged=True, heads=16, window=0,
             sinks=0, block=64),
        # four positions of 128 heads on the 8-bit cache, whole context
        dict(name="f8_16x4x8k_h128", op="attend", requests=16, context=8192, new=4, ragged=True, heads=128, window=0,
             sinks=0, block=128),
        # a prompt chunk over the 8-bit cache, windowed layer, odd heads
        dict(name="f8_chunk_2048_h20", op="attend", requests=1, context=16384, new=2048, ragged=False, heads=20,
             window=1024, sinks=4, block=64),
        # one short request with a small tree, 16 heads: latency
        dict(name="tree_bf16_1x16_4k_h16", op="tree", format="bf16", requests=1, context=4096, new=16, ragged=False,
             heads=16, window=0, sinks=0, block=64),
        # a batch of trees under all heads
        dict(name="tree_bf16_16x32_8k_h128", op="tree", format="bf16", requests=16, context=8192, new=32, ragged=True,
             heads=128, window=0, sinks=0, block=64),
        # wide trees with a tensor-parallel share of the heads on the 8-bit cache
        dict(name="tree_f8_32x64_16k_h16", op="tree", format="f8", requests=32, context=16384, new=64, ragged=True,
             heads=16, window=0, sinks=0, block=64),
        # odd trees in a windowed layer on the 4-bit cache
        dict(name="tree_q4_9x61_12k_h20", op="tree", format="q4", requests=9, context=12289, new=61, ragged=True,
             heads=20, window=1024, sinks=4, block=24),
        # the end of a draft step: the 16-request, 8-layer batch, trees of 32 nodes
        dict(name="step_16x32_8_layers", op="step", format="bf16", requests=16, context=2048, new=32, ragged=False,
             layers=8, window=0, sinks=0, block=64),
        # a server's mixed draft step: ragged trees, windowed layers on the 8-bit cache
        dict(name="step_251x61_3_layers", op="step", format="f8", requests=251, context=700, new=61, ragged=True,
             layers=3, window=256, sinks=16, block=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rows", "step", "attend", "attend", "tree", "tree"])
    block = rng.choice([8, 16, 24, 64, 128])
    if op == "rows":
        return dict(op="rows", rows=_log(rng, 1, 65531), block=block)
    if op == "step":
        while True:
            c = dict(op="step", format=rng.choice(["bf16", "q4", "f8"]), requests=_log(rng, 1, 251),
                     context=_log(rng, 16, 4096), new=_log(rng, 1, 100), ragged=rng.random() < 0.7,
                     layers=rng.randint(1, 8), window=rng.choice([0, _log(rng, 64, 512)]), sinks=rng.choice([0, 4, 64]),
                     block=block)
            if c["requests"] * (c["context"] + c["new"]) * c["layers"] * ROW_BYTES[c["format"]] <= 3.2e8:
                return c
    while True:
        c = dict(op=op, requests=_log(rng, 1, 64), context=_log(rng, 16, 262144),
                 new=1 if op == "attend" and rng.random() < 0.4 else _log(rng, 1, 1024 if op == "attend" else 128),
                 ragged=rng.random() < 0.6, heads=_log(rng, 1, 128),
                 window=rng.choice([0, 0, _log(rng, 32, 8192)]), sinks=rng.choice([0, 4, 64]), block=block)
        if op == "tree":
            c["format"] = rng.choice(["bf16", "q4", "f8"])
        c["context"] = max(c["context"], c["new"])
        span = _span(c)
        if (work(c)["flops"] <= 2.5e11 and c["requests"] * c["context"] <= (1 << 21) and c["requests"] * span <= (1 << 20)
                and c["requests"] * c["new"] * c["heads"] * span <= (1 << 29)):
            return c


def _span(c):
    """Rows of the cache that a request's query tokens can see, at most."""
    return min(c["context"], c["window"] + c["sinks"] + c["new"]) if c["window"] else c["context"]


# ---- inputs ---------------------------------------------------------------------------------

def _lengths(c):
    """(cached lengths with the new tokens, new tokens) of each request: the case's alone."""
    R = c["requests"]
    g = np.random.default_rng([R, c["context"], c["new"]])
    kv = np.full(R, c["context"] + (c["new"] if c["op"] == "step" else 0), np.int64)
    new = np.full(R, c["new"], np.int64)
    if c["ragged"]:
        kv = np.maximum(1, (kv * g.uniform(0.4, 1.0, R)).astype(np.int64))
        new = np.maximum(1, (new * g.uniform(0.3, 1.0, R)).astype(np.int64))
        kv[0], new[0] = c["context"], c["new"]
    return np.maximum(kv, new), new


def _tree(n, g):
    """Parents of a tree of n nodes: the root, then nodes whose parents tend to be recent ones."""
    i = np.arange(1, n)
    back = np.minimum(i, 1 + np.floor(-4.0 * np.log(1.0 - g.random(n - 1))).astype(np.int64)) if n > 1 else i
    return np.concatenate([[-1], i - back])


def _values(i):
    """E2M1 codes (0..15) -> values."""
    t = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                     dtype=torch.float32, device=i.device)
    return t[i.long()]


def _pack_q4(x, block):
    """Blocks of the 4-bit cache from rows: codes [block][288], then E4M3 scales [block][36] of 16 elements each."""
    x = x.float().view(-1, ROW // GROUP, GROUP)
    s = (x.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    f = s.float()[..., None]
    a = torch.where(f > 0, x.abs() / torch.where(f > 0, f, torch.ones_like(f)), torch.zeros_like(x))
    m = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte()
         + (a >= 3.5).byte() + (a > 5.0).byte()) | ((x < 0).byte() << 3)
    n = x.shape[0] // block
    e = m.reshape(n, block * ROW // 2, 2)
    return torch.cat([e[..., 0] | (e[..., 1] << 4), s.view(torch.uint8).reshape(n, block * ROW // GROUP)], dim=1)


def _quantize(rows):
    """Rows [n][576] -> (codes [n][576] E4M3, scales [n] float32): the scale is the least power of two, 2^-32 .. 2^32,
    with which no element passes 448, and NaN where an element is not finite."""
    x = rows.float()
    fine = torch.isfinite(x).all(-1)
    x = torch.where(fine[:, None], x, torch.zeros_like(x))
    f, e = torch.frexp(x.abs().amax(-1) / 448.0)
    e = torch.where(f > 0.5, e, e - 1).clamp(LOW, HIGH)
    e = torch.where(f > 0, e, torch.full_like(e, LOW))
    two = lambda n: ((n + 127) << 23).view(torch.float32)  # noqa: E731  (exact on every device)
    codes = (x * two(-e)[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes, torch.where(fine, two(e), torch.full_like(f, math.nan))


def _pack_f8(codes, scales, block):
    """Blocks of the 8-bit cache: codes [block][576], then scales [block]."""
    n = codes.shape[0] // block
    return torch.cat([codes.view(torch.uint8).reshape(n, block * ROW),
                      scales.contiguous().view(torch.uint8).reshape(n, block * 4)], dim=1)


def _rows_at(pool, fmt, block, at):
    """float32 rows [.., 576] of the cache at slots `at`."""
    if fmt == "bf16":
        return pool.view(torch.bfloat16).view(-1, ROW)[at].float()
    if fmt == "f8":
        codes = pool[:, :block * ROW].reshape(-1, ROW)[at].view(torch.float8_e4m3fn).float()
        scales = pool[:, block * ROW:].contiguous().view(torch.float32).reshape(-1)[at]
        return codes.mul_(scales[..., None])
    codes = pool[:, :block * ROW // 2].reshape(-1, ROW // 2)[at]
    scales = pool[:, block * ROW // 2:].reshape(-1, ROW // GROUP)[at].view(torch.float8_e4m3fn).float()
    e = torch.stack([codes & 15, codes >> 4], dim=-1)
    return (_values(e.reshape(*at.shape, ROW // GROUP, GROUP)) * scales[..., None]).reshape(*at.shape, ROW)


def _fill(n_blocks, block, fmt, tg, dev):
    """A cache's pool [n_blocks][bytes] of random rows."""
    pool = torch.empty(n_blocks, ROW_BYTES[fmt] * block, dtype=torch.uint8, device=dev)
    step = max(1, (1 << 17) // block)
    for a in range(0, n_blocks, step):
        b = min(n_blocks, a + step)
        x = torch.randn((b - a) * block, ROW, generator=tg, device=dev).bfloat16()
        if fmt == "bf16":
            pool[a:b] = x.view(torch.uint8).view(b - a, -1)
        else:
            pool[a:b] = _pack_f8(*_quantize(x), block) if fmt == "f8" else _pack_q4(x, block)
    return pool


def prepare(case, seed):
    c, dev = case, _device()
    g = np.random.default_rng(seed)
    tg = torch.Generator(device=dev).manual_seed(seed)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)  # noqa: E731
    B = c["block"]
    if c["op"] == "rows":
        n = c["rows"]
        n_blocks = -(-n // B) + 3
        slots = g.permutation(n_blocks * B)[:n]
        slots[g.random(n) < 0.02] = -1  # padding rows
        rows = torch.randn(n, ROW, generator=tg, device=dev) * torch.exp(torch.randn(n, 1, generator=tg, device=dev))
        return dict(op="rows", block=B, n_blocks=n_blocks, rows=rows.bfloat16(), slots=i32(slots),
                    pool=torch.zeros(n_blocks, ROW_BYTES["f8"] * B, dtype=torch.uint8, device=dev))
    R = c["requests"]
    kv, new = _lengths(c)
    cu = np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1])
    fmt = c.get("format", "f8")
    M = -(-int(kv.max()) // B) + 2
    used = -(-kv // B)
    n_blocks = int(used.sum()) + 2
    ids = g.permutation(n_blocks)
    table = np.full((R, M), -1, np.int64)
    table[np.arange(M)[None, :] < used[:, None]] = ids[:int(used.sum())]
    s = dict(op=c["op"], format=fmt, block=B, n_blocks=n_blocks, table=i32(table), kv=i32(kv), cu=i32(cu),
             window=c["window"], sinks=c["sinks"], steps=c["new"])
    if c["op"] == "step":
        parents, drafted, chosen = np.empty(T, np.int64), np.empty(T, np.int64), np.empty(T, np.int64)
        for r in range(R):
            n, at = int(new[r]), int(cu[r])
            p = _tree(n, g)
            # an accepted path: the root and the last `a` nodes, one below the other
            a = int(g.integers(0, (n - 1) // 2 + 1))
            p[n - a:] = np.arange(n - a - 1, n - 1)
            if a:
                p[n - a] = 0
            parents[at:at + n] = p
            drafted[at:at + n] = g.integers(0, 120000, n)
            chosen[at:at + n] = g.integers(120000, 129280, n)
            on = np.concatenate([[0], np.arange(n - a, n)])
            chosen[at + on[:-1]] = drafted[at + on[1:]]
        pools = torch.cat([_fill(n_blocks, B, fmt, tg, dev) for _ in range(c["layers"])])
        ring = np.full(2 * n_blocks + 8, -1, np.int64)
        ring[5:5 + n_blocks - int(used.sum())] = ids[int(used.sum()):]
        return dict(s, parents=i32(parents), drafted=i32(drafted), chosen=i32(chosen), pools=pools, layers=c["layers"],
                    lengths=i32(kv), ring=i32(ring), words=-(-c["new"] // 32),
                    bounds=torch.tensor([5, 5 + n_blocks - int(used.sum())], dtype=torch.int64, device=dev))
    s["pool"] = _fill(n_blocks, B, fmt, tg, dev)
    s["q"] = torch.randn(T, c["heads"], ROW, generator=tg, device=dev).bfloat16()
    s["span"], s["context"] = _span(c), c["context"]
    if c["op"] == "tree":
        words = -(-c["new"] // 32)
        masks, depths = np.zeros((T, 32 * words), np.uint8), np.zeros(T, np.int64)
        for r in range(R):
            p = _tree(int(new[r]), g)
            for i in range(int(new[r])):
                at = int(cu[r]) + i
                if p[i] >= 0:
                    masks[at] = masks[int(cu[r]) + p[i]]
                masks[at, i] = 1
        depths = masks.sum(1) - 1
        s["masks"] = i32(np.packbits(masks, axis=1, bitorder="little").view(np.uint32).view(np.int32))
        s["depths"] = i32(depths)
    return s


# ---- the operators --------------------------------------------------------------------------

def run(state):
    s = state
    if own:
        return _own(s)
    if s["op"] == "rows":
        return _rows(s)
    if s["op"] == "step":
        return _step(s)
    return _attend(s)


def _own(s):
    from top_cache_gb300 import kvo as K
    fmt = FORMATS[s.get("format", "f8")]
    if s["op"] == "rows":
        K.kvo_paged_write(s["rows"], s["slots"], s["pool"], s["n_blocks"], s["block"], fmt)
        back = torch.zeros_like(s["rows"])
        K.kvo_paged_read(s["pool"], s["n_blocks"], s["block"], fmt, s["slots"], back)
        return back
    dev = s["kv"].device
    if s["op"] == "step":
        R, T = s["kv"].numel(), s["parents"].numel()
        e = lambda *n: torch.empty(n, dtype=torch.int32, device=dev)  # noqa: E731
        out = dict(masks=e(T, s["words"]), depths=e(T), path=e(T), accepted=e(R), next=e(R), lengths=e(R),
                   bounds=torch.empty(2, dtype=torch.int64, device=dev))
        K.kvo_tree_masks(s["parents"], s["cu"], out["masks"], out["depths"])
        K.kvo_tree_accept(s["parents"], s["drafted"], s["chosen"], s["cu"], s["kv"], out["path"], out["accepted"],
                          out["next"])
        K.kvo_paged_commit(s["lengths"], s["kv"], s["cu"], out["accepted"], s["block"], s["table"], s["ring"],
                           s["bounds"], out["bounds"], out["lengths"], window=s["window"], sinks=s["sinks"])
        K.kvo_paged_move(s["pools"], s["n_blocks"], s["block"], fmt, s["table"], s["kv"], s["cu"], out["path"],
                         out["accepted"], n_pools=s["layers"])
        out["ring"], out["pools"] = s["ring"], s["pools"]
        return out
    T, H = s["q"].shape[0], s["q"].shape[1]
    out = torch.empty(T, H, VAL, dtype=torch.bfloat16, device=dev)
    lse = torch.empty(T, H, dtype=torch.float32, device=dev)
    if s["op"] == "tree":
        K.kvo_paged_attend_tree(s["pool"], s["n_blocks"], s["block"], fmt, s["table"], s["kv"], s["cu"], s["masks"],
                                s["q"], SCALE, out, lse, depths=s["depths"], window=s["window"], sinks=s["sinks"])
    else:
        K.kvo_paged_attend(s["pool"], s["n_blocks"], s["block"], fmt, s["table"], s["kv"], s["cu"], s["q"], SCALE, out,
                           lse, window=s["window"], sinks=s["sinks"])
    return out, lse


def _rows(s):
    """Rows into the 8-bit cache at their slots, and the cache's values at those slots."""
    codes, scales = _quantize(s["rows"])
    x = (codes.float() * scales[:, None]).bfloat16()
    return torch.where((s["slots"] >= 0)[:, None], x, torch.zeros_like(x))


def _attend(s):
    """Attention over each query token's visible rows: by position, or, for a tree, the context and the mask's nodes."""
    R, B, W, S = s["kv"].numel(), s["block"], s["window"], s["sinks"]
    dev, span, P, H = s["q"].device, s["span"], s["steps"], s["q"].shape[1]
    kv, cu = s["kv"].long(), s["cu"].long()
    new = cu[1:] - cu[:-1]
    first = kv - new
    x = torch.arange(span, device=dev)[None, :]
    if span < s["context"]:  # [sinks |] lo .. kv - 1
        lo = (first - W + 1).clamp(min=0)
        t = torch.where(x < S, x, lo[:, None] + x - S)
        ok = (x < S) | (t >= S)
    else:
        t = x.expand(R, span)
        ok = torch.ones_like(t, dtype=torch.bool)
    ok = ok & (t < kv[:, None])
    t = torch.minimum(t, kv[:, None] - 1).clamp(min=0)
    slot = s["table"].long().gather(1, t // B) * B + t % B
    k = _rows_at(s["pool"], s["format"], B, slot)                            # [R][span][576]
    i = torch.arange(P, device=dev)[None, :]
    qi = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][qi].float().flatten(1, 2)                                     # [R][P * H][576]
    if s["op"] == "tree":
        node = t - first[:, None]                                            # [R][span], < 0: the context
        j = node.clamp(min=0)
        m = s["masks"][qi].long()                                            # [R][P][words]
        bit = (m.gather(2, (j // 32)[:, None, :].expand(R, P, span)) >> (j % 32)[:, None, :]) & 1
        see = ok[:, None, :] & ((node < 0)[:, None, :] | (bit == 1))
        # a node lies at its depth, not at its row
        depths = s["depths"].long()
        pos = first[:, None] + depths[qi]
        at = torch.where(node < 0, t, first[:, None] + depths[(cu[:-1, None] + j).clamp(max=s["q"].shape[0] - 1)])
    else:
        pos, at = first[:, None] + i, t
        see = ok[:, None, :] & (t[:, None, :] <= pos[..., None])
    if W > 0:
        see = see & ((at[:, None, :] > pos[..., None] - W) | (at[:, None, :] < S))
    z = torch.matmul(q, k.transpose(1, 2)).view(R, P, H, span).mul_(SCALE)
    z.masked_fill_(~see[:, :, None, :], -math.inf)
    m = z.amax(-1, keepdim=True).clamp(min=-1e30)
    z = z.sub_(m).exp_()
    l = z.sum(-1, keepdim=True)
    o = torch.matmul(z.view(R, P * H, span), k[..., :VAL]).view(R, P, H, VAL) / torch.where(l > 0, l, torch.ones_like(l))
    lse = (m + l.log()).squeeze(-1)
    real = i < new[:, None]
    return o[real].to(torch.bfloat16), lse[real]


def _step(s):
    """Ancestor masks and depths of the trees, the accepted paths, the lengths, blocks and rows after them."""
    dev, B, W = s["kv"].device, s["block"], s["window"]
    R, T, P, words, S = s["kv"].numel(), s["parents"].numel(), s["steps"], s["words"], -(-s["sinks"] // s["block"])
    kv, cu, table = s["kv"].long(), s["cu"].long(), s["table"].long()
    new = cu[1:] - cu[:-1]
    i = torch.arange(P, device=dev)
    real = i[None, :] < new[:, None]
    node = (cu[:-1, None] + i).clamp(max=T - 1)
    parent = torch.where(real, s["parents"].long()[node], torch.full_like(node, -1))
    # ancestors, itself among them, by squaring
    up = torch.eye(P, device=dev).expand(R, P, P).clone()
    up.scatter_(2, parent.clamp(min=0)[..., None], torch.where(parent >= 0, 1.0, up.gather(2, parent.clamp(min=0)[..., None])[..., 0])[..., None])
    for _ in range(max(1, P - 1).bit_length()):
        up = (torch.matmul(up, up) > 0).float()
    bits = torch.zeros(R, P, 32 * words, dtype=torch.int64, device=dev)
    bits[..., :P] = up.long()
    masks = (bits.view(R, P, words, 32) << torch.arange(32, device=dev)).sum(-1)
    masks = torch.where(masks >= 1 << 31, masks - (1 << 32), masks)
    depth = up.sum(-1).long() - 1
    drafted, chosen = s["drafted"].long()[node], s["chosen"].long()[node]
    agree = real & ((i == 0) | ((parent >= 0) & (drafted == chosen.gather(1, parent.clamp(min=0)))))
    held = real & ((up * (~agree)[:, None, :].float()).sum(-1) == 0) & (kv >= new)[:, None]
    d1 = torch.where(held, depth + 1, torch.zeros_like(depth))
    accepted = d1.amax(1)
    last = (d1 == accepted[:, None]).float().argmax(1)
    some = accepted > 0
    chain = up.gather(1, last[:, None, None].expand(R, 1, P))[:, 0].bool() & some[:, None]
    order = torch.where(chain, depth, torch.full_like(depth, P)).argsort(dim=1, stable=True)
    path = torch.where(i[None, :] < accepted[:, None], order, torch.full_like(order, -1))
    nxt = torch.where(some, chosen.gather(1, last[:, None])[:, 0], torch.full_like(last, -1))
    # lengths and blocks
    first = kv - new
    served = (new > 0) & (kv >= new)
    length = torch.where(served, first + accepted, s["lengths"].long())
    M, F = table.shape[1], s["ring"].numel()
    j = torch.arange(M, device=dev)[None, :]
    dead = lambda L: ((L - W + 1).clamp(min=0) // B).clamp(min=S) if W > 0 else torch.full_like(L, S)  # noqa: E731
    hi = torch.minimum(dead(length), -(-length // B))
    gone = served[:, None] & (((j >= dead(first)[:, None]) & (j < hi[:, None]))
                              | ((j >= -(-length // B)[:, None]) & (j < -(-kv // B)[:, None])))
    tail = s["bounds"][1]
    place = (tail + gone.reshape(-1).long().cumsum(0) - 1) % F
    ring = torch.cat([s["ring"].long(), s["ring"].new_zeros(1).long()])
    ring[torch.where(gone.reshape(-1), place, torch.full_like(place, F))] = table.reshape(-1)
    s["ring"].copy_(ring[:F])
    # rows of the accepted path, together behind the context
    slot = lambda t: table.gather(1, (t // B).clamp(0, M - 1)) * B + t % B  # noqa: E731
    move = (i[None, :] < accepted[:, None]) & (path != i[None, :])
    src, dst = slot(first[:, None] + path.clamp(min=0))[move], slot(first[:, None] + i)[move]
    bytes_of = {"bf16": [(1152, 0)], "f8": [(ROW, 0), (4, B * ROW)], "q4": [(ROW // 2, 0), (ROW // GROUP, B * ROW // 2)]}
    for layer in s["pools"].view(s["layers"], s["n_blocks"], -1):
        for width, at in bytes_of[s["format"]]:
            part = layer[:, at:at + width * B].unflatten(1, (B, width))
            part[dst // B, dst % B] = part[src // B, src % B]
    i32 = lambda x: x.to(torch.int32)  # noqa: E731
    return dict(masks=i32(masks[real]), depths=i32(depth[real]), path=i32(path[real]), accepted=i32(accepted),
                next=i32(nxt), lengths=i32(length), bounds=torch.stack([s["bounds"][0], tail + gone.sum()]),
                ring=s["ring"], pools=s["pools"])


def work(case):
    c = case
    if c["op"] == "rows":
        return {"bytes": c["rows"] * (2 * 1152 + 2 * 580 + 8.0), "flops": 0.0}
    kv, new = _lengths(c)
    R, T = c["requests"], float(new.sum())
    one = ROW_BYTES[c.get("format", "f8")]
    if c["op"] == "step":
        # trees, tokens, lengths in; masks, depths, paths, lengths out; about a quarter of the nodes' rows move
        return {"bytes": T * (12 + 8 + 4.0 * -(-c["new"] // 32)) + R * 28.0 + c["layers"] * one * T / 2, "flops": 0.0}
    W, S = c["window"], c["sinks"]
    pairs = rows = 0.0
    for L, n in zip(kv, new):
        low = max(0, L - n - W + 1) if W else 0
        rows += L - low + min(S, low)
        if c["op"] == "tree":  # the context, and about a logarithm of the nodes
            pairs += n * (L - n - low + min(S, low) + math.log2(n + 1))
        else:
            p = np.arange(L - n, L)
            at = np.maximum(0, p - W + 1) if W else np.zeros_like(p)
            pairs += (p + 1 - at + np.minimum(S, at)).sum()
    return {"bytes": rows * one + T * c["heads"] * (1152 + 1024 + 4.0), "flops": 2.0 * (ROW + VAL) * pairs * c["heads"]}


# ---- from the definitions, in 64 bits ---------------------------------------------------------

def exact(case, seed):
    c = case
    if c["op"] == "step":
        return None  # whole numbers only, and rows that are copied
    s = prepare(case, seed)
    if c["op"] == "rows":
        return _exact_rows(s)
    if 2.0 * 1088 * c["requests"] * c["new"] * c["heads"] * _span(c) > 6e12:
        return None  # more than about 20 seconds in 64 bits
    return _exact_attend(s)


def _exact_rows(s):
    x = s["rows"].double()
    grid = torch.arange(127, dtype=torch.uint8, device=x.device).view(torch.float8_e4m3fn).double()
    # the scale: the first power of two under which the largest element fits
    powers = torch.tensor([2.0 ** k for k in range(LOW, HIGH + 1)], dtype=torch.float64, device=x.device)
    e = torch.searchsorted(448.0 * powers, x.abs().amax(-1)).clamp(max=HIGH - LOW)
    f = powers[e][:, None]
    a = (x.abs() / f).clamp(max=448.0)
    hi = torch.searchsorted(grid, a.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    d = (grid[hi] - a) - (a - grid[lo])
    v = torch.where((d < 0) | ((d == 0) & (hi % 2 == 0)), grid[hi], grid[lo])
    return torch.where((s["slots"] >= 0)[:, None], v * f * torch.sign(x), torch.zeros_like(x))


def _exact_attend(s):
    """One request and a few tokens at a time: the formula over the rows that the token sees."""
    outs, lses = [], []
    kv, cu, W, S = s["kv"].tolist(), s["cu"].tolist(), s["window"], s["sinks"]
    for r in range(len(kv)):
        n = cu[r + 1] - cu[r]
        first = kv[r] - n
        t = torch.arange(kv[r], device=s["q"].device)
        if W:
            t = t[(t < S) | (t > first - W)]
        rows = _rows_at(s["pool"], s["format"], s["block"],
                        s["table"][r].long()[t // s["block"]] * s["block"] + t % s["block"]).double()
        place = t.clone()  # position of every row
        if s["op"] == "tree":
            depths = s["depths"][cu[r]:cu[r + 1]].long()
            drafted = t >= first
            place[drafted] = first + depths[t[drafted] - first]
        step = max(1, (1 << 25) // (len(t) * s["q"].shape[1]))
        for a in range(0, n, step):
            b = min(n, a + step)
            if s["op"] == "tree":
                p = first + depths[a:b, None]
                words = s["masks"][cu[r] + a:cu[r] + b].long() & 0xFFFFFFFF
                bits = ((words[:, :, None] // 2 ** torch.arange(32, device=t.device)) % 2).flatten(1)
                hidden = torch.zeros(b - a, len(t), dtype=torch.bool, device=t.device)
                hidden[:, drafted] = bits[:, t[drafted] - first] == 0
            else:
                p = (first + torch.arange(a, b, device=t.device))[:, None]
                hidden = t[None, :] > p
            if W:
                hidden = hidden | ((place[None, :] <= p - W) & (place[None, :] >= S))
            z = torch.einsum("phd,td->pht", s["q"][cu[r] + a:cu[r] + b].double(), rows) * SCALE
            z = z.masked_fill(hidden[:, None, :], -math.inf)
            lse = torch.logsumexp(z, -1)
            outs.append(torch.einsum("pht,td->phd", torch.exp(z - lse[..., None]), rows[:, :VAL]))
            lses.append(lse)
    return torch.cat(outs), torch.cat(lses)
