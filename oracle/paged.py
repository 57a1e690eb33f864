"""Plain definitions of the paged device cache's operators, in Python and 64-bit numpy.

Block plan (requests one after another), 8-bit rows, draft trees, 4-bit rows (E2M1 codes, one E4M3 scale per 16
elements, both by exhaustive nearest value) and window attention (one query token at a
time over the tokens that it sees).  Test infrastructure; shares nothing with the kernels.
"""
import numpy as np

OK, ERANGE, ECAPACITY = 0, -3, -6
ROW, VAL, GROUP = 576, 512, 16


def bf16_values(bits):
    """float64 values of bf16 bit patterns."""
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def bf16_bits(x):
    """Nearest bf16 bits (ties to even) of values that are finite in float32 and exact there."""
    b = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)


def plan(lengths, new, block, table, ring, bounds, n_slots, window=0, sinks=0):
    """Returns dict(lengths, kv_lens, cu, slots, status, table, ring, bounds); inputs are not changed."""
    R, M = table.shape
    table, ring = table.copy(), ring.copy()
    head, tail = int(bounds[0]), int(bounds[1])
    F = len(ring)
    free = [int(ring[(head + i) % F]) for i in range(tail - head)]
    first_window_block = -(-sinks // block)

    def hidden(L):
        """Blocks that no position from L on sees."""
        if window == 0:
            return set()
        return {j for j in range(first_window_block, M) if (j + 1) * block - 1 < L - window + 1}

    out = dict(lengths=np.array(lengths, np.int32), kv_lens=np.zeros(R, np.int32), cu=np.zeros(R + 1, np.int32),
               slots=np.full(n_slots, -1, np.int32), status=np.zeros(R, np.int32))
    at = wanted = taken = 0
    released = []
    for r in range(R):
        L, n = int(lengths[r]), max(0, int(new[r]))
        begin, at = at, at + n
        out["cu"][r + 1] = at
        have, want = -(-L // block), -(-(L + n) // block)
        if L < 0 or L + n > M * block or (n > 0 and at > n_slots):
            out["status"][r] = ERANGE
            continue
        wanted += want - have
        if want > have and wanted > len(free):
            out["status"][r] = ECAPACITY
            continue
        for j in range(have, want):
            table[r, j] = free[taken]
            taken += 1
        if new[r] < 0:
            released += [int(table[r, j]) for j in range(have) if j not in hidden(L)]
            out["lengths"][r] = 0
        else:
            released += [int(table[r, j]) for j in range(want) if j in hidden(L + n) and j not in hidden(L)]
            out["lengths"][r] = out["kv_lens"][r] = L + n
        for i in range(n):
            b = int(table[r, (L + i) // block])
            out["slots"][begin + i] = b * block + (L + i) % block if 0 <= b and b * block + block <= 2 ** 31 else -1
    for i, b in enumerate(released):
        ring[(tail + i) % F] = b
    return dict(out, table=table, ring=ring, bounds=np.array([head + taken, tail + len(released)], np.int64))


_E4M3 = np.array([(m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
                  for e in range(16) for m in range(8)][:127])
_E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _nearest(x, grid):
    """Index of the nearest grid value, ties to the even index, beyond the last one the last."""
    d = np.abs(np.minimum(x, grid[-1])[..., None] - grid)
    low = d.argmin(-1)
    up = np.minimum(low + 1, len(grid) - 1)
    tie = np.take_along_axis(d, up[..., None], -1)[..., 0] == np.take_along_axis(d, low[..., None], -1)[..., 0]
    return np.where(tie & (up != low) & (low % 2 == 1), up, low)


def quantize(rows):
    """bf16 bits [n][576] -> (codes [n][576], scale bytes [n][36]); a group that is not finite: 0, 0x7f."""
    x = bf16_values(rows).reshape(-1, ROW // GROUP, GROUP)
    fine = np.isfinite(x).all(-1)
    x = np.where(fine[..., None], x, 0.0)
    sb = _nearest(np.abs(x).max(-1) / 6.0, _E4M3)
    s = _E4M3[sb]
    a = np.where(s[..., None] > 0, np.abs(x) / np.where(s > 0, s, 1.0)[..., None], 0.0)
    c = _nearest(a, _E2M1) | np.where((s[..., None] > 0) & np.signbit(x), 8, 0)
    return c.reshape(-1, ROW).astype(np.uint8), np.where(fine, sb, 0x7F).astype(np.uint8)


def dequantize(codes, scales):
    """float64 values [n][576]."""
    s = np.append(_E4M3, np.nan)[scales]
    v = np.append(_E2M1, -_E2M1)[codes].reshape(-1, ROW // GROUP, GROUP)
    return (v * s[..., None]).reshape(-1, ROW)


def pack_block(codes, scales):
    """One block's bytes from its rows' codes and scales."""
    c = codes.reshape(-1, 2)
    return np.concatenate([(c[:, 0] | (c[:, 1] << 4)).astype(np.uint8), scales.reshape(-1)])


def visible(p, window, sinks):
    """Tokens that position p sees."""
    t = np.arange(max(p, -1) + 1)
    return t if window == 0 else t[(t > p - window) | (t < sinks)]


def attend(rows_of, q, positions, scale, window=0, sinks=0):
    """Attention of query tokens q [T][H][576] (float64) of one request at `positions`.

    rows_of(t) -> (float64 rows [len(t)][576], mapped [len(t)]).  Returns out, lse, and for the tolerances
    sum_t w_t |v_t| and the largest |scale| sum_i |q_i k_ti| of a seen token per (token, head).
    """
    T, H = q.shape[:2]
    out, lse = np.zeros((T, H, VAL)), np.full((T, H), -np.inf)
    mag, dot, count = np.zeros((T, H, VAL)), np.zeros((T, H)), np.zeros(T, np.int64)
    for i, p in enumerate(positions):
        t = visible(int(p), window, sinks)
        if len(t) == 0:
            continue
        k, ok = rows_of(t)
        k = k[ok]
        count[i] = len(k)
        if len(k) == 0:
            continue
        with np.errstate(invalid="ignore", over="ignore"):
            z = scale * (q[i] @ k.T)
            m = z.max(-1, keepdims=True)
            w = np.exp(z - m)
            s = w.sum(-1, keepdims=True)
            out[i] = (w / s) @ k[:, :VAL]
            mag[i] = (w / s) @ np.abs(k[:, :VAL])
            dot[i] = abs(scale) * (np.abs(q[i]) @ np.abs(k).T).max(-1)
            lse[i] = (m + np.log(s))[:, 0]
    return out, lse, mag, dot, count


# ---- 8-bit rows -------------------------------------------------------------------------------

def quantize8(rows):
    """bf16 bits [n][576] -> (codes [n][576], scale bits [n] uint32); a row that is not finite: 0, a NaN."""
    x = bf16_values(rows)
    fine = np.isfinite(x).all(-1)
    x = np.where(fine[:, None], x, 0.0)
    top = np.abs(x).max(-1)
    exps = np.arange(-32, 33)
    fits = top[:, None] <= 448.0 * 2.0 ** exps
    e = np.where(fits.any(-1), exps[fits.argmax(-1)], 32)
    a = np.abs(x) / (2.0 ** e)[:, None]
    c = np.empty(a.shape, np.uint8)
    for i in range(0, len(a), 256):
        c[i:i + 256] = _nearest(a[i:i + 256], _E4M3)
    c |= np.where(fine[:, None] & (bf16_bits_sign(rows) != 0), 128, 0).astype(np.uint8)
    bits = (2.0 ** e).astype(np.float32).view(np.uint32)
    return c, np.where(fine, bits, 0x7FC00000).astype(np.uint32)


def bf16_bits_sign(bits):
    return np.asarray(bits, np.uint16) >> 15


def dequantize8(codes, scale_bits):
    """float64 values [n][576]; a scale that is no power of two from 2^-32 to 2^32 reads as NaN."""
    with np.errstate(invalid="ignore"):
        s = np.asarray(scale_bits, np.uint32).view(np.float32).astype(np.float64)
        m, e = np.frexp(np.where(np.isfinite(s), s, 0.0))
    s = np.where((m == 0.5) & (e - 1 >= -32) & (e - 1 <= 32), s, np.nan)
    grid = np.append(_E4M3, np.nan)
    with np.errstate(invalid="ignore"):
        return np.append(grid, -grid)[codes] * s[:, None]


def pack_block8(codes, scale_bits):
    """One block's bytes from its rows' codes and scales."""
    return np.concatenate([codes.reshape(-1), np.ascontiguousarray(scale_bits, np.uint32).view(np.uint8)])


# ---- draft trees ------------------------------------------------------------------------------

def ancestors(parents):
    """bool [n][n]: row i has i and its ancestors; a parent that is not before its node makes a root."""
    n = len(parents)
    a = np.zeros((n, n), bool)
    for i, p in enumerate(parents):
        if 0 <= p < i:
            a[i] = a[p]
        a[i, i] = True
    return a


def mask_words(a, words):
    """int32 words [n][words] of boolean rows."""
    b = np.zeros((len(a), 32 * words), np.uint8)
    b[:, :a.shape[1]] = a
    return np.packbits(b, axis=1, bitorder="little").view(np.int32).reshape(len(a), words)


def accept(parents, drafted, chosen):
    """The nodes of the longest path from node 0 whose drafts were chosen at their parents, the first of equals."""
    best, paths = [], {}
    for i, p in enumerate(parents):
        if i == 0:
            paths[0] = [0]
        elif 0 <= p < i and p in paths and drafted[i] == chosen[p]:
            paths[i] = paths[p] + [i]
        if i in paths and len(paths[i]) > len(best):
            best = paths[i]
    return best


def commit(lengths, kv_lens, new, accepted, block, table, ring, bounds, window=0, sinks=0):
    """(lengths, ring, bounds) after `accepted` of the `new` tokens of every request."""
    ring, out, back = ring.copy(), np.array(lengths, np.int32), []
    keep = -(-sinks // block)

    def hidden(L):
        return set() if window == 0 else {j for j in range(keep, table.shape[1]) if (j + 1) * block - 1 < L - window + 1}

    for r, n in enumerate(new):
        if n <= 0 or kv_lens[r] < n or kv_lens[r] > table.shape[1] * block:
            continue
        first = kv_lens[r] - n
        L = first + min(max(int(accepted[r]), 0), n)
        out[r] = L
        used = -(-L // block)
        back += [int(table[r, j]) for j in range(used) if j in hidden(L) and j not in hidden(first)]
        back += [int(table[r, j]) for j in range(used, -(-kv_lens[r] // block))]
    for i, b in enumerate(back):
        ring[(int(bounds[1]) + i) % len(ring)] = b
    return out, ring, np.array([bounds[0], bounds[1] + len(back)], np.int64)


def tree_seen(kv, n, masks, depths, t, window=0, sinks=0):
    """bool [n][len(t)]: which of the tokens t (rows' places) node i sees; masks bool [n][n]."""
    first = kv - n
    t = np.asarray(t)
    if first < 0:
        return np.zeros((n, len(t)), bool)
    depths = np.asarray(depths)
    see = np.zeros((n, len(t)), bool)
    for i in range(n):
        j = t - first
        own = j >= 0
        inside = np.clip(j, 0, n - 1)
        place = np.where(own, first + depths[inside], t)
        see[i] = ~own | ((j < n) & (j <= i) & np.asarray(masks)[i, inside])
        if window:
            see[i] &= (place > first + depths[i] - window) | (place < sinks)
    return see


def attend_seen(rows, q, seen, scale):
    """Attention of q [T][H][576] over rows [n][576], token i over those of seen[i].  Returns out, lse, and for the
    tolerances sum_t w_t |v_t|, the largest |scale| sum_i |q_i k_ti|, the seen rows' number and the weights [T][H][n]."""
    T, H = q.shape[:2]
    out, lse = np.zeros((T, H, VAL)), np.full((T, H), -np.inf)
    mag, dot, count = np.zeros((T, H, VAL)), np.zeros((T, H)), seen.sum(1)
    weights = np.zeros((T, H, len(rows)))
    for i in range(T):
        at = np.flatnonzero(seen[i])
        if len(at) == 0:
            continue
        k = rows[at]
        with np.errstate(invalid="ignore", over="ignore"):
            z = scale * (q[i] @ k.T)
            m = z.max(-1, keepdims=True)
            w = np.exp(z - m)
            s = w.sum(-1, keepdims=True)
            weights[i][:, at] = w / s
            out[i] = (w / s) @ k[:, :VAL]
            mag[i] = (w / s) @ np.abs(k[:, :VAL])
            dot[i] = abs(scale) * (np.abs(q[i]) @ np.abs(k).T).max(-1)
            lse[i] = (m + np.log(s))[:, 0]
    return out, lse, mag, dot, count, weights
