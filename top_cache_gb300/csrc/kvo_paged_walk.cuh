// Shared by the attention kernels of the paged device cache: how the work is
// listed and split over the CTAs.
//
// Up to 2,048 tiles are listed with their blocks.  kTree: the query tokens are
// the nodes of a tree; a tile then walks the blocks that the causal order would
// give it, from the window of the context's end on (a node's position is its
// depth behind the context, at most its row's).
#pragma once

#include "kvo_paged_tc.cuh"

namespace kvo {
namespace paged {

constexpr int kBlk = 128;            // tokens per block of the walk: M of S^T, K of O^T
constexpr int kListTiles = 2048;     // most tiles that are listed, and may be split
constexpr int kTileCost = 1;         // a tile's own cost, in blocks (queries in, output out)
// Least units a CTA is given when the list is split.  Measured with 1, 2, 4 (16 heads, us): one request of 1k 12.0, 14.0,
// 16.3; of 4k 13.3, 15.0, 18.5; of 16k 18.2, 16.7, 19.7; of 64k 25.2 with each; 5 x 700 of 24 heads (4 bits) 23.0, 26.3,
// 32.6; 32 of 32k 152 with each.  1 writes and joins more parts: faster up to 4k, slower at 16k.
constexpr int kMinShare = 2;
// What splitting over `used` of the CTAs costs, in blocks' time: one more launch that does something, and the parts
// written and read (one or two of N x 2 KB a CTA).  Measured as nothing, as this, as four times this (us): 128 requests
// of 2k 68, 62, 62; 16 x 4 positions of 128 heads over a window of 4,096 108, 98, 97; a windowed chunk of 4,096 277, 279,
// 278; 100 requests of 2k 56, 56, 51; 40 x 2 positions of 64 heads of 2k (4 bits) 59, 58, 72; one request of 1k 14, 14, 24.
__device__ __forceinline__ int64_t split_cost(int N, int used, int workers) { return 2 + (int64_t)(N / 12) * used / workers; }

// ---- the work -------------------------------------------------------------------------------
// One tile, or the part of its blocks that this CTA has.
struct Seg {
  int r;                 // request
  int grow;              // first row of the tile among all (token, head) rows
  int row0, nrows;       // first row within the request, rows
  int pos0;              // position of the request's first query token
  int pmin, pmax;        // positions of the tile's first and last row; kTree: the context's last token, the last node's row
  int lo;                // window part starts here; tokens below a.sinks are seen by all positions at or past them
  int wlo, nsb;          // first block of the window part, blocks of the sinks before it
  int b0, b1;            // this CTA's blocks of the tile's list
  int part;              // -1: whole tile, else its partial slot
  __device__ __forceinline__ int block(int b) const { return b < nsb ? b : wlo + (b - nsb); }
  __device__ __forceinline__ bool any_sees(const PagedAttendArgs& a, int t) const {
    return t <= pmax && (t >= lo || t < a.sinks);
  }
};

// Fills all but the CTA's share; returns the tile's blocks.
template <bool kTree>
__device__ __forceinline__ int tile_of(const PagedAttendArgs& a, int N, int r, int row0, Seg& s) {
  const int c0 = min(max(a.cu[r], 0), a.n_tokens), c1 = min(max(a.cu[r + 1], c0), a.n_tokens);
  const int nq = c1 - c0;
  const int kv = (int)min((int64_t)max(a.kv_lens[r], 0), (int64_t)a.M * a.B);
  s.r = r;
  s.row0 = row0;
  s.nrows = min(N, nq * a.H - row0);
  s.grow = c0 * a.H + row0;
  s.pos0 = kv - nq;
  s.pmin = s.pos0 + row0 / a.H;
  s.pmax = s.pos0 + (row0 + s.nrows - 1) / a.H;
  s.lo = a.window > 0 ? max(0, s.pmin - a.window + 1) : 0;
  s.wlo = 0;
  s.nsb = 0;
  if (kTree) {
    s.pmin = s.pos0 - 1;
    s.lo = a.window > 0 ? max(0, s.pos0 - a.window + 1) : 0;  // (the root's window reaches furthest back)
    if (s.pos0 < 0) s.pmax = -1;                              // nodes whose rows are not all cached see nothing
  }
  if (s.pmax < 0) return 0;
  const int nsb = (min(a.sinks, s.pmax + 1) + kBlk - 1) / kBlk;
  const int wlo = s.lo / kBlk;
  if (nsb < wlo) {
    s.nsb = nsb;
    s.wlo = wlo;
  }
  return s.nsb + s.pmax / kBlk - s.wlo + 1;
}
__device__ __forceinline__ int request_rows(const PagedAttendArgs& a, int r) {
  const int c0 = min(max(a.cu[r], 0), a.n_tokens), c1 = min(max(a.cu[r + 1], c0), a.n_tokens);
  return (c1 - c0) * a.H;
}

// Parts of the workspace header.
constexpr int kHdListed = 0, kHdTiles = 1, kHdWorkers = 2, kHdShared = 3;

// The list of tiles, built by a kernel of its own or, if it is short, by every CTA of the attention kernel for itself.
constexpr int kOwnTiles = 256;     // most tiles (and requests) of a list that each CTA builds
struct List {
  int32_t off[kOwnTiles + 1];      // tiles before each request
  int32_t before[kOwnTiles];       // units before each tile
  int64_t warp_sums[33];
  int64_t units;
  int32_t n_tiles, used, n_shared, most;
};

// Tiles per request; if they are few, the units before each, and how many CTAs share them evenly (0: each tile goes to
// one CTA whole).  kThreads threads call it; `off` holds R + 1, `before` kMost entries.  publish: what the attention and
// the join read is written to the workspace.
constexpr int64_t kNoList = (int64_t)1 << 32;  // counted for a request whose tokens or length are not what they may be
// Its tokens end before they start, or its cache ends behind its block table, or tokens that see something lie outside
// the queries: cut to what fits, its positions would be others.  (A plan counts the tokens of refused requests, which
// may pass the queries; they see nothing.)
__device__ __forceinline__ bool misplaced(const PagedAttendArgs& a, int r) {
  const int c0 = a.cu[r], c1 = a.cu[r + 1], kv = a.kv_lens[r];
  return c1 < c0 || (int64_t)kv > (int64_t)a.M * a.B || (kv > 0 && c1 > c0 && (c0 < 0 || c1 > a.n_tokens));
}
template <int kThreads, int kMost, bool kTree>
__device__ __forceinline__ void build_list(const PagedAttendArgs& a, int N, int32_t* off, int32_t* before, List& t,
                                           bool publish) {
  const int tid = threadIdx.x;
  int64_t total = 0, sum;
  if (tid == 0) t.n_shared = t.most = 0;
  for (int base = 0; base < a.R; base += kThreads) {
    const int r = base + tid;
    int64_t n = 0;
    if (r < a.R) n = misplaced(a, r) ? kNoList : (request_rows(a, r) + N - 1) / N;
    const int64_t at = total + block_exclusive_sum<kThreads>(n, t.warp_sums, &sum);
    if (r < a.R) off[r] = (int32_t)at;
    total += sum;
  }
  const bool valid = total < kNoList;  // (else off is not what it says, and nothing reads it)
  const int n_tiles = valid ? (int)total : 0;
  if (tid == 0) {
    off[a.R] = n_tiles;
    t.n_tiles = n_tiles;
    t.used = 0;
    if (publish) {
      a.head[kHdListed] = 0;
      a.head[kHdTiles] = n_tiles;
      *a.status = valid ? 0u : kErrPlan;
    }
  }
  __syncthreads();
  if (n_tiles > kMost) return;
  constexpr int kPer = (kMost + kThreads - 1) / kThreads;  // tiles of a thread, side by side
  int cost[kPer], grow[kPer], nrows[kPer];
  int64_t mine = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int i = kPer * tid + k;
    cost[k] = grow[k] = nrows[k] = 0;
    if (i < n_tiles) {
      const int r = segment_of(off, a.R, i);
      Seg s;
      const int nblk = tile_of<kTree>(a, N, r, (i - off[r]) * N, s);
      cost[k] = nblk + kTileCost;
      grow[k] = s.grow;
      nrows[k] = s.nrows;
      atomicMax(&t.most, cost[k]);
      if (publish) a.tiles[i] = make_int2(r, s.row0);
    }
    mine += cost[k];
  }
  // at most kListTiles tiles of at most 2^23 + 1 units: a sum past 2^31, which `before` does not hold, is not split
  int64_t units, at = block_exclusive_sum<kThreads>(mine, t.warp_sums, &units);
  const int64_t at0 = at;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if (kPer * tid + k < kMost) before[kPer * tid + k] = (int32_t)at;
    at += cost[k];
  }
  const int64_t share = max((int64_t)kMinShare, (units + a.workers - 1) / a.workers);
  const int used = (int)min((int64_t)a.workers, (units + share - 1) / share);
  __syncthreads();
  // whole tiles, if the longest of them for every round take no longer than even shares and what joining them costs
  if (units > INT32_MAX ||
      (int64_t)((n_tiles + a.workers - 1) / a.workers) * t.most <=
      (units + used - 1) / max(used, 1) + split_cost(N, used, a.workers))
    return;
  if (tid == 0) {
    t.used = used;
    t.units = units;
  }
  if (publish) {
    // the CTAs of a tile's first and last block; the first one's part lies in slot 1 if it also has the tile's own unit
    at = at0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (cost[k] > kTileCost) {
        const int w0 = (int)(((at + kTileCost + 1) * used - 1) / units), w1 = (int)(((at + cost[k]) * used - 1) / units);
        if (w1 > w0)
          a.shared[atomicAdd(&t.n_shared, 1)] =
              make_int4(grow[k], 2 * nrows[k] + ((int64_t)w0 * units / used <= at ? 1 : 0), w0, w1);
      }
      at += cost[k];
    }
  }
  __syncthreads();
  if (publish && tid == 0) {
    a.head[kHdListed] = 1;
    a.head[kHdWorkers] = used;
    a.head[kHdShared] = t.n_shared;
  }
}
// Where CTA w's even share starts: the tile and the unit in it.
__device__ __forceinline__ int2 share_start(const int32_t* before, int n_tiles, int64_t units, int used, int w) {
  if (w >= used) return make_int2(n_tiles, 0);
  const int64_t u = (int64_t)w * units / used;
  const int i = segment_of(before, n_tiles, (int)u);
  return make_int2(i, (int)(u - before[i]));
}

// The segments of one CTA, in order; every warp that walks them calls next()
// with all lanes.  `t`: the CTA's own list (a.own_list).
template <int N, bool kOwn, bool kTree>
struct Walk {
  bool listed;
  int tile, unit, end_tile, end_unit, n_tiles;
  __device__ __forceinline__ void begin(const PagedAttendArgs& a, const List& t) {
    const bool own = kOwn && a.own_list;
    listed = own ? t.used > 0 : a.head[kHdListed] != 0;
    n_tiles = own ? t.n_tiles : a.head[kHdTiles];
    tile = (int)blockIdx.x;
    unit = 0;
    end_tile = n_tiles;
    end_unit = 0;
    if (listed) {
      const int used = own ? t.used : a.head[kHdWorkers], w = min((int)blockIdx.x, used), w1 = min(w + 1, used);
      const int2 s = own ? share_start(t.before, n_tiles, t.units, used, w) : a.start[w];
      const int2 e = own ? share_start(t.before, n_tiles, t.units, used, w1) : a.start[w1];
      tile = s.x;
      unit = s.y;
      end_tile = e.x;
      end_unit = e.y;
    }
  }
  __device__ __forceinline__ bool next(const PagedAttendArgs& a, const List& t, Seg& s) {
    const bool own = kOwn && a.own_list;
    if (!listed) {
      if (tile >= n_tiles) return false;
      int lo = 0;
      if (own) {
        lo = segment_of(t.off, a.R, tile);
      } else {
        // request of the tile: 32-way search in tile_off
        const int lane = threadIdx.x & 31;
        int hi = a.R;
        while (hi - lo > 1) {
          const int step = (hi - lo + 31) / 32, i = min(lo + (lane + 1) * step, hi);
          const int below = __popc(__ballot_sync(kFull, i < hi && a.tile_off[i] <= tile));
          hi = min(lo + (below + 1) * step, hi);
          lo = lo + below * step;
        }
      }
      s.b1 = tile_of<kTree>(a, N, lo, (tile - (own ? t.off[lo] : a.tile_off[lo])) * N, s);
      s.b0 = 0;
      s.part = -1;
      tile += (int)gridDim.x;
      return true;
    }
    while (tile < end_tile || (tile == end_tile && unit < end_unit)) {
      int r, row0;
      if (own) {
        r = segment_of(t.off, a.R, tile);
        row0 = (tile - t.off[r]) * N;
      } else {
        const int2 d = a.tiles[tile];
        r = d.x;
        row0 = d.y;
      }
      const int nblk = tile_of<kTree>(a, N, r, row0, s);
      const int last = tile == end_tile ? end_unit : nblk + kTileCost;
      s.b0 = max(unit - kTileCost, 0);
      s.b1 = max(last - kTileCost, 0);
      const bool first = unit < kTileCost;  // has the tile's own unit
      s.part = s.b0 == 0 && s.b1 == nblk ? -1 : (first ? 1 : 0);
      ++tile;
      unit = 0;
      if (s.b0 < s.b1 || (nblk == 0 && first)) return true;
    }
    return false;
  }
};

// Entry of a request's block table that token t is in.
__device__ __forceinline__ int entry_of(const PagedAttendArgs& a, int t) { return a.b_shift >= 0 ? t >> a.b_shift : t / a.B; }
// Token t's row of the pool (-1: its block is not mapped).
__device__ __forceinline__ int64_t pool_row(const PagedAttendArgs& a, const int32_t* table, int t) {
  const int j = entry_of(a, t);
  const int32_t b = __ldg(table + j);
  return b < 0 || (int64_t)b >= a.n_blocks ? -1 : (int64_t)b * a.B + (t - j * a.B);
}

// ---- trees ------------------------------------------------------------------------------
// Depth of node i of the segment's request: at most its row's place, so that its window reaches no further back than
// the root's and no further forward than its own row.
__device__ __forceinline__ int node_depth(const PagedAttendArgs& a, const Seg& s, int i) {
  const int n0 = (s.grow - s.row0) / a.H;  // the request's first query token
  return min(max(__ldg(a.depths + n0 + i), 0), i);
}
// Bit c: row c of NC (node node[c], position pos[c]) sees token t.  A token of the context is seen unless it is out of the
// window; node j by the nodes at or behind it whose mask has bit j.
template <int NC>
__device__ __forceinline__ uint32_t tree_sees(const PagedAttendArgs& a, const Seg& s, int t, const int32_t* pos,
                                              const int32_t* node) {
  const int j = t - s.pos0;
  const int place = j >= 0 && a.depths ? s.pos0 + node_depth(a, s, j) : t;
  const int reach = a.window == 0 || place < a.sinks ? 0x7fffffff : a.window;  // seen from positions below place + reach
  const int64_t n0 = (s.grow - s.row0) / a.H;
  const bool listed = j < 32 * a.mask_words;
  const uint32_t* words = a.masks + n0 * a.mask_words + (j >> 5);
  uint32_t vis = 0u, word = 0u;
  int last = -1;
#pragma unroll 1
  for (int c = 0; c < NC; ++c) {
    const int i = node[c];
    bool see = pos[c] - place < reach;
    if (j >= 0) {
      if (i != last && listed && j <= i) word = __ldg(words + (int64_t)i * a.mask_words);  // (rows of a node stand together)
      last = i;
      see = see && listed && j <= i && ((word >> (j & 31)) & 1u);
    }
    vis |= (uint32_t)see << c;
  }
  return vis;
}

// Rounds a size up to 256.
inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// A launch whose set-up may overlap the last one's end (it calls grid_wait before it reads anything).
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), int grid, int threads, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)grid);
  c.blockDim = dim3((unsigned)threads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  c.attrs = &at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, args...);
}

}  // namespace paged

cudaError_t launch_paged_schedule(const PagedAttendArgs& a, int N, cudaStream_t s);
cudaError_t launch_paged_join(const PagedAttendArgs& a, int N, float bias, cudaStream_t s);

}  // namespace kvo
