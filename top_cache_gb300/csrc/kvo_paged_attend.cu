// Attention over the paged device cache: the calls' dispatch, the list of tiles
// and the join of partial results; the kernel over 16 and 4 bits
// (kvo_paged_attend.cuh) with tokens in causal order.
#include "kvo_paged_attend.cuh"

namespace kvo {

namespace {

// ---------------------------------------------------------------------------
// schedule: the list of a call where the attention's CTAs do not make it, one
// CTA; as many threads as a short list has tiles (4.7 us for 128 tiles of 16
// requests; 1,024 threads 6.5).
// ---------------------------------------------------------------------------
constexpr int kSchedThreads = 1024;

template <int kThreads, int kTiles, int kRequests, bool kTree>
__global__ void __launch_bounds__(kThreads) schedule_paged_kernel(PagedAttendArgs a, int N) {
  __shared__ List t;
  __shared__ int32_t off[kRequests + 1], before[kTiles];
  launch_dependents();
  build_list<kThreads, kTiles, kTree>(a, N, off, before, t, true);
  __syncthreads();
  for (int r = threadIdx.x; r <= a.R; r += kThreads) a.tile_off[r] = off[r];
  if (t.used > 0)
    for (int w = threadIdx.x; w <= t.used; w += kThreads) a.start[w] = share_start(before, t.n_tiles, t.units, t.used, w);
}

// ---------------------------------------------------------------------------
// join: the parts of a tile that several CTAs share, in a fixed order.  A warp
// has a row, or with few rows (one long request) up to eight warps do: each sums
// every eighth part, and they meet in shared memory.  Latency bound: the list,
// the parts' (m, l) and the parts themselves are read one after another, and the
// kernel's code is cold.  So the loop over the parts stays short: 8,192 rows in 280
// parts of 64, 36 MB, 5.6 us (two parts a turn 7.8, four 7.4); 512 rows 4.8 us (6.7,
// 7.3).  A CTA of 512 threads per four rows, with the weights in shared memory,
// took 11.5 and 8.4 us; an empty list takes 1.8.  Teams where there are more warps
// than rows: 16 rows of 64k tokens 9.0 us, a warp a row 40; 128 rows of 256k (4
// bits) 8.5 and 31.9; 8,192 rows 5.6 and 5.4 (no team there).
// ---------------------------------------------------------------------------
constexpr int kJoinWarps = 8;
constexpr int kJoinThreads = kJoinWarps * 32;
constexpr int kJoinParts = 256;  // most parts of a row
static_assert(kMaxWorkers <= kJoinParts, "a tile has a part of every CTA at most");

template <int N>
__global__ void __launch_bounds__(kJoinThreads) join_paged_kernel(PagedAttendArgs a, float bias) {
  __shared__ float4 acc[kJoinWarps][kVal / 4];
  constexpr int kPer = kJoinParts / 32, kCols = kVal / 4 / 32;  // parts, float4s of a lane
  grid_wait();
  if (a.head[kHdListed] == 0) return;
  const int warp = (int)threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int items = a.head[kHdShared] * N;
  int team = kJoinWarps;  // warps of a row
  while (team > 1 && items * team > kJoinWarps * (int)gridDim.x) team >>= 1;
  const int member = warp & (team - 1), rows = kJoinWarps / team;
  for (int first = (int)blockIdx.x * rows; first < items; first += (int)gridDim.x * rows) {
    const int mine = first + warp / team, item = min(mine, items - 1), row = item % N;
    const int4 sh = a.shared[item / N];  // first row, 2 rows + slot of the first CTA's part (0 for the others), CTAs
    const bool in = row < (sh.y >> 1) && mine < items;
    const int n = in ? sh.w - sh.z + 1 : 0;  // at most the CTAs of the launch
    auto slot = [&](int k) -> int64_t { return (int64_t)(sh.z + k) * 2 + (k == 0 ? sh.y & 1 : 0); };
    // the weight of every part: 2^(m - largest m), and the sum of their l
    float f[kPer], g[kPer], m = kNone, l = 0.f;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int k = 32 * j + lane;
      f[j] = kNone;
      g[j] = 0.f;
      if (k < n) {
        const float* ml = a.part_ml + slot(k) * 2 * N + row;
        f[j] = ml[0];
        g[j] = ml[N];
      }
      m = fmaxf(m, f[j]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      f[j] = ex2(f[j] - m);
      l += f[j] * g[j];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(kFull, l, o);
    float4 x[kCols];
#pragma unroll
    for (int c = 0; c < kCols; ++c) x[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int end = min(32, n - 32 * j);
#pragma unroll 1
      for (int k = member; k < end; k += team) {
        const float4* src = reinterpret_cast<const float4*>(a.part_o + (slot(32 * j + k) * N + row) * kVal) + lane;
        const float w = __shfl_sync(kFull, f[j], k);
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          const float4 y = src[32 * c];
          x[c].x += w * y.x;
          x[c].y += w * y.y;
          x[c].z += w * y.z;
          x[c].w += w * y.w;
        }
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint2* out = reinterpret_cast<uint2*>(a.out + ((int64_t)sh.x + row) * kVal);
    auto store = [&](int col, float4 y) {
      const __nv_bfloat162 h0 = __floats2bfloat162_rn(y.x * inv, y.y * inv), h1 = __floats2bfloat162_rn(y.z * inv, y.w * inv);
      out[col] = make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
    };
    if (in && a.lse && member == 0 && lane == 0)
      a.lse[sh.x + row] = l == 0.f ? -INFINITY : (m - bias + log2f(l)) * 0.6931471805599453f;
    if (team == 1) {
#pragma unroll
      for (int c = 0; c < kCols; ++c)
        if (in) store(32 * c + lane, x[c]);
    } else {
#pragma unroll
      for (int c = 0; c < kCols; ++c) acc[warp][32 * c + lane] = x[c];
      __syncthreads();
      for (int col = 32 * member + lane; in && col < kVal / 4; col += 32 * team) {
        float4 y = acc[warp - member][col];
        for (int k = 1; k < team; ++k) {
          const float4 z = acc[warp - member + k][col];
          y.x += z.x;
          y.y += z.y;
          y.z += z.z;
          y.w += z.w;
        }
        store(col, y);
      }
      __syncthreads();  // the next rows take these ones' place
    }
  }
}

}  // namespace

// Rows per tile: the mean rows of a request, up to 64.  Measured, 16 requests of 32k, us with tiles of 16, 32, 64 rows:
// 16 rows 111, 115, 120 (4 bits 93, 119, 131); 24 rows 205, 116, 120 (161, 119, 132); 48 rows 297, 210, 123 (228, 210,
// 136); 128 rows 756, 396, 223 (572, 390, 237).  One height for uneven requests is the best of the three, or within 2 %
// of it, but short of two calls: 255 decode requests of 8k with a chunk of 512 tokens, 16 heads (mean 48 rows), 662, 529,
// 524 (4 bits 866, 774, 640), apart 406 + 152 (322 + 205); 300 of 2k with a chunk of 200 (mean 32) 265, 201, 197, apart
// 134 + 72.
int paged_tile_rows(int n_requests, int n_tokens, int H) {
  const int64_t rows = ((int64_t)n_tokens + n_requests - 1) / n_requests * H;
  return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}
// With tiles of N rows.
static size_t workspace_of(size_t N, int n_requests, int workers) {
  const size_t W = (size_t)workers;
  return 256 + up256(((size_t)n_requests + 1) * 4) + up256(kListTiles * sizeof(int2)) + up256((W + 1) * sizeof(int2)) +
         up256(W * sizeof(int4)) + up256(W * 4 * N * 4) + W * 2 * N * kVal * 4;
}
size_t paged_attend_workspace(int n_requests, int n_tokens, int H, int workers) {
  return workspace_of((size_t)paged_tile_rows(n_requests, n_tokens, H), n_requests, workers);
}
// The tiles are highest where one request has all tokens.
size_t paged_attend_workspace_most(int n_requests, int n_tokens, int H, int workers) {
  return workspace_of((size_t)paged_tile_rows(1, n_tokens, H), n_requests, workers);
}
void paged_attend_carve(PagedAttendArgs& a, uint8_t* w) {
  const size_t N = (size_t)paged_tile_rows(a.R, a.n_tokens, a.H), W = (size_t)a.workers;
  a.head = reinterpret_cast<int32_t*>(w);
  if (!a.status) a.status = reinterpret_cast<uint32_t*>(w + 64);
  w += 256;
  a.tile_off = reinterpret_cast<int32_t*>(w);
  w += up256(((size_t)a.R + 1) * 4);
  a.tiles = reinterpret_cast<int2*>(w);
  w += up256(kListTiles * sizeof(int2));
  a.start = reinterpret_cast<int2*>(w);
  w += up256((W + 1) * sizeof(int2));
  a.shared = reinterpret_cast<int4*>(w);
  w += up256(W * sizeof(int4));
  a.part_ml = reinterpret_cast<float*>(w);
  w += up256(W * 4 * N * 4);
  a.part_o = reinterpret_cast<float*>(w);
}
cudaError_t launch_paged_schedule(const PagedAttendArgs& a, int N, cudaStream_t s) {
  if (a.masks) {
    if (a.few_tiles)
      schedule_paged_kernel<kOwnTiles, kOwnTiles, kOwnTiles, true><<<1, kOwnTiles, 0, s>>>(a, N);
    else
      schedule_paged_kernel<kSchedThreads, kListTiles, kMaxRequests, true><<<1, kSchedThreads, 0, s>>>(a, N);
  } else if (a.few_tiles) {
    schedule_paged_kernel<kOwnTiles, kOwnTiles, kOwnTiles, false><<<1, kOwnTiles, 0, s>>>(a, N);
  } else {
    schedule_paged_kernel<kSchedThreads, kListTiles, kMaxRequests, false><<<1, kSchedThreads, 0, s>>>(a, N);
  }
  return cudaGetLastError();
}
cudaError_t launch_paged_join(const PagedAttendArgs& a, int N, float bias, cudaStream_t s) {
  const int grid = 4 * a.workers;
  return N == 16   ? launch_after(join_paged_kernel<16>, grid, kJoinThreads, 0, s, a, bias)
         : N == 32 ? launch_after(join_paged_kernel<32>, grid, kJoinThreads, 0, s, a, bias)
                   : launch_after(join_paged_kernel<64>, grid, kJoinThreads, 0, s, a, bias);
}
cudaError_t launch_paged_attend(const PagedAttendArgs& args, int format, cudaStream_t s) {
  const bool q4 = format == KVO_CACHE_Q4, f8 = format == KVO_CACHE_F8;
  PagedAttendArgs a = args;
  const int N = paged_tile_rows(a.R, a.n_tokens, a.H);
  // A list that is short whatever the requests' shares of the tokens are is built by each CTA: no launch before the
  // attention.  Measured, 16 heads: one request of 4k 15.0 us, with the kernel that lists 17.7; 64 of 1k 22.0 and 24.0; at
  // the limit, 128 of 1k 37.5 and 41.2, one chunk of 1,016 tokens 144.6 and 150.6.
  a.few_tiles = a.R <= kOwnTiles && a.R + ((int64_t)a.n_tokens * a.H + N - 1) / N <= kOwnTiles;
  a.own_list = !((q4 || f8) && N == 64) && a.few_tiles;  // (8 bits: no room in shared memory)
  if (a.n_tokens == 0) return cudaMemsetAsync(a.status, 0, 4, s);
  if (f8) return launch_paged_f8(a, N, s);
  if (a.masks) return launch_paged_tree(a, N, q4, s);
  return launch_attend<false>(a, N, q4, s);
}

}  // namespace kvo
