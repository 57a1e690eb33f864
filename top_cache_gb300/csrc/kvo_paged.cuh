// Shared by the kernels of the paged device cache (kvo_paged.cu,
// kvo_paged_attend.cu): the layout of its blocks.
//
// A row is 576 elements (latent 512, which is also the value | rope key 64);
// token t of a request is row t mod block_tokens of block table[t /
// block_tokens].  A block is
//   KVO_CACHE_BF16  [block_tokens][576] bf16
//   KVO_CACHE_Q4    [block_tokens][288] bytes of codes, then [block_tokens][36]
//                   bytes of scales: 36 groups of 16 elements, an element's
//                   value is its E2M1 code (element 2b in the low four bits of
//                   byte b, 2b + 1 in the high ones) times its group's E4M3
//                   scale.  The product has at most 6 significant bits, so it
//                   is exact in fp16 and in bf16.
//   KVO_CACHE_F8    [block_tokens][576] E4M3 codes, then [block_tokens] fp32
//                   scales, powers of two from 2^-32 to 2^32 (what is none of
//                   them reads as NaN); an element's value is its code times
//                   its row's scale: 4 significant bits, exact in bf16.
#pragma once

#include "kvo_internal.cuh"

namespace kvo {
namespace paged {

constexpr int kRow = 576;             // elements per row
constexpr int kVal = 512;             // value (latent) elements
constexpr int kGroup = 16;            // elements that share a scale
constexpr int kGroups = kRow / kGroup;
constexpr int kCodeBytes = kRow / 2;  // codes of one row
constexpr int kRowBytesQ4 = kCodeBytes + kGroups;
constexpr int kRowBytes16 = kRow * 2;
constexpr int kRowBytesF8 = kRow + 4;
constexpr int kScaleExp = 32;         // exponents of 8-bit rows' scales: -32 .. 32
constexpr int kMaxRequests = 4096;    // per call: the requests' arrays fit shared memory
constexpr int kMaxWorkers = 256;      // CTAs of the attention launch (one per SM)
constexpr int64_t kMaxTokens = (int64_t)1 << 30;  // tokens a block table reaches; rows of a pool are below 2^31

// Exclusive prefix sum over the CTA's threads (kThreads a multiple of 32, at
// most 1024); *total gets the sum.  `warp_sums`: 33 entries of shared memory.
template <int kThreads>
__device__ __forceinline__ int64_t block_exclusive_sum(int64_t v, int64_t* warp_sums, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // the last call's sums have been read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int64_t s = lane < kThreads / 32 ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(kFull, s, o);
      if (lane >= o) s += y;
    }
    if (lane < kThreads / 32) warp_sums[lane] = s;
  }
  __syncthreads();
  *total = warp_sums[kThreads / 32 - 1];
  return x - v + (warp > 0 ? warp_sums[warp - 1] : 0);
}

// Whether bits are the scale of an 8-bit row: a power of two within the limits.
__device__ __forceinline__ bool row_scale_valid(uint32_t bits) {
  return (bits & 0x807fffffu) == 0u && (bits >> 23) - (127u - kScaleExp) <= 2u * kScaleExp;
}

// Largest i in [0, n) with off[i] <= x (off non-decreasing, off[0] <= x).
__device__ __forceinline__ int segment_of(const int32_t* off, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (off[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

}  // namespace paged

// Launch-side structures.
struct PagedPlanArgs {
  const int32_t* lengths;     // [R]
  const int32_t* new_tokens;  // [R], < 0: the request ends
  int32_t R, B, M, window, sinks, ring_size, n_slots;
  int32_t* table;             // [R][M]
  int32_t* ring;              // [ring_size]
  const int64_t* ring_in;     // head, tail
  int64_t* ring_out;
  int32_t* lengths_out;       // [R]
  int32_t* kv_lens;           // [R]
  int32_t* cu_new;            // [R + 1]
  int32_t* slots;             // [n_slots]
  int32_t* status;            // [R]
};
struct PagedRowsArgs {
  uint8_t* pool;
  int64_t pool_rows;      // blocks * block_tokens
  int32_t B;
  const int32_t* slots;   // [n]
  int64_t n;
  uint16_t* rows;         // [n][576] bf16
};
struct PagedAttendArgs {
  const uint8_t* pool;
  int64_t n_blocks;
  int32_t B, M, R;
  int32_t b_shift;         // log2(B), -1 if B is no power of two
  const int32_t* table;    // [R][M]
  const int32_t* kv_lens;  // [R]
  const int32_t* cu;       // [R + 1]
  const uint16_t* q;       // [n_tokens][H][576]
  int32_t n_tokens, H;
  int32_t window, sinks;   // window 0: none
  const uint32_t* masks;   // [n_tokens][mask_words], null: causal order
  const int32_t* depths;   // [n_tokens] or null (no window)
  int32_t mask_words;
  float scale_log2;
  uint16_t* out;           // [n_tokens][H][512]
  float* lse;              // [n_tokens][H] or null
  uint32_t* status;        // error word
  uint64_t wait_ns;
  int32_t workers;         // CTAs of the attention launch
  int32_t device;
  bool few_tiles, own_list;  // the list is short; each CTA makes it for itself
  // workspace
  int32_t* head;           // listed, tiles, CTAs in use, shared tiles
  int32_t* tile_off;       // [R + 1] tiles before each request
  int2* tiles;             // [kListTiles] request, first row
  int2* start;             // [workers + 1] tile, unit
  int4* shared;            // [workers] first row; 2 rows + slot of the first CTA's part; first and last CTA
  float* part_ml;          // [workers][2][2][N]
  float* part_o;           // [workers][2][N][512]
};
cudaError_t launch_paged_plan(const PagedPlanArgs& a, cudaStream_t s);
// The cache's shape: KVO_OK, or the error that every call on a pool gives.
int check_paged_cache(const void* pool, int64_t n_blocks, int32_t block_tokens, int32_t format);
cudaError_t launch_paged_write(const PagedRowsArgs& a, int format, cudaStream_t s);
cudaError_t launch_paged_read(const PagedRowsArgs& a, int format, cudaStream_t s);
int paged_tile_rows(int n_requests, int n_tokens, int H);
size_t paged_attend_workspace(int n_requests, int n_tokens, int H, int workers);       // of this call
size_t paged_attend_workspace_most(int n_requests, int n_tokens, int H, int workers);  // of every call no larger
void paged_attend_carve(PagedAttendArgs& a, uint8_t* workspace);
cudaError_t launch_paged_attend(const PagedAttendArgs& a, int format, cudaStream_t s);
cudaError_t launch_paged_tree(const PagedAttendArgs& a, int N, bool q4, cudaStream_t s);  // kTree kernels
cudaError_t launch_paged_f8(const PagedAttendArgs& a, int N, cudaStream_t s);             // 8 bits

}  // namespace kvo
