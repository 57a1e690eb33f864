// Draft trees over the paged device cache: ancestor masks, the accepted path,
// lengths and blocks after it, and its rows moved together.
//
// Node i of a request (its query tokens in order) has parent p < i, or is a
// root.  A warp closes a group of 32 nodes with five rounds of pointer doubling
// in registers: `anc` has the node's ancestors in its group, itself among them,
// `exit` the parent outside the group that the chain leaves it by.  The rest of
// a node's ancestors are those of its exit: at most one hop a group, instead of
// one a node.  All of it is latency (device time, 16 trees of 32 nodes; 251 of up to
// 61): masks 2.0 and 2.1 us, accept 2.6 and 2.9, commit 3.0 and 4.6, move 4.5 (8
// pools of 16 bits) and 6.6 (3 of 8 bits; looked up row by row it took 12.9).
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvo_paged.cuh"

namespace kvo {

using namespace paged;

namespace {

constexpr int kMaxNodes = 1024;  // nodes of a request: 32 words of a mask
constexpr int kTreeThreads = 128;

struct Tree {
  uint32_t anc[kMaxNodes];
  int16_t exit[kMaxNodes];
  uint32_t hit[kMaxNodes / 32];  // accept: nodes that agree with what was chosen at their parents
  uint32_t best;
};

// The request's nodes among the tokens; false: they are not all there.
__device__ __forceinline__ bool nodes_of(const int32_t* cu, int r, int n_tokens, int& first, int& n) {
  const int c0 = cu[r], c1 = cu[r + 1];
  first = min(max(c0, 0), n_tokens);
  n = min(max(c1, first), n_tokens) - first;
  return c0 >= 0 && c1 >= c0 && c1 <= n_tokens;
}
__device__ __forceinline__ int parent_of(const int32_t* parents, int first, int i) {
  const int p = __ldg(parents + first + i);
  return p >= 0 && p < i ? p : -1;
}
// Closes every group of n <= kMaxNodes nodes (all threads).  hit(i, p): see Tree.
template <typename Hit>
__device__ __forceinline__ void close_groups(Tree& t, const int32_t* parents, int first, int n, Hit hit) {
  const int lane = threadIdx.x & 31;
  for (int g = threadIdx.x >> 5; 32 * g < n; g += kTreeThreads / 32) {
    const int i = 32 * g + lane;
    const int p = i < n ? parent_of(parents, first, i) : -1;
    const uint32_t h = __ballot_sync(kFull, i < n && hit(i, p));
    uint32_t anc = 1u << lane;
    int up = p >= 32 * g ? p - 32 * g : lane;  // in the group; a group's root points to itself
#pragma unroll
    for (int k = 0; k < 5; ++k) {
      anc |= __shfl_sync(kFull, anc, up);
      up = __shfl_sync(kFull, up, up);
    }
    const int leave = __shfl_sync(kFull, p, up);
    t.anc[i] = anc;
    t.exit[i] = (int16_t)leave;
    if (lane == 0) t.hit[g] = h;
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------
// masks: one CTA a request, a thread a node.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kTreeThreads) tree_masks_kernel(const int32_t* parents, const int32_t* cu, int n_tokens,
                                                                  uint32_t* masks, int words, int32_t* depths,
                                                                  uint32_t* status) {
  __shared__ Tree t;
  int first, n;
  nodes_of(cu, blockIdx.x, n_tokens, first, n);
  const bool fits = n <= 32 * words;
  if (fits) close_groups(t, parents, first, n, [](int, int) { return false; });
  if (!fits && threadIdx.x == 0 && status) atomicOr(status, kErrPlan);
  for (int i = threadIdx.x; i < n; i += kTreeThreads) {
    uint32_t* row = masks + (int64_t)(first + i) * words;
    int cur = fits ? i : -1, count = 0;
    for (int w = words - 1; w >= 0; --w) {
      uint32_t bits = 0u;
      if (cur >= 32 * w) {
        bits = t.anc[cur];
        cur = t.exit[cur];
      }
      count += __popc(bits);
      row[w] = bits;
    }
    if (depths) depths[first + i] = max(count - 1, 0);
  }
}

// ---------------------------------------------------------------------------
// accept: one CTA a request.  A node is accepted when it and all its ancestors
// agree; the deepest accepted one ends the path, the first of equals.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kTreeThreads) tree_accept_kernel(const int32_t* parents, const int32_t* drafted,
                                                                   const int32_t* chosen, const int32_t* cu,
                                                                   const int32_t* kv_lens, int n_tokens, int32_t* path,
                                                                   int32_t* accepted, int32_t* next_tokens) {
  __shared__ Tree t;
  const int r = blockIdx.x;
  int first, n;
  bool fits = nodes_of(cu, r, n_tokens, first, n);
  fits = fits && n <= kMaxNodes && kv_lens[r] >= n;
  int a = 0, last = -1;
  if (fits && n > 0) {
    if (threadIdx.x == 0) t.best = 0u;
    close_groups(t, parents, first, n, [&](int i, int p) {
      return i == 0 || (p >= 0 && __ldg(drafted + first + i) == __ldg(chosen + first + p));
    });
    for (int i = threadIdx.x; i < n; i += kTreeThreads) {
      int count = 0;
      bool held = true;
      for (int cur = i; cur >= 0; cur = t.exit[cur]) {
        const uint32_t bits = t.anc[cur];
        held = held && (bits & ~t.hit[cur >> 5]) == 0u;
        count += __popc(bits);
      }
      if (held) atomicMax(&t.best, (uint32_t)count << 16 | (uint32_t)(kMaxNodes - i));
    }
    __syncthreads();
    a = (int)(t.best >> 16);
    last = kMaxNodes - (int)(t.best & 0xffffu);
    if (threadIdx.x < 32) {
      const int lane = threadIdx.x;
      int end = a;
      for (int cur = last; cur >= 0; cur = t.exit[cur]) {
        const uint32_t bits = t.anc[cur];
        end -= __popc(bits);
        if ((bits >> lane) & 1u) path[first + end + __popc(bits & ((1u << lane) - 1u))] = (cur & ~31) + lane;
      }
    }
  }
  for (int k = a + threadIdx.x; k < n; k += kTreeThreads) path[first + k] = -1;
  if (threadIdx.x == 0) {
    accepted[r] = a;
    if (next_tokens) next_tokens[r] = a > 0 ? chosen[first + last] : -1;
  }
}

// ---------------------------------------------------------------------------
// commit: one CTA.  Prefix sums of the blocks that every request gives back,
// then a flat list of them, as in the plan.
// ---------------------------------------------------------------------------
constexpr int kCommitThreads = 1024;

struct CommitArgs {
  const int32_t *lengths, *kv_lens, *cu, *accepted;
  int32_t R, B, M, window, sinks, ring_size;
  const int32_t* table;
  int32_t* ring;
  const int64_t* ring_in;
  int64_t* ring_out;
  int32_t* lengths_out;
};
// A request's blocks that go: out of the window [w0, w1), behind the accepted path [t0, t1).
struct Gone {
  int length, w0, w1, t0, t1;
  __device__ __forceinline__ int count() const { return w1 - w0 + t1 - t0; }
};
__device__ __forceinline__ int hidden_end(const CommitArgs& a, int L, int sb) {
  if (a.window <= 0) return sb;
  const int low = L - a.window + 1;
  return max(sb, low > 0 ? low / a.B : 0);
}
__device__ __forceinline__ Gone gone_of(const CommitArgs& a, int r) {
  const int64_t n = (int64_t)a.cu[r + 1] - a.cu[r];
  const int kv = a.kv_lens[r];
  Gone g{-1, 0, 0, 0, 0};
  if (n <= 0 || kv < n || (int64_t)kv > (int64_t)a.M * a.B) return g;
  const int before = kv - (int)n, sb = (a.sinks + a.B - 1) / a.B;
  g.length = before + (int)min(max((int64_t)a.accepted[r], (int64_t)0), n);
  g.t0 = (g.length + a.B - 1) / a.B;
  g.t1 = (kv + a.B - 1) / a.B;
  g.w0 = hidden_end(a, before, sb);
  g.w1 = max(g.w0, min(hidden_end(a, g.length, sb), g.t0));
  return g;
}
__global__ void __launch_bounds__(kCommitThreads) commit_paged_kernel(CommitArgs a) {
  __shared__ int64_t warp_sums[33];
  __shared__ int32_t rel[kMaxRequests];  // blocks given back before each request
  const int tid = threadIdx.x;
  const int64_t head = a.ring_in[0], tail = a.ring_in[1], F = a.ring_size;
  int64_t total = 0;
  for (int base = 0; base < a.R; base += kCommitThreads) {
    const int r = base + tid;
    Gone g{-1, 0, 0, 0, 0};
    if (r < a.R) g = gone_of(a, r);
    int64_t sum;
    const int64_t at = total + block_exclusive_sum<kCommitThreads>(g.count(), warp_sums, &sum);
    total += sum;
    if (r < a.R) {
      rel[r] = (int32_t)min(at, F);
      const int keep = a.lengths[r];
      a.lengths_out[r] = g.length >= 0 ? g.length : keep;
    }
  }
  __syncthreads();
  const int n_rel = (int)min(total, F);
  if (tid == 0) {
    a.ring_out[0] = head;
    a.ring_out[1] = tail + n_rel;
  }
  const int64_t tail0 = tail < 0 ? 0 : tail % F;
  for (int i = tid; i < n_rel; i += kCommitThreads) {
    const int r = segment_of(rel, a.R, i), nth = i - rel[r];
    const Gone g = gone_of(a, r);
    const int j = nth < g.w1 - g.w0 ? g.w0 + nth : g.t0 + nth - (g.w1 - g.w0);
    const int64_t at = tail0 + i;
    a.ring[at < F ? at : at - F] = a.table[(int64_t)r * a.M + j];
  }
}

// ---------------------------------------------------------------------------
// move: a CTA a request and pool.  Where the rows lie is found for many of them
// at once; then a thread has one piece of every row (16 bytes of codes, 4 of
// scales).  The path's nodes ascend and node path[k] lies at or behind place k,
// so rows go forward only: a batch's sources are read before its places are
// written, and no place of it is a later batch's source.  Threads share no bytes.
// ---------------------------------------------------------------------------
constexpr int kMoveThreads = 96;  // 72 pieces of a bf16 row; 37 of 8 bits; 27 of 4
constexpr int kMoveBatch = 8;

struct MoveArgs {
  uint8_t* pools;
  int64_t stride, n_blocks;
  int32_t B, M, n_tokens;
  const int32_t *table, *kv_lens, *cu, *path, *accepted;
  int32_t row_bytes, scale_bytes;  // of a row: codes (or elements), scales behind the block's codes
};
__global__ void __launch_bounds__(kMoveThreads) move_paged_kernel(MoveArgs a) {
  const int r = blockIdx.x;
  int first, n;
  if (!nodes_of(a.cu, r, a.n_tokens, first, n)) return;
  const int kv = a.kv_lens[r], count = min(a.accepted[r], n);
  if (count <= 0 || kv < n || (int64_t)kv > (int64_t)a.M * a.B) return;
  __shared__ int4 rows[kMoveThreads];  // from: cache block (-1: none moves), row in it; to
  const int before = kv - n, tid = threadIdx.x;
  const int wide = a.row_bytes / 16, narrow = a.scale_bytes / 4;
  const bool is_wide = tid < wide, mine = tid < wide + narrow;
  const int64_t block_bytes = (int64_t)a.B * (a.row_bytes + a.scale_bytes);
  const int32_t* table = a.table + (int64_t)r * a.M;
  uint8_t* pool = a.pools + (int64_t)blockIdx.y * a.stride;
  auto piece = [&](int blk, int in) -> uint8_t* {  // this thread's piece of a row
    uint8_t* base = pool + blk * block_bytes;
    return is_wide ? base + (int64_t)in * a.row_bytes + 16 * tid
                   : base + (int64_t)a.B * a.row_bytes + (int64_t)in * a.scale_bytes + 4 * (tid - wide);
  };
  for (int k0 = 0; k0 < count; k0 += kMoveThreads) {
    const int k = k0 + tid;
    int4 row = make_int4(-1, 0, 0, 0);
    const int p = k < count ? __ldg(a.path + first + k) : -1;
    if (p > k && p < n) {
      const int s = (before + p) / a.B, d = (before + k) / a.B;
      const int32_t bs = __ldg(table + s), bd = __ldg(table + d);
      if (bs >= 0 && (int64_t)bs < a.n_blocks && bd >= 0 && (int64_t)bd < a.n_blocks)
        row = make_int4(bs, before + p - s * a.B, bd, before + k - d * a.B);
    }
    rows[tid] = row;
    __syncthreads();
    const int some = min(kMoveThreads, count - k0);
    for (int j = 0; mine && j < some; j += kMoveBatch) {
      uint4 v[kMoveBatch];
#pragma unroll
      for (int i = 0; i < kMoveBatch; ++i) {
        if (j + i >= some || rows[j + i].x < 0) continue;
        const uint8_t* src = piece(rows[j + i].x, rows[j + i].y);
        if (is_wide)
          v[i] = *reinterpret_cast<const uint4*>(src);
        else
          v[i].x = *reinterpret_cast<const uint32_t*>(src);
      }
#pragma unroll
      for (int i = 0; i < kMoveBatch; ++i) {
        if (j + i >= some || rows[j + i].x < 0) continue;
        uint8_t* dst = piece(rows[j + i].z, rows[j + i].w);
        if (is_wide)
          *reinterpret_cast<uint4*>(dst) = v[i];
        else
          *reinterpret_cast<uint32_t*>(dst) = v[i].x;
      }
    }
    __syncthreads();
  }
}

int fail(int code, const char* msg) { return set_error(code, msg); }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
template <typename... P>
bool aligned4(const P*... p) {
  return (aligned(p, 4) && ...);
}
int launched(const char* what) {
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? KVO_OK : set_cuda_error(e, what);
}
int check_requests(int32_t n_requests, int32_t n_tokens) {
  if (n_requests < 1 || n_requests > kMaxRequests) return fail(KVO_EINVAL, "n_requests must be in 1 .. 4096");
  if (n_tokens < 0 || n_tokens >= 1 << 30) return fail(KVO_EINVAL, "n_tokens must be in 0 .. 2^30 - 1");
  return KVO_OK;
}
int check_table(int32_t block_tokens, int32_t max_blocks) {
  if (block_tokens < 8 || block_tokens > 65536 || block_tokens % 8 != 0)
    return fail(KVO_EINVAL, "block_tokens must be a multiple of 8 in 8 .. 65536");
  if (max_blocks < 1 || (int64_t)max_blocks * block_tokens > kMaxTokens)
    return fail(KVO_EINVAL, "max_blocks * block_tokens must be in 1 .. 2^30");
  return KVO_OK;
}

}  // namespace

}  // namespace kvo

extern "C" {

int kvo_tree_masks(const int32_t* parents, const int32_t* cu_tokens, int32_t n_requests, int32_t n_tokens, uint32_t* masks,
                   int32_t mask_words, int32_t* depths, uint32_t* status, void* stream) {
  using namespace kvo;
  const int rc = check_requests(n_requests, n_tokens);
  if (rc != KVO_OK) return rc;
  if (!cu_tokens || (n_tokens > 0 && (!parents || !masks))) return fail(KVO_EINVAL, "NULL argument");
  if (!aligned4(parents, cu_tokens, masks, depths, status)) return fail(KVO_EINVAL, "array not aligned to its elements");
  if (mask_words < 1 || mask_words > kMaxNodes / 32) return fail(KVO_EINVAL, "mask_words must be in 1 .. 32");
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (status) {
    const cudaError_t e = cudaMemsetAsync(status, 0, 4, s);
    if (e != cudaSuccess) return set_cuda_error(e, "tree masks status");
  }
  tree_masks_kernel<<<n_requests, kTreeThreads, 0, s>>>(parents, cu_tokens, n_tokens, masks, mask_words, depths, status);
  return launched("tree masks launch");
}

int kvo_tree_accept(const int32_t* parents, const int32_t* drafted, const int32_t* chosen, const int32_t* cu_tokens,
                    const int32_t* kv_lens, int32_t n_requests, int32_t n_tokens, int32_t* path, int32_t* accepted,
                    int32_t* next_tokens, void* stream) {
  using namespace kvo;
  const int rc = check_requests(n_requests, n_tokens);
  if (rc != KVO_OK) return rc;
  if (!cu_tokens || !kv_lens || !accepted || (n_tokens > 0 && (!parents || !drafted || !chosen || !path)))
    return fail(KVO_EINVAL, "NULL argument");
  if (!aligned4(parents, drafted, chosen, cu_tokens, kv_lens, path, accepted, next_tokens))
    return fail(KVO_EINVAL, "array not aligned to its elements");
  tree_accept_kernel<<<n_requests, kTreeThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      parents, drafted, chosen, cu_tokens, kv_lens, n_tokens, path, accepted, next_tokens);
  return launched("tree accept launch");
}

int kvo_paged_commit(const int32_t* lengths, const int32_t* kv_lens, const int32_t* cu_tokens, const int32_t* accepted,
                     int32_t n_requests, int32_t block_tokens, int32_t max_blocks, int32_t window, int32_t sinks,
                     const int32_t* block_table, int32_t* ring, int32_t ring_size, const int64_t* ring_in,
                     int64_t* ring_out, int32_t* lengths_out, void* stream) {
  using namespace kvo;
  if (!lengths || !kv_lens || !cu_tokens || !accepted || !block_table || !ring || !ring_in || !ring_out || !lengths_out)
    return fail(KVO_EINVAL, "NULL argument");
  if (!aligned4(lengths, kv_lens, cu_tokens, accepted, block_table, ring, lengths_out) || !aligned(ring_in, 8) ||
      !aligned(ring_out, 8))
    return fail(KVO_EINVAL, "array not aligned to its elements");
  int rc = check_requests(n_requests, 0);
  if (rc == KVO_OK) rc = check_table(block_tokens, max_blocks);
  if (rc != KVO_OK) return rc;
  if (ring_size < 1 || window < 0 || sinks < 0) return fail(KVO_EINVAL, "ring_size, window or sinks out of range");
  CommitArgs a{};
  a.lengths = lengths;
  a.kv_lens = kv_lens;
  a.cu = cu_tokens;
  a.accepted = accepted;
  a.R = n_requests;
  a.B = block_tokens;
  a.M = max_blocks;
  a.window = (int32_t)(window < kMaxTokens ? window : kMaxTokens);
  a.sinks = (int32_t)(sinks < kMaxTokens ? sinks : kMaxTokens);
  a.ring_size = ring_size;
  a.table = block_table;
  a.ring = ring;
  a.ring_in = ring_in;
  a.ring_out = ring_out;
  a.lengths_out = lengths_out;
  commit_paged_kernel<<<1, kCommitThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return launched("paged commit launch");
}

int kvo_paged_move(void* pools, int64_t pool_stride, int32_t n_pools, int64_t n_blocks, int32_t block_tokens, int32_t format,
                   const int32_t* block_table, int32_t max_blocks, const int32_t* kv_lens, const int32_t* cu_tokens,
                   int32_t n_requests, const int32_t* path, int32_t n_tokens, const int32_t* accepted, void* stream) {
  using namespace kvo;
  int rc = check_paged_cache(pools, n_blocks, block_tokens, format);
  if (rc == KVO_OK) rc = check_requests(n_requests, n_tokens);
  if (rc == KVO_OK) rc = check_table(block_tokens, max_blocks);
  if (rc != KVO_OK) return rc;
  if (!block_table || !kv_lens || !cu_tokens || !accepted || (n_tokens > 0 && !path)) return fail(KVO_EINVAL, "NULL argument");
  if (!aligned4(block_table, kv_lens, cu_tokens, path, accepted)) return fail(KVO_EINVAL, "array not aligned to its elements");
  if (n_pools < 1 || n_pools > 65535) return fail(KVO_EINVAL, "n_pools must be in 1 .. 65535");
  const int64_t bytes = kvo_paged_block_bytes(format, block_tokens) * n_blocks;
  if (n_pools > 1 && (pool_stride < bytes || pool_stride % 16 != 0))
    return fail(KVO_EINVAL, "pool_stride must be a multiple of 16 and no less than a pool");
  if (n_tokens == 0) return KVO_OK;
  MoveArgs a{};
  a.pools = static_cast<uint8_t*>(pools);
  a.stride = pool_stride;
  a.n_blocks = n_blocks;
  a.B = block_tokens;
  a.M = max_blocks;
  a.n_tokens = n_tokens;
  a.table = block_table;
  a.kv_lens = kv_lens;
  a.cu = cu_tokens;
  a.path = path;
  a.accepted = accepted;
  a.row_bytes = format == KVO_CACHE_BF16 ? kRowBytes16 : format == KVO_CACHE_Q4 ? kCodeBytes : kRow;
  a.scale_bytes = format == KVO_CACHE_BF16 ? 0 : format == KVO_CACHE_Q4 ? kGroups : 4;
  move_paged_kernel<<<dim3((unsigned)n_requests, (unsigned)n_pools), kMoveThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return launched("paged move launch");
}

}  // extern "C"
