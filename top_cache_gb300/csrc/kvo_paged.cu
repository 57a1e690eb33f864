// Paged device cache: block tables and slot maps built on the GPU, rows written
// into the cache (16 bits, or quantized to 8 or 4) and read back.  Layout of a block:
// kvo_paged.cuh.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "kvo_paged.cuh"

namespace kvo {

using namespace paged;

namespace {

constexpr int kPlanThreads = 1024;

// Every thread of the launch (one CTA, or a cluster).
__device__ __forceinline__ void plan_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// First block that a position at or after length L can still see behind the
// sinks' blocks: blocks [sb, dead_end(L)) are seen by none.
__device__ __forceinline__ int dead_end(int L, int B, int window, int sb) {
  if (window <= 0) return sb;
  const int low = L - window + 1;  // lowest visible token of position L
  return max(sb, low > 0 ? low / B : 0);
}

// ---------------------------------------------------------------------------
// plan: one CTA, or a cluster of kPlanCtas when there are many slots to write.
// Each CTA reads the requests and prefix-sums their needs (new tokens, new
// blocks, released blocks) for itself; after a barrier (outputs may be the
// inputs) the flat lists of new blocks, slots and released blocks are shared
// out over all threads, each entry finding its request by a search in the
// prefix arrays (shared memory).  A few KB to a few hundred KB are moved, so
// latency is all it costs (device time, L2 warm): 5.3 us for 16 requests, 11.4
// for 509 requests of 61 new tokens at most, windowed, with 31,054 slots (13.3
// with a cold L2; one CTA 37).
// ---------------------------------------------------------------------------
constexpr int kPlanCtas = 8;
constexpr int kPlanSlots = 1024;  // slots that one CTA writes alone (1,029: 5.7 us, with eight 5.6; 4,101: 7.6 and 5.4)

constexpr size_t plan_smem(int R) { return (5 * (size_t)R + 2) * 4; }  // bytes of the prefix arrays

__global__ void __launch_bounds__(kPlanThreads) plan_paged_kernel(PagedPlanArgs a) {
  extern __shared__ int32_t sm[];
  __shared__ int64_t warp_sums[33];
  __shared__ int32_t taken;
  const int R = a.R, B = a.B;
  int32_t* cu = sm;              // [R + 1] new tokens before each request
  int32_t* nb = cu + R + 1;      // [R] new blocks before each request
  int32_t* rel = nb + R;         // [R + 1] released blocks before each request
  int32_t* old = rel + R + 1;    // [R] cached tokens; -1: refused
  int32_t* ends = old + R;       // [R] 1: the request ends
  const int tid = threadIdx.x, cta = blockIdx.x;
  const uint32_t flat = cta * kPlanThreads + tid, step = kPlanThreads * gridDim.x;  // unsigned: 2^31 entries and a step pass an int
  const int sb = (a.sinks + B - 1) / B;
  const int64_t head = a.ring_in[0], tail = a.ring_in[1];
  const int64_t F = a.ring_size;
  int64_t avail = tail - head;
  avail = avail < 0 || head < 0 ? 0 : (avail > F ? F : avail);
  if (tid == 0) taken = 0;
  int64_t tok0 = 0, blk0 = 0, rel0 = 0;
  for (int base = 0; base < R; base += kPlanThreads) {
    const int r = base + tid;
    int len = 0, n = 0, have = 0;
    int64_t grow = 0, need = 0;
    bool fits = true;
    if (r < R) {
      len = a.lengths[r];
      n = a.new_tokens[r];
      grow = n > 0 ? n : 0;
      fits = len >= 0 && (int64_t)len + grow <= (int64_t)a.M * B;
    }
    int64_t total;
    const int64_t c = tok0 + block_exclusive_sum<kPlanThreads>(grow, warp_sums, &total);
    tok0 += total;
    if (r < R) {
      cu[r] = (int32_t)(c < INT32_MAX ? c : INT32_MAX);
      if (grow > 0 && c + grow > a.n_slots) fits = false;
      have = fits ? (len + B - 1) / B : 0;
      need = fits ? (int)(len + grow + B - 1) / B - have : 0;
    }
    const int64_t nb_at = blk0 + block_exclusive_sum<kPlanThreads>(need, warp_sums, &total);
    blk0 += total;
    // blocks are taken in request order: the served requests that need some are
    // a prefix of those, so what comes before a served one is served too
    const bool served = fits && (need == 0 || nb_at + need <= avail);
    int64_t gone = 0;
    if (r < R) {
      nb[r] = (int32_t)(nb_at < avail ? nb_at : avail);
      if (served && need > 0) atomicMax(&taken, (int32_t)(nb_at + need));
      if (served && n < 0) {
        gone = min(sb, have) + max(0, have - dead_end(len, B, a.window, sb));
      } else if (served) {
        const int hi = min(dead_end(len + (int)grow, B, a.window, sb), have + (int)need);
        gone = max(0, hi - dead_end(len, B, a.window, sb));
      }
      old[r] = served ? len : fits ? -1 : -2;
      ends[r] = n < 0 ? 1 : 0;
    }
    const int64_t rel_at = rel0 + block_exclusive_sum<kPlanThreads>(gone, warp_sums, &total);
    rel0 += total;
    if (r < R) rel[r] = (int32_t)(rel_at < F ? rel_at : F);
  }
  if (tid == 0) {
    cu[R] = (int32_t)(tok0 < INT32_MAX ? tok0 : INT32_MAX);
    rel[R] = (int32_t)(rel0 < F ? rel0 : F);
  }
  plan_barrier();  // every input but the table and the ring has been read
  const int n_new = taken, n_rel = rel[R];
  const auto ring_at = [&](int64_t i) -> int64_t { return i < F ? i : i - F; };
  const int64_t head0 = head < 0 ? 0 : head % F, tail0 = tail < 0 ? 0 : tail % F;
  for (int r = (int)flat; r < R; r += (int)step) {
    const int len = old[r], grow = cu[r + 1] - cu[r];
    a.cu_new[r] = cu[r];
    if (len >= 0) {
      const int after = ends[r] ? 0 : len + grow;
      a.lengths_out[r] = after;
      a.kv_lens[r] = after;
      a.status[r] = KVO_OK;
    } else {
      // a refused request keeps its length: in place already, unless the arrays differ
      if (a.lengths_out != a.lengths) a.lengths_out[r] = a.lengths[r];
      a.kv_lens[r] = 0;
      a.status[r] = len == -1 ? KVO_ECAPACITY : KVO_ERANGE;
    }
  }
  if (cta == 0 && tid == 0) {
    a.cu_new[R] = cu[R];
    a.ring_out[0] = head + n_new;
    a.ring_out[1] = tail + n_rel;
  }
  for (uint32_t k = flat; k < (uint32_t)n_new; k += step) {
    const int i = (int)k;
    // the last request that starts at or before entry i (those of its place that need none come before it)
    const int r = segment_of(nb, R, i);
    a.table[(int64_t)r * a.M + (old[r] + B - 1) / B + (i - nb[r])] = a.ring[ring_at(head0 + i)];
  }
  for (uint32_t k = flat; k < (uint32_t)a.n_slots; k += step) {
    const int i = (int)k;
    int32_t slot = -1;
    if (i < cu[R]) {
      const int r = segment_of(cu, R, i);
      if (old[r] >= 0) {
        const int t = old[r] + (i - cu[r]), j = t / B, have = (old[r] + B - 1) / B;
        // the request's last old block, or one of its new ones (another thread may not have written that entry yet)
        const int32_t b = j < have ? a.table[(int64_t)r * a.M + j] : a.ring[ring_at(head0 + nb[r] + (j - have))];
        const int64_t x = (int64_t)b * B + (t - j * B);
        slot = b >= 0 && x <= INT32_MAX ? (int32_t)x : -1;
      }
    }
    a.slots[i] = slot;
  }
  if (n_rel == 0) return;
  plan_barrier();  // tables complete, and every taken entry of the ring read
  for (uint32_t k = flat; k < (uint32_t)n_rel; k += step) {
    const int i = (int)k;
    const int r = segment_of(rel, R, i);
    const int nth = i - rel[r], len = old[r];
    int j = dead_end(len, B, a.window, sb) + nth;
    if (ends[r]) {
      const int s = min(sb, (len + B - 1) / B);
      j = nth < s ? nth : j - s;
    }
    a.ring[ring_at(tail0 + i)] = a.table[(int64_t)r * a.M + j];
  }
}

// ---------------------------------------------------------------------------
// Rows.  A thread handles one group of 16 elements (32 bytes of a bf16 row);
// a CTA eight rows.  HBM bound, cold L2: 65,531 rows into the cache as bf16 25.4
// us and out 25.5 (5.9 TB/s), into 4 bits 21.1 (4.6), out 17.1 (5.7).  A row goes
// into 4 bits as 288 bytes of codes and 36 of scales in two places, 8 bytes and one
// a thread, so its last sectors are written in part.  Not faster (20.5 and 17.4
// then): 32-byte loads and stores (22.8 and 19.2 us), 4, 7 or 16 rows a CTA (22.9
// to 25.1), no streaming hints (21.9 and 18.2).
// ---------------------------------------------------------------------------
constexpr int kRowsPerCta = 8;
constexpr int kRowThreads = kRowsPerCta * kGroups;

// Two codes (low four bits: x) of values already multiplied by 1 / scale in fp32.  A bf16 value that is not exactly on
// the border between two codes is off it by at least 2^-8 of it, one that is may be off by the reciprocal's and the
// product's rounding, 2^-22 of it: rounding to 11 bits first puts it back on the border, and moves no other across.
// The conversion rounds to nearest, a tie to the even code, and saturates.
__device__ __forceinline__ uint32_t e2m1_pair(float x, float y) {
  const float2 r = __half22float2(__floats2half2_rn(x, y));
  uint32_t c;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\tmov.b32 %0, {t, 0, 0, 0};\n\t}" : "=r"(c) : "f"(r.x), "f"(r.y));
  return c;
}

template <bool kQ4>
__global__ void __launch_bounds__(kRowThreads) write_paged_kernel(PagedRowsArgs a) {
  const uint32_t local = threadIdx.x / kGroups, g = threadIdx.x % kGroups;
  const int64_t i = (int64_t)blockIdx.x * kRowsPerCta + local;
  if (i >= a.n) return;
  const int32_t slot = __ldg(a.slots + i);
  const uint4* src = reinterpret_cast<const uint4*>(a.rows + i * kRow + g * kGroup);
  const uint4 x0 = __ldcs(src), x1 = __ldcs(src + 1);
  if (slot < 0 || slot >= a.pool_rows) return;
  if (!kQ4) {
    uint4* dst = reinterpret_cast<uint4*>(a.pool + (int64_t)slot * kRowBytes16 + g * kGroup * 2);
    dst[0] = x0;
    dst[1] = x1;
    return;
  }
  const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
  // the largest magnitude, by its bits: NaN above infinity above every finite value
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) top = __vmaxu2(top, w[k] & 0x7fff7fffu);
  top = max(top & 0xffffu, top >> 16);
  uint32_t c[2] = {0u, 0u};
  uint32_t sbits = 0x7f;  // a group that is not finite reads as NaN
  if (top < 0x7f80u) {
    const float amax = __uint_as_float(top << 16);
    sbits = __nv_cvt_float_to_fp8(__fdiv_rn(amax, 6.f), __NV_SATFINITE, __NV_E4M3);
    const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw((uint8_t)sbits, __NV_E4M3)));
    if (s > 0.f) {
      const float inv = __frcp_rn(s);
#pragma unroll
      for (int k = 0; k < 8; ++k) c[k >> 2] |= e2m1_pair(bf_lo(w[k]) * inv, bf_hi(w[k]) * inv) << (8 * (k & 3));
    }
  }
  const uint32_t blk = (uint32_t)slot / (uint32_t)a.B, in = (uint32_t)slot - blk * (uint32_t)a.B;
  uint8_t* base = a.pool + (int64_t)blk * ((int64_t)a.B * kRowBytesQ4);
  *reinterpret_cast<uint2*>(base + in * kCodeBytes + g * (kGroup / 2)) = make_uint2(c[0], c[1]);
  base[a.B * kCodeBytes + in * kGroups + g] = (uint8_t)sbits;
}

template <bool kQ4>
__global__ void __launch_bounds__(kRowThreads) read_paged_kernel(PagedRowsArgs a) {
  const uint32_t local = threadIdx.x / kGroups, g = threadIdx.x % kGroups;
  const int64_t i = (int64_t)blockIdx.x * kRowsPerCta + local;
  if (i >= a.n) return;
  const int32_t slot = __ldg(a.slots + i);
  if (slot < 0 || slot >= a.pool_rows) return;
  uint4* dst = reinterpret_cast<uint4*>(a.rows + i * kRow + g * kGroup);
  if (!kQ4) {
    const uint4* src = reinterpret_cast<const uint4*>(a.pool + (int64_t)slot * kRowBytes16 + g * kGroup * 2);
    const uint4 x0 = src[0], x1 = src[1];
    dst[0] = x0;
    dst[1] = x1;
    return;
  }
  const uint32_t blk = (uint32_t)slot / (uint32_t)a.B, in = (uint32_t)slot - blk * (uint32_t)a.B;
  const uint8_t* base = a.pool + (int64_t)blk * ((int64_t)a.B * kRowBytesQ4);
  const uint2 codes = *reinterpret_cast<const uint2*>(base + in * kCodeBytes + g * (kGroup / 2));
  const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw(base[a.B * kCodeBytes + in * kGroups + g], __NV_E4M3)));
  uint32_t w[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    uint32_t h;
    asm("{\n\t.reg .b8 t, u0, u1, u2;\n\tmov.b32 {t, u0, u1, u2}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}"
        : "=r"(h)
        : "r"((k < 4 ? codes.x : codes.y) >> (8 * (k & 3))));
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
    const __nv_bfloat162 p = __floats2bfloat162_rn(v.x * s, v.y * s);  // exact
    w[k] = *reinterpret_cast<const uint32_t*>(&p);
  }
  __stcs(dst, make_uint4(w[0], w[1], w[2], w[3]));
  __stcs(dst + 1, make_uint4(w[4], w[5], w[6], w[7]));
}

// 8 bits.  Eight lanes have a row, nine pieces of 8 elements each, so a row's
// largest magnitude is three shuffles away and every piece is read once.  HBM
// bound: 65,531 rows into the cache and out 36 us, cold L2 (6.3 TB/s, 0.93 of the
// copy rate).
constexpr int kRowLanes = 8;
constexpr int kPieces = kRow / 8 / kRowLanes;
constexpr int kRowThreadsF8 = 128;
constexpr int kRowsPerCtaF8 = kRowThreadsF8 / kRowLanes;

__global__ void __launch_bounds__(kRowThreadsF8) write_paged_f8_kernel(PagedRowsArgs a) {
  const int l = threadIdx.x % kRowLanes;
  const int64_t i = (int64_t)blockIdx.x * kRowsPerCtaF8 + threadIdx.x / kRowLanes;
  const int32_t slot = i < a.n ? __ldg(a.slots + i) : -1;
  const bool to = slot >= 0 && slot < a.pool_rows;
  uint4 x[kPieces];
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    x[k] = make_uint4(0u, 0u, 0u, 0u);
    if (to) x[k] = __ldcs(reinterpret_cast<const uint4*>(a.rows + i * kRow) + l + k * kRowLanes);
  }
  // the largest magnitude, by its bits: NaN above infinity above every finite value
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    top = __vmaxu2(top, __vmaxu2(x[k].x & 0x7fff7fffu, x[k].y & 0x7fff7fffu));
    top = __vmaxu2(top, __vmaxu2(x[k].z & 0x7fff7fffu, x[k].w & 0x7fff7fffu));
  }
#pragma unroll
  for (int o = 1; o < kRowLanes; o <<= 1) top = __vmaxu2(top, __shfl_xor_sync(kFull, top, o));
  if (!to) return;
  top = max(top & 0xffffu, top >> 16);
  // m 2^k <= 448 2^e = 1.75 2^(8 + e): the least e is k - 8 up to m = 1.75, else k - 7
  const bool fine = top < 0x7f80u;
  const int k0 = (int)(top >> 7) - 127;
  const int e = min(max(k0 - 8 + ((top & 127u) > 96u ? 1 : 0), -kScaleExp), kScaleExp);
  const float down = __uint_as_float((uint32_t)(127 - e) << 23);
  const uint32_t blk = (uint32_t)slot / (uint32_t)a.B, in = (uint32_t)slot - blk * (uint32_t)a.B;
  uint8_t* base = a.pool + (int64_t)blk * ((int64_t)a.B * kRowBytesF8);
  uint2* dst = reinterpret_cast<uint2*>(base + (int64_t)in * kRow) + l;
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c[j] = __nv_cvt_float2_to_fp8x2(make_float2(bf_lo(w[j]) * down, bf_hi(w[j]) * down), __NV_SATFINITE, __NV_E4M3);
    dst[k * kRowLanes] = fine ? make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16) : make_uint2(0u, 0u);
  }
  if (l == 0)
    *reinterpret_cast<uint32_t*>(base + (int64_t)a.B * kRow + in * 4) = fine ? (uint32_t)(127 + e) << 23 : 0x7fffffffu;
}

__global__ void __launch_bounds__(kRowThreadsF8) read_paged_f8_kernel(PagedRowsArgs a) {
  const int l = threadIdx.x % kRowLanes;
  const int64_t i = (int64_t)blockIdx.x * kRowsPerCtaF8 + threadIdx.x / kRowLanes;
  if (i >= a.n) return;
  const int32_t slot = __ldg(a.slots + i);
  if (slot < 0 || slot >= a.pool_rows) return;
  const uint32_t blk = (uint32_t)slot / (uint32_t)a.B, in = (uint32_t)slot - blk * (uint32_t)a.B;
  const uint8_t* base = a.pool + (int64_t)blk * ((int64_t)a.B * kRowBytesF8);
  const uint2* src = reinterpret_cast<const uint2*>(base + (int64_t)in * kRow) + l;
  uint2 c[kPieces];
#pragma unroll
  for (int k = 0; k < kPieces; ++k) c[k] = src[k * kRowLanes];
  uint32_t bits = *reinterpret_cast<const uint32_t*>(base + (int64_t)a.B * kRow + in * 4);
  if (!row_scale_valid(bits)) bits = 0x7fffffffu;
  const float s = __uint_as_float(bits);
  uint4* dst = reinterpret_cast<uint4*>(a.rows + i * kRow) + l;
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t two = (j < 2 ? c[k].x : c[k].y) >> (16 * (j & 1));
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xffffu), __NV_E4M3);
      const float2 v = __half22float2(__half2(h));
      const __nv_bfloat162 p = __floats2bfloat162_rn(v.x * s, v.y * s);  // exact
      w[j] = *reinterpret_cast<const uint32_t*>(&p);
    }
    __stcs(dst + k * kRowLanes, make_uint4(w[0], w[1], w[2], w[3]));
  }
}

template <typename K>
cudaError_t launch_rows(K kernel, int rows_per_cta, int threads, const PagedRowsArgs& a, cudaStream_t s) {
  if (a.n <= 0) return cudaSuccess;
  const int64_t grid = (a.n + rows_per_cta - 1) / rows_per_cta;
  kernel<<<(unsigned)grid, threads, 0, s>>>(a);
  return cudaGetLastError();
}

int fail(int code, const char* msg) { return set_error(code, msg); }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int rows_call(PagedRowsArgs& a, const void* rows, const int32_t* slots, int64_t n_rows, const void* pool,
              int64_t n_blocks, int32_t block_tokens, int32_t format) {
  const int rc = check_paged_cache(pool, n_blocks, block_tokens, format);
  if (rc != KVO_OK) return rc;
  if (n_rows < 0 || n_rows >= (int64_t)1 << 31) return fail(KVO_EINVAL, "n_rows out of range");
  if (n_rows > 0 && (!rows || !slots)) return fail(KVO_EINVAL, "NULL argument");
  if (!aligned(rows, 16) || !aligned(slots, 4)) return fail(KVO_EINVAL, "rows not 16-byte or slots not 4-byte aligned");
  a.pool = static_cast<uint8_t*>(const_cast<void*>(pool));
  a.pool_rows = n_blocks * block_tokens;
  a.B = block_tokens;
  a.slots = slots;
  a.n = n_rows;
  a.rows = static_cast<uint16_t*>(const_cast<void*>(rows));
  return KVO_OK;
}

}  // namespace

int check_paged_cache(const void* pool, int64_t n_blocks, int32_t block_tokens, int32_t format) {
  if (!pool) return fail(KVO_EINVAL, "pool is NULL");
  if (!aligned(pool, 16)) return fail(KVO_EINVAL, "pool not 16-byte aligned");
  if (format != KVO_CACHE_BF16 && format != KVO_CACHE_Q4 && format != KVO_CACHE_F8)
    return fail(KVO_EINVAL, "unknown cache format");
  if (block_tokens < 8 || block_tokens > 65536 || block_tokens % 8 != 0)
    return fail(KVO_EINVAL, "block_tokens must be a multiple of 8 in 8 .. 65536");
  if (n_blocks < 1 || n_blocks > INT32_MAX / block_tokens)
    return fail(KVO_EINVAL, "n_blocks * block_tokens must be positive and below 2^31");
  return KVO_OK;
}

cudaError_t launch_paged_plan(const PagedPlanArgs& a, cudaStream_t s) {
  // Asked for once, for the most requests: what a launch may have does not depend on the calls before it or beside it.
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static std::atomic<uint64_t> ready{0};  // devices where the kernel may have its shared memory
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(plan_paged_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)plan_smem(kMaxRequests));
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  const unsigned ctas = a.n_slots > kPlanSlots ? kPlanCtas : 1;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = ctas;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(ctas);
  c.blockDim = dim3(kPlanThreads);
  c.dynamicSmemBytes = plan_smem(a.R);
  c.stream = s;
  c.attrs = &at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, plan_paged_kernel, a);
}
cudaError_t launch_paged_write(const PagedRowsArgs& a, int format, cudaStream_t s) {
  if (format == KVO_CACHE_F8) return launch_rows(write_paged_f8_kernel, kRowsPerCtaF8, kRowThreadsF8, a, s);
  return launch_rows(format == KVO_CACHE_Q4 ? write_paged_kernel<true> : write_paged_kernel<false>, kRowsPerCta, kRowThreads, a, s);
}
cudaError_t launch_paged_read(const PagedRowsArgs& a, int format, cudaStream_t s) {
  if (format == KVO_CACHE_F8) return launch_rows(read_paged_f8_kernel, kRowsPerCtaF8, kRowThreadsF8, a, s);
  return launch_rows(format == KVO_CACHE_Q4 ? read_paged_kernel<true> : read_paged_kernel<false>, kRowsPerCta, kRowThreads, a, s);
}

}  // namespace kvo

extern "C" {

int64_t kvo_paged_block_bytes(int32_t format, int32_t block_tokens) {
  if (block_tokens < 8 || block_tokens > 65536 || block_tokens % 8 != 0) return 0;
  if (format == KVO_CACHE_BF16) return (int64_t)block_tokens * kvo::paged::kRowBytes16;
  if (format == KVO_CACHE_Q4) return (int64_t)block_tokens * kvo::paged::kRowBytesQ4;
  if (format == KVO_CACHE_F8) return (int64_t)block_tokens * kvo::paged::kRowBytesF8;
  return 0;
}

int kvo_paged_plan(const int32_t* lengths, const int32_t* new_tokens, int32_t n_requests, int32_t block_tokens,
                   int32_t max_blocks, int32_t window, int32_t sinks, int32_t* block_table, int32_t* ring,
                   int32_t ring_size, const int64_t* ring_in, int64_t* ring_out, int32_t* lengths_out,
                   int32_t* kv_lens, int32_t* cu_new, int32_t* slots, int32_t n_slots, int32_t* status, void* stream) {
  using namespace kvo;
  if (!lengths || !new_tokens || !block_table || !ring || !ring_in || !ring_out || !lengths_out || !kv_lens ||
      !cu_new || !status || (!slots && n_slots != 0))
    return fail(KVO_EINVAL, "NULL argument");
  if (!aligned(lengths, 4) || !aligned(new_tokens, 4) || !aligned(block_table, 4) || !aligned(ring, 4) ||
      !aligned(ring_in, 8) || !aligned(ring_out, 8) || !aligned(lengths_out, 4) || !aligned(kv_lens, 4) ||
      !aligned(cu_new, 4) || !aligned(slots, 4) || !aligned(status, 4))
    return fail(KVO_EINVAL, "array not aligned to its elements");
  if (n_requests < 1 || n_requests > paged::kMaxRequests) return fail(KVO_EINVAL, "n_requests must be in 1 .. 4096");
  if (block_tokens < 8 || block_tokens > 65536 || block_tokens % 8 != 0)
    return fail(KVO_EINVAL, "block_tokens must be a multiple of 8 in 8 .. 65536");
  if (max_blocks < 1 || (int64_t)max_blocks * block_tokens > paged::kMaxTokens)
    return fail(KVO_EINVAL, "max_blocks * block_tokens must be in 1 .. 2^30");
  if (ring_size < 1 || n_slots < 0 || window < 0 || sinks < 0)
    return fail(KVO_EINVAL, "ring_size, n_slots, window or sinks out of range");
  PagedPlanArgs a{};
  a.lengths = lengths;
  a.new_tokens = new_tokens;
  a.R = n_requests;
  a.B = block_tokens;
  a.M = max_blocks;
  // beyond every token that a table reaches, they say no more
  a.window = (int32_t)(window < paged::kMaxTokens ? window : paged::kMaxTokens);
  a.sinks = (int32_t)(sinks < paged::kMaxTokens ? sinks : paged::kMaxTokens);
  a.table = block_table;
  a.ring = ring;
  a.ring_size = ring_size;
  a.ring_in = ring_in;
  a.ring_out = ring_out;
  a.lengths_out = lengths_out;
  a.kv_lens = kv_lens;
  a.cu_new = cu_new;
  a.slots = slots;
  a.n_slots = n_slots;
  a.status = status;
  const cudaError_t e = launch_paged_plan(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return set_cuda_error(e, "paged plan launch");
  return KVO_OK;
}

int kvo_paged_write(const void* rows, const int32_t* slots, int64_t n_rows, void* pool, int64_t n_blocks,
                    int32_t block_tokens, int32_t format, void* stream) {
  kvo::PagedRowsArgs a{};
  const int rc = kvo::rows_call(a, rows, slots, n_rows, pool, n_blocks, block_tokens, format);
  if (rc != KVO_OK) return rc;
  const cudaError_t e = kvo::launch_paged_write(a, format, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return kvo::set_cuda_error(e, "paged write launch");
  return KVO_OK;
}

int kvo_paged_read(const void* pool, int64_t n_blocks, int32_t block_tokens, int32_t format, const int32_t* slots,
                   int64_t n_rows, void* rows, void* stream) {
  kvo::PagedRowsArgs a{};
  const int rc = kvo::rows_call(a, rows, slots, n_rows, pool, n_blocks, block_tokens, format);
  if (rc != KVO_OK) return rc;
  const cudaError_t e = kvo::launch_paged_read(a, format, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return kvo::set_cuda_error(e, "paged read launch");
  return KVO_OK;
}

size_t kvo_paged_attend_workspace_size(int32_t n_requests, int32_t n_tokens, int32_t n_heads, int32_t device) {
  if (n_requests < 1 || n_requests > kvo::paged::kMaxRequests || n_tokens < 0 || n_heads < 1 || n_heads > 8192) return 0;
  int n_sm = 0;
  if (cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) return 0;
  return kvo::paged_attend_workspace_most(n_requests, n_tokens, n_heads, n_sm < kvo::paged::kMaxWorkers ? n_sm : kvo::paged::kMaxWorkers);
}

// What kvo_paged_attend and kvo_paged_attend_tree share; masks null: causal order.
static int paged_attend_call(const void* pool, int64_t n_blocks, int32_t block_tokens, int32_t format,
                             const int32_t* block_table, int32_t max_blocks, const int32_t* kv_lens,
                             const int32_t* cu_tokens, int32_t n_requests, const uint32_t* masks, int32_t mask_words,
                             const int32_t* depths, const void* queries, int32_t n_tokens, int32_t n_heads, float scale,
                             int32_t window, int32_t sinks, void* out, float* lse, void* workspace,
                             size_t workspace_bytes, uint32_t* status, void* stream) {
  using namespace kvo;
  const int rc = check_paged_cache(pool, n_blocks, block_tokens, format);
  if (rc != KVO_OK) return rc;
  if (!block_table || !kv_lens || !cu_tokens || !workspace) return fail(KVO_EINVAL, "NULL argument");
  if (n_requests < 1 || n_requests > paged::kMaxRequests) return fail(KVO_EINVAL, "n_requests must be in 1 .. 4096");
  if (max_blocks < 1 || (int64_t)max_blocks * block_tokens > paged::kMaxTokens)
    return fail(KVO_EINVAL, "max_blocks * block_tokens must be in 1 .. 2^30");
  if (n_heads < 1 || n_heads > 8192) return fail(KVO_EINVAL, "n_heads must be in 1 .. 8192");
  if (n_tokens < 0 || (int64_t)n_tokens * n_heads >= (int64_t)1 << 30)
    return fail(KVO_EINVAL, "n_tokens * n_heads must be below 2^30");
  if (n_tokens > 0 && (!queries || !out)) return fail(KVO_EINVAL, "NULL argument");
  if (!aligned(queries, 16) || !aligned(out, 16)) return fail(KVO_EINVAL, "queries or out not 16-byte aligned");
  if (!aligned(block_table, 4) || !aligned(kv_lens, 4) || !aligned(cu_tokens, 4) || !aligned(lse, 4) || !aligned(status, 4))
    return fail(KVO_EINVAL, "array not aligned to its elements");
  if (!aligned(workspace, 256)) return fail(KVO_EINVAL, "workspace not 256-byte aligned");
  const float scale_log2 = scale * 1.4426950408889634f;  // log2 e
  if (!(scale_log2 - scale_log2 == 0.f)) return fail(KVO_EINVAL, "scale, or scale * log2 e, is not finite");
  if (window < 0 || sinks < 0) return fail(KVO_EINVAL, "window and sinks must not be negative");
  int dev = 0, n_sm = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return fail(KVO_ECUDA, "no current device");
  if (n_sm > paged::kMaxWorkers) n_sm = paged::kMaxWorkers;
  if (workspace_bytes < paged_attend_workspace(n_requests, n_tokens, n_heads, n_sm))
    return fail(KVO_EINVAL, "workspace too small");
  PagedAttendArgs a{};
  a.pool = static_cast<const uint8_t*>(pool);
  a.n_blocks = n_blocks;
  a.B = block_tokens;
  a.b_shift = (block_tokens & (block_tokens - 1)) == 0 ? __builtin_ctz((unsigned)block_tokens) : -1;
  a.M = max_blocks;
  a.R = n_requests;
  a.table = block_table;
  a.kv_lens = kv_lens;
  a.cu = cu_tokens;
  a.q = static_cast<const uint16_t*>(queries);
  a.n_tokens = n_tokens;
  a.H = n_heads;
  a.window = (int32_t)(window < paged::kMaxTokens ? window : paged::kMaxTokens);
  a.sinks = (int32_t)(sinks < paged::kMaxTokens ? sinks : paged::kMaxTokens);
  a.masks = masks;
  a.mask_words = mask_words;
  a.depths = depths;
  a.scale_log2 = scale_log2;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.status = status;
  a.wait_ns = 2000000000ull;
  a.workers = n_sm;
  a.device = dev;
  paged_attend_carve(a, static_cast<uint8_t*>(workspace));
  const cudaError_t e = launch_paged_attend(a, format, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return set_cuda_error(e, "paged attention launch");
  return KVO_OK;
}

int kvo_paged_attend(const void* pool, int64_t n_blocks, int32_t block_tokens, int32_t format,
                     const int32_t* block_table, int32_t max_blocks, const int32_t* kv_lens, const int32_t* cu_tokens,
                     int32_t n_requests, const void* queries, int32_t n_tokens, int32_t n_heads, float scale,
                     int32_t window, int32_t sinks, void* out, float* lse, void* workspace, size_t workspace_bytes,
                     uint32_t* status, void* stream) {
  return paged_attend_call(pool, n_blocks, block_tokens, format, block_table, max_blocks, kv_lens, cu_tokens, n_requests,
                           nullptr, 0, nullptr, queries, n_tokens, n_heads, scale, window, sinks, out, lse, workspace,
                           workspace_bytes, status, stream);
}

int kvo_paged_attend_tree(const void* pool, int64_t n_blocks, int32_t block_tokens, int32_t format,
                          const int32_t* block_table, int32_t max_blocks, const int32_t* kv_lens, const int32_t* cu_tokens,
                          int32_t n_requests, const uint32_t* masks, int32_t mask_words, const int32_t* depths,
                          const void* queries, int32_t n_tokens, int32_t n_heads, float scale, int32_t window, int32_t sinks,
                          void* out, float* lse, void* workspace, size_t workspace_bytes, uint32_t* status, void* stream) {
  using namespace kvo;
  if (!masks && n_tokens != 0) return fail(KVO_EINVAL, "masks is NULL");
  if (!aligned(masks, 4) || !aligned(depths, 4)) return fail(KVO_EINVAL, "array not aligned to its elements");
  if (mask_words < 1 || mask_words > 32) return fail(KVO_EINVAL, "mask_words must be in 1 .. 32");
  if (window > 0 && !depths && n_tokens != 0) return fail(KVO_EINVAL, "a window needs the nodes' depths");
  return paged_attend_call(pool, n_blocks, block_tokens, format, block_table, max_blocks, kv_lens, cu_tokens, n_requests,
                           masks, mask_words, depths, queries, n_tokens, n_heads, scale, window, sinks, out, lse, workspace,
                           workspace_bytes, status, stream);
}

}  // extern "C"
