// Shared by the attention kernels of the paged device cache: the 5th-generation
// tensor cores' instructions, bounded waits, copies and shared-memory access.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvo_paged.cuh"

namespace kvo {
namespace paged {

constexpr int kSoftWarps = 8;
constexpr int kSoftThreads = kSoftWarps * 32;
constexpr uint32_t kAtom = 1024;             // 8 tokens x 128 bytes
constexpr float kNone = -3.0e38f;            // running maximum before any visible token

// ---- tcgen05 ------------------------------------------------------------------------------
// Shared-memory matrix descriptor, 128-byte swizzle: start address and leading offset (in 16-byte units) in the low
// word; the high word: rows (or tokens) in groups of 8, 1 KB apart, or 2 KB in the ring.
constexpr uint32_t kDescHigh = (kAtom >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kDescHighRing = (2 * kAtom >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t sdesc(uint32_t addr, uint32_t lead) {
  return ((addr >> 4) & 0x3FFFu) | (((lead >> 4) & 0x3FFFu) << 16);
}
// Instruction descriptor of kind::f16: A and B both bf16 or both f16, fp32 D.
constexpr uint32_t idesc(bool bf16, int M, int N, bool a_mn_major, bool b_mn_major) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((a_mn_major ? 1u : 0u) << 15) |
         ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// Issued by the lane whose `el` is set; the warp runs it uniformly.  The operands live in uniform registers, and moving
// one there costs more than the MMA's issue: only the descriptors' low words vary.
template <uint32_t kHighA>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc, uint32_t el) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "mov.b64 da, {%1, %6};\n\tmov.b64 db, {%2, %7};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(acc), "r"(el), "n"(kHighA), "n"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar, uint32_t el) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(el)
      : "memory");
}
__device__ __forceinline__ uint32_t elect() {
  uint32_t el;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(el));
  return el;
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 8 consecutive 32-bit columns of this thread's TMEM lane (kNC in steps of 8).
__device__ __forceinline__ void tmem_ld8(uint32_t t, float* v) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(t)
               : "memory");
#pragma unroll
  for (int c = 0; c < 8; ++c) v[c] = __uint_as_float(r[c]);
}
__device__ __forceinline__ void tmem_st8(uint32_t t, const float* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(t),
               "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
               "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
               "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
               : "memory");
}
template <int NC>
__device__ __forceinline__ void tmem_ld(uint32_t t, float (&v)[NC]) {
#pragma unroll
  for (int c = 0; c < NC; c += 8) tmem_ld8(t + (uint32_t)c, v + c);
}

// Bounded wait on a phase parity; false when limit_ns has passed, or another role has given up.  Reading the timer costs more than most waits here
// last, so it starts late.
__device__ __forceinline__ bool phase_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns,
                                           const volatile uint32_t* abort = nullptr) {
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0) {
      const uint64_t now = global_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > limit_ns || (abort && *abort != 0u)) return false;
    }
  }
}
// ---- shared memory -------------------------------------------------------------------------
// 16-byte chunk c (0..7) of token r in slab `side` of a pair.
__device__ __forceinline__ uint32_t swz_pair(uint32_t pair, int side, int r, int c) {
  return pair + (uint32_t)(r >> 3) * (2 * kAtom) + (uint32_t)side * kAtom + (uint32_t)(r & 7) * 128u + ((uint32_t)(c ^ (r & 7)) << 4);
}
// 16-byte chunk c (0..7) of row r in a 128-byte-swizzled slab (1 KB aligned).
__device__ __forceinline__ uint32_t swz(uint32_t slab, int r, int c) {
  return slab + (uint32_t)r * 128u + ((uint32_t)(c ^ (r & 7)) << 4);
}
// Bytes (a multiple of 16, 16-byte aligned) into L2.
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
// A box of a 2-D tensor map (x: element, y: row), completion counted in bytes on bar.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}
// A box of the pool's rows in two slabs (`slab`, + 1), from row 8 `group` on: see Maps.
__device__ __forceinline__ void tma_pair(uint32_t dst, const CUtensorMap* map, int slab, int group, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(0), "r"(slab), "r"(group), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void st_v4(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 ld_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_u16(uint32_t addr, uint16_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(v) : "memory");
}
// Whether any of the first `threads` threads at barrier `id` has p set.
__device__ __forceinline__ bool named_any(uint32_t id, uint32_t threads, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)p), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}
// Bits whose order as integers is the values' (its own inverse); a positive NaN above all.
__device__ __forceinline__ int32_t as_ordered(float x) {
  const int32_t b = __float_as_int(x);
  return b ^ ((b >> 31) & 0x7fffffff);
}
// 2^x, hardware approximation (relative error near 2^-22); 2^-inf = 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The next launch of the stream may start its set-up; grid_wait: the last one is done and its writes are visible.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

using EncodeTiled = decltype(&cuTensorMapEncodeTiled);

// The driver's tensor-map encoder (the library is linked against the runtime alone).
inline EncodeTiled encoder() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

}  // namespace paged
}  // namespace kvo
