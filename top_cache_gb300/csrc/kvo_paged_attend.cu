// Attention over the paged device cache, in 16 or 4 bits, with a sliding window
// and sinks, on the 5th-generation tensor cores.
//
// Absorbed latent attention (as kvo_attend): a cached row is 576 elements,
// latent 512 (also the value) | rope key 64.  Query token i of request r is at
// position p = kv_len - n_q + i and sees token t when t <= p and (no window, or
// t > p - window, or t < sinks) and its block is mapped; for each head
//   s_t = scale * q . row_t,  out = sum_t softmax(s)_t row_t[0:512],
//   lse = log sum_t exp(s_t);  nothing visible: out 0, lse -inf.
//
// Shape of the work.  The rows of a request's queries, (token, head) in memory
// order, are cut into tiles of N = 16, 32 or 64; a tile walks the 128-token
// blocks that any of its positions sees.  Keys and queries change places in the
// MMAs: S^T = K Q^T has M = 128 tokens and N = the tile's rows, O^T = V^T P^T
// has M = 128 of the 512 value elements.  So a tile of 16 rows costs 16 columns
// (heads on the M side would be padded to 128), and O^T of 64 rows, 4 x 64 fp32
// columns, leaves TMEM room for S^T without splitting the value elements over
// CTAs.  A tcgen05.mma with both operands in shared memory takes the time of
// reading them at 128 bytes a clock: 32 + N / 4 clocks for M = 128, K = 16, when
// the issuing warp runs uniformly (39, 40 and 48 measured at N = 16, 32, 64; 69
// whatever N from inside a one-thread branch).  N = 64 therefore peaks at 2/3
// of the tensor rate.
//
// One persistent CTA per SM, warp-specialised:
//   producers    the tile's queries, then each block's rows into a ring of
//                pairs of 128-byte-swizzled K-major slabs (128 tokens x 64
//                elements, atoms of 8 tokens of the two in turn); the same bytes are the K-major A of S^T and the
//                MN-major A of O^T.  16 bits: one warp, a lane per TMA box of
//                two slabs x the rows of one cache block (runs of 8 to 128).
//                4 bits: 8 warps hold the next block's codes in registers while
//                they expand this one's to fp16 (exact; queries are scaled by a
//                power of two per row to fit fp16, undone in the scores)
//   softmax      8 warps, one token (TMEM lane) per thread and half of the
//                tile's rows.  Per-thread sums; a running maximum that moves
//                only when a score passes it by 2^40 (4 bits: 2^8), so most
//                blocks need no reduction over the tokens, only a vote
//   MMA          one warp: S^T of a block, then, once its weights are there,
//                O^T; each pair of slabs is freed behind its part of O^T
// Every wait is bounded; when one expires the error word is set and the roles
// stop.
//
// What bounds it (152 CTAs, clocks of one block of 128 tokens at N = 64).  16
// bits: S^T 1,730 + O^T 1,520 at the operands' shared-memory rate; the softmax
// between them, 1,550 with its hand-overs, is exposed, since the ring has room
// for one block and no more: 4,800.  Borders of tiles cost 2,000 and more.  0.39
// of the measured bf16 rate on 16 x 4 positions of 128 heads over a window of
// 4,096 (99 us).  4 bits: the expansion's stores add 1,150 clocks to the 3,300 of
// operand reads, and take 1,000 a pair while O^T is read: 6,200.  N = 16 reads 16
// bits at 5.4 to 5.5 TB/s (0.80 of the copy rate: 32 requests of 32k, 154 us).  4
// bits: 2.2 TB/s, 5,250 clocks a block: 2,450 of operand reads beside 3,000
// wavefronts of the load/store path (1,400 stores, 1,400 loads of codes).
// Tried and slower: blocks of 64 tokens with S^T two blocks ahead (the M = 64
// product does not repay twice the hand-overs), keys in TMEM for S^T of 4-bit
// tiles (150 clocks a product), 16 softmax warps (their time is latency), 16
// producer warps at N = 16 (231 us for 218), weights stored before the vote.
//
// Split.  Up to 2,048 tiles are listed with their blocks.  If whole tiles would
// leave CTAs idle (few tiles, or uneven ones), the list's blocks are cut evenly
// over the CTAs, whatever tiles they cross, so one long request fills the GPU; a
// tile that no CTA has alone leaves partial (O, m, l) in the workspace, at most
// two per CTA, and a last kernel joins them in CTA order.  Else CTA c takes tiles
// c, c + CTAs, ... whole (neighbours cost alike).  Measured, 16 heads: 128
// requests of 2k split 68 us, whole 61; 160 of 2k 91 and 107; 100 of 8k (4 bits)
// 135 and 182.  More than 2,048 tiles always go whole, however uneven they are:
// 2,000 requests of 256 tokens and one of 256k 187 us, 2,100 and one 4,092 (apart
// 137 and 70).  Results do not depend on timing.
//
// Rounding.  The weights of the value product are bf16 (fp16 over 4 bits), the
// sum that divides it is of the weights before that, in fp32, so out may be off
// by a weight's rounding where one token has nearly all of it.  A second sum, of
// the rounded weights, kept in TMEM: error against 64 bits the same on normal
// inputs (relative, root mean square, 0.0018 to 0.0021 with it and 0.0018 to
// 0.0022 without), chunks of many tiles 2 to 5 % slower, others up to 4 %.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "kvo_paged.cuh"

namespace kvo {

using namespace paged;

namespace {

constexpr int kBlk = 128;            // tokens per block of the walk: M of S^T, K of O^T
constexpr int kSlabs = kRow / 64;    // 9: eight of the value, then rope
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
constexpr int kSoftWarps = 8;
constexpr int kSoftThreads = kSoftWarps * 32;
constexpr uint32_t kSlab = kBlk * 128;       // bytes of one slab of a block
constexpr uint32_t kPair = 2 * kSlab;
constexpr uint32_t kAtom = 1024;             // 8 tokens x 64 elements; a pair's two slabs alternate atom by atom
constexpr int kMaxRing = 5;
constexpr float kNone = -3.0e38f;            // running maximum before any visible token

template <int N, bool kQ4>
struct Shape {
  static constexpr int kProdWarps = kQ4 ? 8 : 1;
  static constexpr int kProducers = kProdWarps * 32;
  static constexpr int kFillers = kQ4 ? kProducers : 1;  // arrivals that complete a filled slot
  static constexpr int kThreads = kSoftThreads + kProducers + 32;
  static constexpr bool kAhead = !kQ4;                 // softmax holds the next tile beside this one (registers)
  static constexpr bool kOwn = !(kQ4 && N == 64);      // may list the tiles for itself (else registers spill, 88 -> 102 us)
  static constexpr int kNC = N / 2;                    // rows of one softmax thread
  static constexpr bool kSharedP = N == 64;            // P^T lies in the rope slab's place
  static constexpr int kRing = N == 64 ? 4 : kMaxRing; // pairs
  static constexpr uint32_t kQSlab = N * 128;
  static constexpr uint32_t kQOff = 0;
  static constexpr uint32_t kRingOff = kSlabs * kQSlab;
  static constexpr uint32_t kRopeOff = kRingOff + kRing * kPair;
  static constexpr uint32_t kPOff = kSharedP ? kRopeOff : kRopeOff + kSlab;
  static constexpr uint32_t kPBytes = kSharedP ? kSlab : N * 256u;
  static constexpr uint32_t kMiscOff = kPOff + kPBytes;
  // misc: less running maxima, query factors, row positions [2][N], a block's maxima and the tile's sums [8][NC],
  // factors of a move of the running maximum [N], 1 / l [N]
  static constexpr uint32_t kMiscBytes = (3 * 2 * N + 2 * 8 * kNC + 2 * N) * 4;
  static constexpr uint32_t kBarOff = kMiscOff + kMiscBytes;
  static constexpr uint32_t kListOff = kBarOff + 256;      // behind the barriers and flags
  static constexpr uint32_t kSmem = kListOff + (kOwn ? 2400 : 0) + 1024;  // the CTA's own list; alignment slack
  static constexpr uint32_t kTmem = N == 64 ? 512 : N == 32 ? 256 : 128;
  static constexpr uint32_t kColS = 4 * N;             // O^T: value elements 128 i.. at columns i * N
  static constexpr float kBias = kQ4 ? 7.f : 0.f;      // P is 2^kBias exp2(..): keeps small weights out of fp16's subnormals
  // log2: how far a score may pass the running maximum.  bf16 weights are as exact at any size, and 2^40 of them
  // stay far from fp32's range; fp16 ends at 2^16.
  static constexpr float kRescale = kQ4 ? 8.f : 40.f;
  static_assert(kSmem <= 232448, "shared memory of one CTA");
  static_assert(kRingOff % 1024 == 0 && kPOff % 1024 == 0 && kMiscOff % 16 == 0 && kBarOff % 8 == 0,
                "swizzled tiles sit on 1 KB boundaries");
};

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

// ---- the work -------------------------------------------------------------------------------
// One tile, or the part of its blocks that this CTA has.
struct Seg {
  int r;                 // request
  int grow;              // first row of the tile among all (token, head) rows
  int row0, nrows;       // first row within the request, rows
  int pos0;              // position of the request's first query token
  int pmin, pmax;        // positions of the tile's first and last row
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
template <int kThreads, int kMost>
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
      const int nblk = tile_of(a, N, r, (i - off[r]) * N, s);
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

// ---------------------------------------------------------------------------
// schedule: the list of a call where the attention's CTAs do not make it, one
// CTA; as many threads as a short list has tiles (4.7 us for 128 tiles of 16
// requests; 1,024 threads 6.5).
// ---------------------------------------------------------------------------
constexpr int kSchedThreads = 1024;

template <int kThreads, int kTiles, int kRequests>
__global__ void __launch_bounds__(kThreads) schedule_paged_kernel(PagedAttendArgs a, int N) {
  __shared__ List t;
  __shared__ int32_t off[kRequests + 1], before[kTiles];
  launch_dependents();
  build_list<kThreads, kTiles>(a, N, off, before, t, true);
  __syncthreads();
  for (int r = threadIdx.x; r <= a.R; r += kThreads) a.tile_off[r] = off[r];
  if (t.used > 0)
    for (int w = threadIdx.x; w <= t.used; w += kThreads) a.start[w] = share_start(before, t.n_tiles, t.units, t.used, w);
}

// The segments of one CTA, in order; every warp that walks them calls next()
// with all lanes.  `t`: the CTA's own list (a.own_list).
template <int N, bool kOwn>
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
      s.b1 = tile_of(a, N, lo, (tile - (own ? t.off[lo] : a.tile_off[lo])) * N, s);
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
      const int nblk = tile_of(a, N, r, row0, s);
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

// ---------------------------------------------------------------------------
// attention
// ---------------------------------------------------------------------------
struct Bars {
  uint64_t q_full, q_free, r_full, r_free, s_full, p_full, o_done, o_free, fin;
  uint64_t e_full[kMaxRing], e_free[kMaxRing];
  uint32_t tmem, abort;
  uint32_t dead[2][2];  // softmax: a warp of the half gave up, by parity of the barrier's count
};
static_assert(sizeof(Bars) <= 256 && sizeof(List) <= 2400, "barriers; the CTA's own list");

// 16 elements of E2M1 codes (8 bytes) times their scale: 32 bytes of fp16, exact.
__device__ __forceinline__ void expand16(uint32_t c0, uint32_t c1, uint32_t s2, uint4& lo, uint4& hi) {
  uint32_t r[8];
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(c0));
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(c1));
#pragma unroll
  for (int k = 0; k < 8; ++k) asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r[k]) : "r"(r[k]), "r"(s2));
  lo = make_uint4(r[0], r[1], r[2], r[3]);
  hi = make_uint4(r[4], r[5], r[6], r[7]);
}
// Two E4M3 scales (low 16 bits) -> each one twice, as fp16 pairs.
__device__ __forceinline__ void scales2(uint32_t b, uint32_t& s0, uint32_t& s1) {
  uint32_t h;
  asm("{\n\t.reg .b16 t, u;\n\tmov.b32 {t, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(b));
  s0 = __byte_perm(h, h, 0x1010);
  s1 = __byte_perm(h, h, 0x3232);
}

// Entry of a request's block table that token t is in.
__device__ __forceinline__ int entry_of(const PagedAttendArgs& a, int t) { return a.b_shift >= 0 ? t >> a.b_shift : t / a.B; }
// Token t's row of the pool (-1: its block is not mapped).
__device__ __forceinline__ int64_t pool_row(const PagedAttendArgs& a, const int32_t* table, int t) {
  const int j = entry_of(a, t);
  const int32_t b = __ldg(table + j);
  return b < 0 || (int64_t)b >= a.n_blocks ? -1 : (int64_t)b * a.B + (t - j * a.B);
}

// One block's codes and scales of producer thread (token, side): of each slab
// 32 elements.
struct Codes {
  uint4 c[4][2];
  uint32_t s[4];
  uint4 rc;
  uint32_t rs;
};

// 16 bits: the pool in boxes of `run` rows (the largest power of two, at most
// 128, that divides block_tokens).  Value elements are seen as [row / 8][slab]
// [row % 8][64]; a box has two slabs, so it lands as a pair's atoms do whatever
// the run is.  (Small boxes bound the copy unit: 32 requests of 32k in blocks of
// 8 tokens 179 us, with a box per slab 245; in blocks of 64, 152 either way.)
// Rope: 64 elements x run; queries: 64 x N.
struct Maps {
  CUtensorMap pool, rope, q;
  int run;
};

template <int N, bool kQ4>
__global__ void __launch_bounds__(Shape<N, kQ4>::kThreads, 1)
    attend_paged_kernel(PagedAttendArgs a, const __grid_constant__ Maps maps) {
  using C = Shape<N, kQ4>;
  constexpr int NC = C::kNC;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sb = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sb - raw);
  float* less_max = reinterpret_cast<float*>(smem + C::kMiscOff);      // [2][N] kBias - running maximum (log2 units)
  float* q_mul = less_max + 2 * N;                                     // [2][N] (4 bits)
  int32_t* row_pos = reinterpret_cast<int32_t*>(q_mul + 2 * N);        // [2][N]
  float* warp_max = reinterpret_cast<float*>(row_pos + 2 * N);         // [8][NC]
  float* warp_sum = warp_max + 8 * NC;                                 // [8][NC]
  float* move_by = warp_sum + 8 * NC;                                  // [N]
  float* row_inv = move_by + N;                                        // [N]
  Bars& B = *reinterpret_cast<Bars*>(smem + C::kBarOff);
  volatile uint32_t* abort_flag = &B.abort;

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(kFull, tid >> 5, 0);
  constexpr int kProd0 = kSoftWarps, kMmaWarp = kProd0 + C::kProdWarps;  // softmax warps first: whole TMEM lane quadrants
  auto fail = [&]() {
    atomicOr(a.status, kErrTimeout);
    *abort_flag = 1u;
  };
  if (tid == 0) {
    mbar_init(&B.q_full, C::kFillers);
    mbar_init(&B.q_free, kQ4 ? 3 : 1);  // the last S^T done; 4 bits: and both softmax halves have seen the factors in place
    mbar_init(&B.r_full, C::kFillers);
    mbar_init(&B.r_free, 1);
    mbar_init(&B.s_full, 1);
    mbar_init(&B.p_full, kSoftThreads);
    mbar_init(&B.o_done, 1);
    mbar_init(&B.o_free, kSoftThreads);
    mbar_init(&B.fin, 1);
    for (int i = 0; i < kMaxRing; ++i) {
      mbar_init(&B.e_full[i], C::kFillers);
      mbar_init(&B.e_free[i], 1);
    }
    B.abort = 0u;
    B.dead[0][0] = B.dead[0][1] = B.dead[1][0] = B.dead[1][1] = 0u;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&B.tmem)),
                 "r"(C::kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  List& own = *reinterpret_cast<List*>(smem + C::kListOff);
  if (C::kOwn && a.own_list) build_list<C::kThreads, kOwnTiles>(a, N, own.off, own.before, own, blockIdx.x == 0);
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = __shfl_sync(kFull, *reinterpret_cast<volatile uint32_t*>(&B.tmem), 0);
  // a warp's lanes wait together; false: give up
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(kFull, phase_wait(bar, parity & 1u, a.wait_ns, abort_flag));
  };

  grid_wait();
  Walk<N, C::kOwn> walk;
  walk.begin(a, own);
  Seg s;
  int g = 0;   // blocks so far
  int tc = 0;  // segments with blocks so far

  if (warp >= kProd0 && warp < kMmaWarp) {
    if constexpr (!kQ4) {
      // ---- producer, 16 bits --------------------------------------------------------------
      const int run = maps.run, runs = kBlk / run;
      int pairs = 0, ropes = 0;  // filled, or being filled
      bool ok = true;
      while (ok && walk.next(a, own, s)) {
        if (s.b0 >= s.b1) continue;
        if (tc >= 1 && !wait(&B.q_free, (uint32_t)(tc - 1))) { ok = false; break; }
        if (lane == 0) mbar_arrive_expect_tx(&B.q_full, kSlabs * C::kQSlab);
        __syncwarp();
        // rows behind the tile's are the next ones' or zeros, and go nowhere
        if (lane < kSlabs) tma_box(sb + C::kQOff + (uint32_t)lane * C::kQSlab, &maps.q, 64 * lane, s.grow, &B.q_full);
        ++tc;
        const int32_t* table = a.table + (int64_t)s.r * a.M;
        // lanes l and l + 16 hold the pool row of a block's run l (-1: not read): of this block, and of the next one,
        // which is already on its way into L2 (the ring has room for little more than one)
        auto find = [&](int b) -> int {
          const int t = s.block(b) * kBlk + (lane & 15) * run;
          if (b >= s.b1 || (lane & 15) >= runs || t > s.pmax || (t + run - 1 < s.lo && t >= a.sinks)) return -1;
          return (int)pool_row(a, table, t);
        };
        int next = find(s.b0);
        for (int b = s.b0; b < s.b1; ++b, ++g) {
          const int row = next;
          next = find(b + 1);
          if (next >= 0)  // half of the run's rows
            prefetch_l2(a.pool + ((int64_t)next + (lane >> 4) * (run / 2)) * kRowBytes16, (uint32_t)(run / 2) * kRowBytes16);
          const uint32_t got = __popc(__ballot_sync(kFull, row >= 0)) >> 1;  // runs
          const uint32_t off = (uint32_t)((lane & 15) * run) * 128u;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int x = 4 * g + i, slot = x % C::kRing, use = x / C::kRing;
            if (use >= 1 && !wait(&B.e_free[slot], (uint32_t)(use - 1))) { ok = false; break; }
            if (lane == 0) mbar_arrive_expect_tx(&B.e_full[slot], got * 2u * (uint32_t)run * 128u);
            __syncwarp();
            pairs = x + 1;
            if (row >= 0 && lane < 16)
              tma_pair(sb + C::kRingOff + (uint32_t)slot * kPair + 2 * off, &maps.pool, 2 * i, row >> 3, &B.e_full[slot]);
          }
          if (!ok) break;
          if (g >= 1 && !wait(&B.r_free, (uint32_t)(g - 1))) { ok = false; break; }
          if (lane == 0) mbar_arrive_expect_tx(&B.r_full, got * (uint32_t)run * 128u);
          __syncwarp();
          ropes = g + 1;
          if (row >= 0 && lane < 16) tma_box(sb + C::kRopeOff + off, &maps.rope, kVal, row, &B.r_full);
        }
      }
      if (!ok) fail();
      // the CTA may not end before its copies have landed (they have, unless a role gave up)
      bool landed = tc == 0 || phase_wait(&B.q_full, (uint32_t)(tc - 1) & 1u, a.wait_ns);
      if (ropes > 0) landed = phase_wait(&B.r_full, (uint32_t)(ropes - 1) & 1u, a.wait_ns) && landed;
      for (int x = max(0, pairs - C::kRing); x < pairs; ++x)
        landed = phase_wait(&B.e_full[x % C::kRing], (uint32_t)(x / C::kRing) & 1u, a.wait_ns) && landed;
      if (!landed) fail();
    } else {
      // ---- producers, 4 bits ------------------------------------------------------------
      // thread (token, side): half `side` of each of pair i's two slabs, so that two lanes read 32 bytes side by side;
      // the scales of slab 2 i + side
      const int pt = tid - kSoftThreads, tok = pt >> 1, side = pt & 1;
      // 16-byte chunk c of this token's 128 bytes lies at (chunk0 + pair or slab) ^ (c << 4)
      const uint32_t rope0 = swz(0u, tok, 0), pair0 = swz_pair(0u, 0, tok, 0);
      Codes k{};
      // The block whose cache block is being looked up runs two blocks ahead of the one being expanded, that whose
      // codes are being read one.
      Walk<N, C::kOwn> far = walk;
      Seg fs;
      int fb = 0, f_in = 0;
      int32_t f_entry = -1;
      bool f_more = far.next(a, own, fs);
      while (f_more && fs.b0 >= fs.b1) f_more = far.next(a, own, fs);
      fb = fs.b0 - 1;
      auto look_up = [&]() {  // the next block's entry of the table
        if (!f_more) return;
        if (++fb >= fs.b1) {
          do f_more = far.next(a, own, fs); while (f_more && fs.b0 >= fs.b1);
          if (!f_more) return;
          fb = fs.b0;
        }
        const int t = fs.block(fb) * kBlk + tok, j = entry_of(a, t);
        f_in = t - j * a.B;
        f_entry = fs.any_sees(a, t) ? __ldg(a.table + (int64_t)fs.r * a.M + j) : -1;
      };
      const uint8_t *crow = nullptr, *srow = nullptr;  // null: zeros
      auto locate = [&]() {
        crow = nullptr;
        if (f_entry >= 0 && (int64_t)f_entry < a.n_blocks) {
          const uint8_t* base = a.pool + (int64_t)f_entry * (a.B * kRowBytesQ4);
          crow = base + f_in * kCodeBytes;
          srow = base + a.B * kCodeBytes + f_in * kGroups;
        }
      };
      auto load_pair = [&](int i) {
        k.c[i][0] = k.c[i][1] = make_uint4(0u, 0u, 0u, 0u);
        k.s[i] = 0u;
        if (crow) {
          const uint4* p = reinterpret_cast<const uint4*>(crow + i * 64 + side * 16);
          k.c[i][0] = __ldg(p);
          k.c[i][1] = __ldg(p + 2);
          k.s[i] = __ldg(reinterpret_cast<const uint32_t*>(srow + (2 * i + side) * 4));
        }
      };
      auto load_rope = [&]() {
        k.rc = make_uint4(0u, 0u, 0u, 0u);
        k.rs = 0u;
        if (crow) {
          k.rc = __ldg(reinterpret_cast<const uint4*>(crow + 256 + side * 16));
          k.rs = __ldg(reinterpret_cast<const uint16_t*>(srow + 32 + side * 2));
        }
      };
      look_up();
      bool pre = f_more;
      if (pre) {
        locate();
#pragma unroll
        for (int i = 0; i < 4; ++i) load_pair(i);
        load_rope();
        look_up();
      }
      bool ok = true;
      while (ok && walk.next(a, own, s)) {
        if (s.b0 >= s.b1) continue;
        if (tc >= 1 && !wait(&B.q_free, (uint32_t)(tc - 1))) { ok = false; break; }
        // queries: one warp per row; scaled by 2^-e so that the largest magnitude is in [2^14, 2^15)
        for (int r = warp - kProd0; r < N; r += C::kProdWarps) {
          const uint4* src = reinterpret_cast<const uint4*>(a.q + (int64_t)(s.grow + r) * kRow);
          uint4 v[3];
          uint32_t top = 0u;
#pragma unroll
          for (int m = 0; m < 3; ++m) {
            const int c = lane + 32 * m;
            v[m] = make_uint4(0u, 0u, 0u, 0u);
            if (r < s.nrows && c < 72) v[m] = __ldg(src + c);
            const uint32_t w[4] = {v[m].x, v[m].y, v[m].z, v[m].w};
#pragma unroll
            for (int x = 0; x < 4; ++x) top = max(top, max(w[x] & 0x7fffu, (w[x] >> 16) & 0x7fffu));
          }
          top = __reduce_max_sync(kFull, top);
          const int e = min(max((int)(top >> 7) - 127 - 14, -112), 112);
          const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
          for (int m = 0; m < 3; ++m) {
            const int c = lane + 32 * m;
            if (c < 72) {
              const uint32_t w[4] = {v[m].x, v[m].y, v[m].z, v[m].w};
              uint32_t h[4];
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const __half2 p = __floats2half2_rn(bf_lo(w[x]) * down, bf_hi(w[x]) * down);
                h[x] = *reinterpret_cast<const uint32_t*>(&p);
              }
              st_v4(swz(sb + C::kQOff + (uint32_t)(c >> 3) * C::kQSlab, r, c & 7), make_uint4(h[0], h[1], h[2], h[3]));
            }
          }
          if (lane == 0) q_mul[(tc & 1) * N + r] = a.scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23);
        }
        mbar_arrive(&B.q_full);
        ++tc;
        for (int b = s.b0; b < s.b1; ++b, ++g) {
          pre = f_more;
          if (pre) {
            locate();
            look_up();
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int x = 4 * g + i, slot = x % C::kRing, use = x / C::kRing;
            if (use >= 1 && !wait(&B.e_free[slot], (uint32_t)(use - 1))) { ok = false; break; }
            // eight lanes, both halves of four tokens' rows, write eight different chunks
            const uint32_t dst = (sb + C::kRingOff + (uint32_t)slot * kPair + pair0) ^ (uint32_t)side << 6;
            const uint32_t other = __shfl_xor_sync(kFull, k.s[i], 1);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              uint32_t s0, s1;
              scales2(__byte_perm(side == p ? k.s[i] : other, 0u, side ? 0x4432 : 0x4410), s0, s1);
              const uint4 c = k.c[i][p];
              uint4 x[4];
              expand16(c.x, c.y, s0, x[0], x[1]);
              expand16(c.z, c.w, s1, x[2], x[3]);
#pragma unroll
              for (int q = 0; q < 4; ++q) st_v4((dst + (uint32_t)p * kAtom) ^ (uint32_t)q << 4, x[q]);
            }
            mbar_arrive(&B.e_full[slot]);
            if (pre) load_pair(i);
          }
          if (!ok) break;
          if (g >= 1 && !wait(&B.r_free, (uint32_t)(g - 1))) { ok = false; break; }
          const uint32_t dst = (sb + C::kRopeOff + rope0) ^ (uint32_t)side << 6;
          uint32_t s0, s1;
          scales2(k.rs, s0, s1);
          uint4 lo, hi;
          expand16(k.rc.x, k.rc.y, s0, lo, hi);
          st_v4(dst, lo);
          st_v4(dst ^ 1u << 4, hi);
          expand16(k.rc.z, k.rc.w, s1, lo, hi);
          st_v4(dst ^ 2u << 4, lo);
          st_v4(dst ^ 3u << 4, hi);
          mbar_arrive(&B.r_full);
          if (pre) load_rope();
        }
      }
      if (!ok) fail();
    }
  } else if (warp == kMmaWarp) {
    // ---- MMA issue ------------------------------------------------------------------------
    // The proxy fences stand here, behind the waits, for the bytes that other threads wrote with ordinary stores: in
    // the writers, a fence waits for whatever the thread still has to load.
    const uint32_t el = elect();
    constexpr uint32_t kIdS = idesc(!kQ4, kBlk, N, false, false);
    constexpr uint32_t kIdO = idesc(!kQ4, kBlk, N, true, C::kSharedP);
    const uint32_t ring_k = sdesc(sb + C::kRingOff, 16);     // K-major slabs
    const uint32_t ring_v = sdesc(sb + C::kRingOff, kAtom);  // MN-major: two slabs, 128 value elements
    const uint32_t rope = sdesc(sb + C::kRopeOff, 16);
    const uint32_t qd = sdesc(sb + C::kQOff, 16);
    const uint32_t pd = sdesc(sb + C::kPOff, 16);
    bool ok = true;
    while (ok && walk.next(a, own, s)) {
      if (s.b0 >= s.b1) continue;
      if (!wait(&B.q_full, (uint32_t)tc)) { ok = false; break; }
      for (int b = s.b0; b < s.b1; ++b, ++g) {
        const uint32_t dS = tmem + C::kColS;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int x = 4 * g + i, slot = x % C::kRing, use = x / C::kRing;
          if (!wait(&B.e_full[slot], (uint32_t)use)) { ok = false; break; }
          fence_proxy_async_smem();
          tc_after();
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ss<kDescHighRing>(
                   dS, ring_k + (((uint32_t)slot * kPair + (uint32_t)(kk >> 2) * kAtom) >> 4) + (uint32_t)((kk & 3) * 2),
                   qd + (((uint32_t)(2 * i + (kk >> 2)) * C::kQSlab) >> 4) + (uint32_t)((kk & 3) * 2), kIdS,
                   (i | kk) ? 1u : 0u, el);
        }
        if (!ok || !wait(&B.r_full, (uint32_t)g)) { ok = false; break; }
        fence_proxy_async_smem();
        tc_after();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ss<kDescHigh>(dS, rope + (uint32_t)(kk * 2), qd + ((8u * C::kQSlab) >> 4) + (uint32_t)(kk * 2), kIdS, 1u, el);
        mma_commit(&B.s_full, el);
        if (!C::kSharedP) mma_commit(&B.r_free, el);
        if (b + 1 == s.b1) mma_commit(&B.q_free, el);
        if (!wait(&B.p_full, (uint32_t)g)) { ok = false; break; }
        if (b == s.b0 && tc >= 1 && !wait(&B.o_free, (uint32_t)(tc - 1))) { ok = false; break; }
        fence_proxy_async_smem();
        tc_after();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int slot = (4 * g + i) % C::kRing;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            // P^T: N = 64 MN-major (16 tokens are 2 KB), else K-major (64 tokens a slab of N rows)
            const uint32_t p = C::kSharedP ? pd + ((uint32_t)kk * 2048u >> 4)
                                           : pd + (((uint32_t)(kk >> 2) * (N * 128u)) >> 4) + (uint32_t)((kk & 3) * 2);
            mma_ss<kDescHighRing>(tmem + (uint32_t)(i * N), ring_v + (((uint32_t)slot * kPair + (uint32_t)kk * 4 * kAtom) >> 4),
                                  p, kIdO, (b > s.b0 || kk > 0) ? 1u : 0u, el);
          }
          mma_commit(&B.e_free[slot], el);
        }
        if (C::kSharedP) mma_commit(&B.r_free, el);
        if (b + 1 == s.b1) mma_commit(&B.o_done, el);
      }
      ++tc;
    }
    if (!ok) fail();
    // everything issued is complete before TMEM is freed (the tensor pipe waits on nothing outside this CTA)
    mma_commit(&B.fin, el);
    if (!__all_sync(kFull, phase_wait(&B.fin, 0, a.wait_ns > 2000000000ull ? a.wait_ns : 2000000000ull))) fail();
  } else {
    // ---- softmax ---------------------------------------------------------------------------
    const int st = tid, hw = warp >> 2, quad = warp & 3;  // half of the rows; lane quadrant
    const int tok = 32 * quad + lane;                     // this thread's token of a block
    const int c0 = hw * NC;                               // its first row of the tile
    const uint32_t lane_addr = (uint32_t)(32 * quad) << 16;
    const uint32_t bar_half = 1u + (uint32_t)hw;          // 128 threads with the same rows
    // A warp whose wait expires still meets the others of its half at their next barrier and tells them there, so
    // that all four leave together: the flag of a barrier is set before it and read after it, and no warp can be two
    // barriers that carry one ahead of another.
    int meets = 0;
    bool dead = false;
    auto meet = [&](bool vote, bool& any) -> bool {  // false: leave
      volatile uint32_t* f = &B.dead[meets & 1][hw];
      ++meets;
      if (dead) *f = 1u;
      any = named_any(bar_half, 128, vote);
      return *f == 0u;
    };
    bool ok = true, any;
    // kAhead: the next tile is looked up behind the first block's weights, when these warps have time
    Seg after;
    bool more = walk.next(a, own, after);
    while (ok && more) {
      s = after;
      if (s.b0 >= s.b1) {  // nothing visible
        more = walk.next(a, own, after);
        for (int i = st; i < s.nrows * (kVal / 8); i += kSoftThreads)
          reinterpret_cast<uint4*>(a.out + (int64_t)s.grow * kVal)[i] = make_uint4(0u, 0u, 0u, 0u);
        if (a.lse && st < s.nrows) a.lse[s.grow + st] = -INFINITY;
        continue;
      }
      float* lm = less_max + (tc & 1) * N;
      int32_t* pos = row_pos + (tc & 1) * N;
      const float* qm = q_mul + (tc & 1) * N;
      if (quad == 0 && lane < NC) {
        lm[c0 + lane] = C::kBias - kNone;
        pos[c0 + lane] = s.pos0 + (s.row0 + min(c0 + lane, s.nrows - 1)) / a.H;
      }
      if (kQ4) {  // the factors; the next tile's queries may not be announced before both halves have seen these
        dead = dead || !wait(&B.q_full, (uint32_t)tc);
      }
      if (!meet(false, any)) { ok = false; break; }
      if (kQ4 && quad == 0 && lane == 0) mbar_arrive(&B.q_free);
      const int32_t* table = a.table + (int64_t)s.r * a.M;
      float l[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) l[c] = 0.f;
      auto mapped = [&](int b) -> bool {
        const int t = s.block(b) * kBlk + tok;
        return b < s.b1 && s.any_sees(a, t) && pool_row(a, table, t) >= 0;
      };
      bool here_next = mapped(s.b0);
      for (int b = s.b0; b < s.b1; ++b, ++g) {
        const bool here = here_next;
        here_next = mapped(b + 1);
        const int t = s.block(b) * kBlk + tok;
        // the token is seen by every position of the tile, or by some
        const bool all = here && t <= s.pmin && (a.window == 0 || t > s.pmax - a.window || t < a.sinks);
        const bool plain = __all_sync(kFull, all);
        // bit c: row c0 + c sees the token.  Position p sees token t when p - t is in [0, span).
        uint32_t vis = kFull;
        if (!plain) {
          const uint32_t span = !here ? 0u : (a.window == 0 || t < a.sinks) ? 0x7fffffffu : (uint32_t)a.window;
          vis = 0u;
#pragma unroll
          for (int c = 0; c < NC; c += 4) {
            const int4 p = *reinterpret_cast<const int4*>(pos + c0 + c);
            vis |= (uint32_t)((uint32_t)(p.x - t) < span) << c;
            vis |= (uint32_t)((uint32_t)(p.y - t) < span) << (c + 1);
            vis |= (uint32_t)((uint32_t)(p.z - t) < span) << (c + 2);
            vis |= (uint32_t)((uint32_t)(p.w - t) < span) << (c + 3);
          }
        }
        dead = dead || !wait(&B.s_full, (uint32_t)g);
        tc_after();
        const uint32_t sS = tmem + lane_addr + C::kColS + (uint32_t)c0;
        float v[NC];
        // v: scores in log2 units less the running maximum (plus kBias); -inf where hidden.  Where the maximum has
        // just moved the product is rounded as the maximum was, so that its own score is no less than 0 however
        // large it is; else the two are fused.
        bool odd = false;  // the token's raw scores are not finite: so is, or may be, its row
        auto scores = [&](auto fused) {
          auto less = [&](float x, float m, float y) {
            return decltype(fused)::value ? fmaf(x, m, y) : __fadd_rn(__fmul_rn(x, m), y);
          };
          tmem_ld<NC>(sS, v);
          tmem_wait_ld();
          odd = !(fabsf(v[0]) < INFINITY);
#pragma unroll
          for (int c = 0; c < NC; c += 4) {
            const float4 x = *reinterpret_cast<const float4*>(lm + c0 + c);
            float4 y = make_float4(a.scale_log2, a.scale_log2, a.scale_log2, a.scale_log2);
            if (kQ4) y = *reinterpret_cast<const float4*>(qm + c0 + c);
            v[c] = less(v[c], y.x, x.x);
            v[c + 1] = less(v[c + 1], y.y, x.y);
            v[c + 2] = less(v[c + 2], y.z, x.z);
            v[c + 3] = less(v[c + 3], y.w, x.w);
          }
          if (!plain) {
#pragma unroll
            for (int c = 0; c < NC; ++c) v[c] = (vis >> c) & 1u ? v[c] : -INFINITY;
          }
        };
        scores(std::true_type{});
        float top = v[0];
#pragma unroll
        for (int c = 1; c < NC; ++c) top = fmaxf(top, v[c]);
        if (!meet(b == s.b0 || top > C::kRescale + C::kBias, any)) { ok = false; break; }
        if (any) {
          // the tokens' maximum of each row; then the running maximum, the sums and O^T move to it
          tmem_ld<NC>(sS, v);
          tmem_wait_ld();
          int32_t mine = 0;
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const float x = (vis >> c) & 1u ? __fmul_rn(v[c], kQ4 ? qm[c0 + c] : a.scale_log2) : -INFINITY;
            const int32_t w = __reduce_max_sync(kFull, as_ordered(x));
            if (lane == c) mine = w;
          }
          if (lane < NC) warp_max[warp * NC + lane] = __int_as_float(as_ordered(__int_as_float(mine)));
          named_sync(bar_half, 128);
          if (quad == 0 && lane < NC) {
            const float* wm = warp_max + 4 * hw * NC + lane;
            const float old = C::kBias - lm[c0 + lane];
            const float now = fmaxf(old, fmaxf(fmaxf(wm[0], wm[NC]), fmaxf(wm[2 * NC], wm[3 * NC])));
            lm[c0 + lane] = C::kBias - now;
            move_by[c0 + lane] = ex2(old - now);
          }
          named_sync(bar_half, 128);
#pragma unroll
          for (int c = 0; c < NC; ++c) l[c] *= move_by[c0 + c];
          if (b > s.b0) {
            // s_full came after every earlier MMA, so O^T is at rest
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              tmem_ld<NC>(tmem + lane_addr + (uint32_t)(i * N + c0), v);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < NC; c += 4) {
                const float4 y = *reinterpret_cast<const float4*>(move_by + c0 + c);
                v[c] *= y.x;
                v[c + 1] *= y.y;
                v[c + 2] *= y.z;
                v[c + 3] *= y.w;
              }
#pragma unroll
              for (int c = 0; c < NC; c += 8) tmem_st8(tmem + lane_addr + (uint32_t)(i * N + c0 + c), v + c);
            }
            tmem_wait_st();
          }
          scores(std::false_type{});
          named_sync(bar_half, 128);  // move_by is free
        }
        // weights
        uint32_t p[NC / 2];
#pragma unroll
        for (int c = 0; c < NC; c += 2) {
          const float e0 = v[c] = ex2(v[c]), e1 = v[c + 1] = ex2(v[c + 1]);
          if (kQ4) {
            const __half2 h = __floats2half2_rn(e0, e1);
            p[c / 2] = *reinterpret_cast<const uint32_t*>(&h);
          } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(e0, e1);
            p[c / 2] = *reinterpret_cast<const uint32_t*>(&h);
          }
        }
        if (C::kSharedP) {  // [token][64 rows]
#pragma unroll
          for (int c = 0; c < NC / 8; ++c)
            st_v4(swz(sb + C::kPOff, tok, c0 / 8 + c), make_uint4(p[4 * c], p[4 * c + 1], p[4 * c + 2], p[4 * c + 3]));
        } else {  // [64 tokens of a slab] of each row
          const uint32_t slab = sb + C::kPOff + (uint32_t)(tok >> 6) * (N * 128u);
          const int in = tok & 63;
#pragma unroll
          for (int c = 0; c < NC; ++c)
            st_u16(swz(slab, c0 + c, in >> 3) + (uint32_t)(in & 7) * 2u, (uint16_t)(p[c / 2] >> (16 * (c & 1))));
        }
        if (!plain) {
          // A weight of 0 times a value that is not finite would be NaN: the value elements of rows that a position
          // of the tile does not see (another position's, or what lies in an unread place) that are not finite
          // become 0.  A row with such an element has no finite score (0 times infinity is NaN, and nothing finite
          // comes of either), so the score of any one query tells, and a position that sees the row is not misled.
          uint32_t edge = __ballot_sync(kFull, !all && odd);
          const int i = 2 * hw + (lane >> 4), x4 = 4 * g + i;  // this half's two pairs: 32 chunks of 8 elements
          if (!phase_wait(&B.e_full[x4 % C::kRing], (uint32_t)(x4 / C::kRing) & 1u, a.wait_ns)) fail();  // (S^T has read it)
          const uint32_t pair = sb + C::kRingOff + (uint32_t)(x4 % C::kRing) * kPair;
          while (edge) {
            const int r = 32 * quad + __ffs(edge) - 1;
            edge &= edge - 1u;
            const uint32_t at = swz_pair(pair, (lane >> 3) & 1, r, lane & 7);
            const uint4 x = ld_v4(at);
            constexpr uint32_t kExp = kQ4 ? 0x7c00u : 0x7f80u;
            uint32_t w[4] = {x.x, x.y, x.z, x.w};
            bool bad = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if ((w[e] & kExp) == kExp) { w[e] &= 0xffff0000u; bad = true; }
              if ((w[e] & (kExp << 16)) == (kExp << 16)) { w[e] &= 0x0000ffffu; bad = true; }
            }
            if (bad) st_v4(at, make_uint4(w[0], w[1], w[2], w[3]));
          }
        }
        tc_before();
        mbar_arrive(&B.p_full);
        // the sums keep the weights in fp32; behind the arrival, while the MMAs run (before it, 4 bits at N = 64: 121 us
        // for 119 over one request of 256k)
#pragma unroll
        for (int c = 0; c < NC; ++c) l[c] += v[c];
        if (C::kAhead && b == s.b0) more = walk.next(a, own, after);
      }
      if (!ok) break;
      // sums over the tokens of each row: halves of the rows change lanes until a lane has one (row lane mod NC)
      {
#pragma unroll
        for (int o = NC / 2; o > 0; o >>= 1) {
          const bool up = (lane & o) != 0;
#pragma unroll
          for (int c = 0; c < o; ++c) {
            const float give = up ? l[c] : l[c + o], keep = up ? l[c + o] : l[c];
            l[c] = keep + __shfl_xor_sync(kFull, give, o);
          }
        }
#pragma unroll
        for (int o = NC; o < 32; o <<= 1) l[0] += __shfl_xor_sync(kFull, l[0], o);
        if (lane < NC) warp_sum[warp * NC + lane] = l[0];
      }
      named_sync(bar_half, 128);
      if (quad == 0 && lane < NC) {
        const float* ws = warp_sum + 4 * hw * NC + lane;
        const float sum = (ws[0] + ws[NC]) + (ws[2 * NC] + ws[3 * NC]);
        const int row = c0 + lane;
        row_inv[row] = sum == 0.f ? 0.f : 1.f / sum;
        if (s.part >= 0) {
          float* ml = a.part_ml + ((int64_t)blockIdx.x * 2 + s.part) * 2 * N;
          ml[row] = C::kBias - lm[row];
          ml[N + row] = sum;
        } else if (a.lse && row < s.nrows) {
          a.lse[s.grow + row] = sum == 0.f ? -INFINITY : (log2f(sum) - lm[row]) * 0.6931471805599453f;
        }
      }
      named_sync(bar_half, 128);
      dead = dead || !wait(&B.o_done, (uint32_t)tc);
      tc_after();
#pragma unroll 1
      for (int i = 0; i < 4 && !dead; ++i) {
        float o[NC];
        tmem_ld<NC>(tmem + lane_addr + (uint32_t)(i * N + c0), o);
        tmem_wait_ld();
        const int e = i * 128 + tok;  // value element
        if (s.part >= 0) {
          float* dst = a.part_o + (((int64_t)blockIdx.x * 2 + s.part) * N + c0) * kVal + e;
#pragma unroll
          for (int c = 0; c < NC; ++c)
            if (c0 + c < s.nrows) dst[(size_t)c * kVal] = o[c];
        } else {
          // lanes 2 k and 2 k + 1 trade elements so that each stores a pair: the even one of row c, the odd one of c + 1
          uint16_t* dst = a.out + (int64_t)(s.grow + c0) * kVal + (e & ~1);
          const bool odd = lane & 1;
#pragma unroll
          for (int c = 0; c < NC; c += 2) {
            const float x0 = o[c] * row_inv[c0 + c], x1 = o[c + 1] * row_inv[c0 + c + 1];
            const float y = __shfl_xor_sync(kFull, odd ? x0 : x1, 1);
            const __nv_bfloat162 h = odd ? __floats2bfloat162_rn(y, x1) : __floats2bfloat162_rn(x0, y);
            const int row = c + (odd ? 1 : 0);
            if (c0 + row < s.nrows) *reinterpret_cast<__nv_bfloat162*>(dst + (size_t)row * kVal) = h;
          }
        }
      }
      tc_before();
      mbar_arrive(&B.o_free);
      ++tc;
      if (!C::kAhead) more = walk.next(a, own, after);
    }
    if (!ok || dead) fail();
  }
  tc_before();
  __syncthreads();
  launch_dependents();
  if (warp == kMmaWarp) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmem) : "memory");
  }
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

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

using EncodeTiled = decltype(&cuTensorMapEncodeTiled);

// The driver's tensor-map encoder (the library is linked against the runtime alone).
EncodeTiled encoder() {
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

// [rows][576] bf16 in boxes of 64 elements x box_rows, 128-byte swizzled.
bool encode_rows(CUtensorMap* m, const void* base, int64_t rows, int box_rows) {
  const EncodeTiled fn = encoder();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)kRow, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)kRowBytes16};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, step[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The value elements of the pool's rows as [row / 8][slab][row % 8][64] (the slabs' stride is less than a row's).
bool encode_pairs(CUtensorMap* m, const void* base, int64_t rows, int box_rows) {
  const EncodeTiled fn = encoder();
  if (!fn) return false;
  const cuuint64_t dims[4] = {64, 8, (cuuint64_t)(kVal / 64), (cuuint64_t)(rows / 8)};
  const cuuint64_t strides[3] = {(cuuint64_t)kRowBytes16, 128, 8 * (cuuint64_t)kRowBytes16};
  const cuuint32_t box[4] = {64, 8, 2, (cuuint32_t)(box_rows / 8)}, step[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

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

template <int N, bool kQ4>
cudaError_t launch(const PagedAttendArgs& a, cudaStream_t s) {
  using C = Shape<N, kQ4>;
  static_assert(kMaxWorkers <= kJoinParts, "parts of a tile");
  if (a.n_tokens == 0) return cudaMemsetAsync(a.status, 0, 4, s);
  cudaError_t e;
  static std::atomic<uint64_t> ready{0};  // devices where the kernel may have its shared memory
  const uint64_t bit = a.device < 64 ? 1ull << a.device : 0ull;
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(attend_paged_kernel<N, kQ4>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  Maps maps{};
  if (!kQ4) {
    maps.run = a.B & -a.B;
    if (maps.run > kBlk) maps.run = kBlk;
    if (!encode_pairs(&maps.pool, a.pool, a.n_blocks * a.B, maps.run) ||
        !encode_rows(&maps.rope, a.pool, a.n_blocks * a.B, maps.run) ||
        !encode_rows(&maps.q, a.q, (int64_t)a.n_tokens * a.H, N))
      return cudaErrorInvalidValue;
  }
  if (a.own_list) {
    attend_paged_kernel<N, kQ4><<<a.workers, C::kThreads, C::kSmem, s>>>(a, maps);
    e = cudaGetLastError();
  } else {
    if (a.few_tiles)
      schedule_paged_kernel<kOwnTiles, kOwnTiles, kOwnTiles><<<1, kOwnTiles, 0, s>>>(a, N);
    else
      schedule_paged_kernel<kSchedThreads, kListTiles, kMaxRequests><<<1, kSchedThreads, 0, s>>>(a, N);
    e = cudaGetLastError();
    if (e == cudaSuccess) e = launch_after(attend_paged_kernel<N, kQ4>, a.workers, C::kThreads, C::kSmem, s, a, maps);
  }
  if (e == cudaSuccess) e = launch_after(join_paged_kernel<N>, 4 * a.workers, kJoinThreads, 0, s, a, C::kBias);
  return e;
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
cudaError_t launch_paged_attend(const PagedAttendArgs& args, bool q4, cudaStream_t s) {
  PagedAttendArgs a = args;
  const int N = paged_tile_rows(a.R, a.n_tokens, a.H);
  // A list that is short whatever the requests' shares of the tokens are is built by each CTA: no launch before the
  // attention.  Measured, 16 heads: one request of 4k 15.0 us, with the kernel that lists 17.7; 64 of 1k 22.0 and 24.0; at
  // the limit, 128 of 1k 37.5 and 41.2, one chunk of 1,016 tokens 144.6 and 150.6.
  a.few_tiles = a.R <= kOwnTiles && a.R + ((int64_t)a.n_tokens * a.H + N - 1) / N <= kOwnTiles;
  a.own_list = !(q4 && N == 64) && a.few_tiles;
  if (q4) return N == 16 ? launch<16, true>(a, s) : N == 32 ? launch<32, true>(a, s) : launch<64, true>(a, s);
  return N == 16 ? launch<16, false>(a, s) : N == 32 ? launch<32, false>(a, s) : launch<64, false>(a, s);
}

}  // namespace kvo
