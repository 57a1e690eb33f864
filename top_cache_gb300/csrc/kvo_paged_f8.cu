// Attention over the paged device cache in 8 bits (E4M3 codes, a power of two a
// row), on the 5th-generation tensor cores in their 8-bit form.
//
// The formula, the tiles and their split over the CTAs are those of
// kvo_paged_attend.cuh: S^T = K Q^T (128 tokens x the tile's N rows), O^T = V^T
// P^T (128 value elements x N).  Here the codes are the operand as they lie in
// the cache: no expansion, and half the bytes of 16 bits everywhere.  What the
// 8-bit products need:
//   queries  q = 2^e (hi + lo / 16), both E4M3: a bf16 value has 8 significant
//            bits, two codes of 4, so the pair is exact down to 2^-14 of the
//            row's largest.  hi and lo are 2 N columns of one product; the
//            scores are D_hi + D_lo / 16, times 2^e and the token's scale.
//   weights  the token's scale t = 2^x goes into the weight: P' = 2^(s + x - m'),
//            m' the running maximum of s + x.  P' is rounded to fp16 and split
//            into three E5M2 codes, each the nearest to what the ones before
//            leave: together off by at most 2^-10 of P', where a bf16 weight is
//            off by 2^-8.  E5M2 for its range: E4M3 codes of the rest, one bit
//            finer, end 2^-17 below the largest weight, and the weights that
//            share what an attention sink leaves lie there (2^-14 of the sink's:
//            outputs off by 3 %).  At N = 16 and 32 the codes are 3 N columns of
//            one product, with sums of their own, and count 1, 2^-4 and 2^-8:
//            2^-8 of a weight down to 2^-26 of the largest.  At N = 64 TMEM has
//            room for one set of sums, which take all three products: 2^-8 down
//            to 2^-20 of the largest, and nothing is off by more than 2^-28 of
//            it.  The sum that divides is of P' / t in fp32.
// A product of E4M3 and E4M3 or E5M2 with fp32 sums is exact but for the sums'
// truncation (measured: 2^-22 of the sum of magnitudes).
//
// One persistent CTA per SM: 8 softmax warps (which also split the next tile's
// queries, as soon as this one's scores are done), a copy warp and an MMA warp.
// The ring has 4 pairs of slabs (two blocks) at N = 64 and 5 below.  S^T has two
// places in TMEM: the next block's is issued before this one's O^T, so that the
// softmax of one block runs beside the products of another.  At N = 64 shared
// memory has no room for the third codes: they lie where the next block's rope
// keys have been, between its S^T and their part of O^T, and come behind an
// arrival of their own while the first two run (597 us over 32 trees of 64 nodes of
// 16k; behind one arrival 638).  A block's rope keys are loaded and used between its
// pairs, and the third codes' products come before the second pair's others, so that
// their place is free early (4,690 clocks a block; rope keys last 4,890).  Every wait
// is bounded, as there.
//
// What bounds it.  N = 16: HBM, 32 ragged requests of 64k, 16 heads, in 136 us
// (6.4 TB/s, 0.93 of the copy rate; with what joins them 143).  The cache's bytes
// are all it reads (ncu: 863 of 862 MB).  Two loads a token stand in the way, its
// table entry and its scale: they are made two blocks and one block ahead and
// the scales are fetched into L2 with the codes (157 us before).  N = 64: 4,700
// clocks a block of 128 tokens.  The products take 1,200 (S^T, 18 of 64 to 78
// clocks) and 2,400 to 3,300 (O^T, 48 of 50 to 69), and their warp waits 750 for the
// next block's codes, whose places the last products free, 240 for its rope keys and
// 440 for weights; the softmax, 3,500, runs beside.  (With two codes 4,200.  The
// 16-bit kernel takes 4,800 and the 4-bit one 6,200.)  These kernels spill 24 to 28
// bytes a thread at 168 registers.  Borders of tiles cost 10,000: the queries 3,000
// to 4,000, the output or the parts 4,000 to 6,000 (64 rows of 2 KB).
// Tried and not faster: four warps of their own for the queries (a latency of
// memory a row: 106 us for 82 over 16 x 4 positions of 128 heads of 8k), votes on
// the running maximum counted behind the weights (73 for 70), 32 columns of TMEM a
// load, all of a tile's queries loaded before any is split (76 for 71), one arrival a
// warp at the barriers.  (Figures of the two-code kernel.)
// Tiles, us with N = 16, 32, 64: 16 requests of 32k and 16 rows 65, 73, 101; 24 rows
// 107, 74, 103; 48 rows 153, 116, 104; 128 rows 356, 200, 174: the rule of the other
// formats holds.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "kvo_paged_walk.cuh"

namespace kvo {

using namespace paged;

namespace {

constexpr uint32_t kSlabF8 = kBlk * 128;       // 128 tokens x 128 elements
constexpr uint32_t kPairF8 = 2 * kSlabF8;      // two slabs, in atoms of 8 tokens of each in turn
constexpr uint32_t kRopeF8 = kBlk * 64;
constexpr int kPairs = 2;                      // pairs of a block
constexpr int kMaxPairs = 5, kMaxRopes = 3;

template <int N>
struct ShapeF8 {
  static constexpr int kThreads = kSoftThreads + 64;
  static constexpr int kNC = N / 2;                        // rows of one softmax thread
  static constexpr bool kApart = N != 64;                  // the three codes of a weight have sums of their own in TMEM
  static constexpr int kRing = N == 64 ? 4 : kMaxPairs;    // pairs
  static constexpr int kRopes = N == 16 ? kMaxRopes : 1;
  static constexpr bool kOwn = N != 64;                    // room for a list of its own
  static constexpr uint32_t kQSlab = 2 * N * 128;          // hi rows, lo rows
  static constexpr uint32_t kQRopeOff = 4 * kQSlab;
  static constexpr uint32_t kRingOff = kQRopeOff + 2 * N * 64;
  static constexpr uint32_t kRopeOff = kRingOff + kRing * kPairF8;
  static constexpr uint32_t kPOff = kRopeOff + kRopes * kRopeF8;
  static constexpr uint32_t kPPart = N * 128;              // a code of every weight: hi, mid and lo
  static constexpr uint32_t kLastOff = kApart ? kPOff + 2 * kPPart : kRopeOff;  // lo; N = 64: in the rope keys' place
  static constexpr uint32_t kMiscOff = kPOff + (kApart ? 3 : 2) * kPPart;
  // misc: less running maxima, row positions, a tree's nodes [N], query factors [2][N], factors of a move of the running
  // maximum or 1 / l [N], a block's maxima or the tile's sums [8][NC]
  static constexpr uint32_t kMiscBytes = (6 * N + 8 * kNC) * 4;
  static constexpr uint32_t kBarOff = kMiscOff + kMiscBytes;
  static constexpr uint32_t kListOff = kBarOff + 256;
  static constexpr uint32_t kSmem = kListOff + (kOwn ? 2400 : 0);
  static constexpr uint32_t kSums = (kApart ? 3 : 1) * N;  // columns of O^T for 128 value elements
  static constexpr uint32_t kColS = 4 * kSums;             // S^T, twice 2 N
  static constexpr uint32_t kTmem = kColS + 4 * N;
  // log2 of the largest weight when the running maximum has moved, and how far a score may pass it (fp16 and E5M2 end
  // behind 2^15).  Codes end at 2^-16, half a step off: 2^-28 of the largest at N = 64.  9 and 6 there move the maximum less
  // often, 4,000 clocks each, but end at 2^-26: 16 x 4 positions of 128 heads over 8k 80 us for 85, a windowed chunk of 2,048
  // tokens 194 for 201, 32 trees of 64 nodes over 16k 590 for 598.
  static constexpr float kBias = kApart ? 9.f : 11.f;
  static constexpr float kRescale = 15.f - kBias;
  static_assert(kSmem <= 232448, "shared memory of one CTA");
  static_assert(kRingOff % 1024 == 0 && kRopeOff % 1024 == 0 && kPOff % 1024 == 0 && kBarOff % 8 == 0,
                "swizzled tiles sit on 1 KB boundaries");
};

// High words of matrix descriptors: distance of groups of 8 rows (or tokens), version, swizzle (2: 128 bytes, 4: 64, 6: 32).
constexpr uint32_t desc_high(uint32_t group, uint32_t swizzle) { return (group >> 4) | (1u << 14) | (swizzle << 29); }
constexpr uint32_t kHighPair = desc_high(2 * kAtom, 2), kHigh128 = desc_high(1024, 2), kHigh64 = desc_high(512, 4),
                   kHigh32 = desc_high(256, 6);
// Instruction descriptor of kind::f8f6f4, fp32 sums: A E4M3; B E4M3 or E5M2.
constexpr uint32_t idesc8(bool b_e5m2, int N, bool a_mn_major, bool b_mn_major) {
  return (1u << 4) | ((b_e5m2 ? 1u : 0u) << 10) | ((a_mn_major ? 1u : 0u) << 15) | ((b_mn_major ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kBlk >> 4) << 24);
}
template <uint32_t kHighA, uint32_t kHighB>
__device__ __forceinline__ void mma8(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc, uint32_t el) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "mov.b64 da, {%1, %6};\n\tmov.b64 db, {%2, %7};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(acc), "r"(el), "n"(kHighA), "n"(kHighB)
      : "memory");
}
// 16-byte chunk c of row r in tiles of 64- and 32-byte rows.
__device__ __forceinline__ uint32_t swz64(uint32_t tile, int r, int c) {
  return tile + (uint32_t)r * 64u + ((uint32_t)(c ^ ((r >> 1) & 3)) << 4);
}
__device__ __forceinline__ uint32_t swz32(uint32_t tile, int r, int c) {
  return tile + (uint32_t)r * 32u + ((uint32_t)(c ^ ((r >> 2) & 1)) << 4);
}
__device__ __forceinline__ void st_v2(uint32_t addr, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void st_u8(uint32_t addr, uint32_t v) {
  asm volatile("{\n\t.reg .b8 t, u0, u1, u2;\n\tmov.b32 {t, u0, u1, u2}, %1;\n\tst.shared.b8 [%0], t;\n\t}" ::"r"(addr), "r"(v)
               : "memory");
}
// Codes of two slabs of `run` rows of a cache block: see MapsF8.
__device__ __forceinline__ void tma_codes(uint32_t dst, const CUtensorMap* map, int slab, int group, int block, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %3, %4, %5}], [%6];" ::"r"(
          dst),
      "l"(map), "r"(0), "r"(slab), "r"(group), "r"(block), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_rope(uint32_t dst, const CUtensorMap* map, int row, int block, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(0), "r"(row), "r"(block), "r"(smem_u32(bar))
      : "memory");
}
// Two weights (at most 2^15) -> three E5M2 codes, each to nearest, of what the ones before leave; kBy: 16 where mid and lo
// have sums of their own, and count 2^-4 and 2^-8, else 1.  An E5M2 code is the high byte of fp16, and leaves at most an
// eighth of the power of two below its value: exact in fp16, and times 16 no larger than that power.  hi, mid: bytes 1
// and 3; lo: the low 16 bits.  A NaN is one in lo.
__device__ __forceinline__ uint32_t high_code(__half2 h) {
  return (*reinterpret_cast<const uint32_t*>(&h) + 0x00800080u) & 0xff00ff00u;
}
template <int kBy>
__device__ __forceinline__ void split_weights(float x, float y, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y), by = __float2half2_rn((float)kBy);
  hi = high_code(h);
  __half2 rest = __hsub2(h, *reinterpret_cast<const __half2*>(&hi));
  if (kBy != 1) rest = __hmul2(rest, by);
  mid = high_code(rest);
  rest = __hsub2(rest, *reinterpret_cast<const __half2*>(&mid));
  if (kBy != 1) rest = __hmul2(rest, by);
  lo = (uint32_t)__nv_cvt_halfraw2_to_fp8x2(__half2_raw(rest), __NV_SATFINITE, __NV_E5M2);
}

// A load where `on`, else `other`, issued where it stands (an ordinary one is moved down to its use, a block later) and
// without a branch (whose end waits for it).
__device__ __forceinline__ uint32_t load_if(bool on, const void* p, uint32_t other) {
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t@q ld.global.nc.b32 %0, [%1];\n\t}"
               : "+r"(other)
               : "l"(p), "r"((uint32_t)on));
  return other;
}

struct BarsF8 {
  uint64_t q_full, p_full, l_full, l_free, o_step, o_done, o_free, fin;
  uint64_t s_full[2], r_full[kMaxRopes], r_free[kMaxRopes], e_full[kMaxPairs], e_free[kMaxPairs];
  uint32_t tmem, abort;
  uint32_t dead[2][2];  // softmax: a warp of the half gave up, by parity of the barrier's count
};
static_assert(sizeof(BarsF8) <= 256 && sizeof(List) <= 2400, "barriers; the CTA's own list");

// The pool in boxes of `run` rows (the largest power of two, at most 128, that divides block_tokens): codes as
// [block][group of 8 rows][slab][8][128], a box has two slabs; rope keys [block][row][64].
struct MapsF8 {
  CUtensorMap codes, rope;
  int run;
};

template <int N, bool kTree>
__global__ void __launch_bounds__(ShapeF8<N>::kThreads, 1)
    attend_paged_f8_kernel(PagedAttendArgs a, const __grid_constant__ MapsF8 maps) {
  using C = ShapeF8<N>;
  constexpr int NC = C::kNC;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  if (sb & 1023u) {  // there is no room to align it here: nothing is computed, and nothing joined
    grid_wait();     // (the list's launch writes both)
    if (threadIdx.x == 0 && blockIdx.x == 0) {
      *a.status = kErrPlan;
      a.head[kHdListed] = 0;
    }
    return;
  }
  float* less_max = reinterpret_cast<float*>(smem + C::kMiscOff);      // [N] kBias - running maximum (log2 units)
  int32_t* row_pos = reinterpret_cast<int32_t*>(less_max + N);         // [N]
  int32_t* row_node = row_pos + N;                                     // [N] (kTree)
  float* q_mul = reinterpret_cast<float*>(row_node + N);               // [2][N]
  float* row_f = q_mul + 2 * N;                                        // [N]
  float* warp_red = row_f + N;                                         // [8][NC]
  BarsF8& B = *reinterpret_cast<BarsF8*>(smem + C::kBarOff);
  volatile uint32_t* abort_flag = &B.abort;

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(kFull, tid >> 5, 0);
  constexpr int kCopyWarp = kSoftWarps, kMmaWarp = kCopyWarp + 1;  // softmax warps first: whole TMEM lane quadrants
  auto fail = [&]() {
    atomicOr(a.status, kErrTimeout);
    *abort_flag = 1u;
  };
  if (tid == 0) {
    mbar_init(&B.q_full, kSoftThreads);
    mbar_init(&B.p_full, kSoftThreads);
    mbar_init(&B.l_full, kSoftThreads);
    mbar_init(&B.l_free, 1);
    mbar_init(&B.o_step, 1);
    mbar_init(&B.o_done, 1);
    mbar_init(&B.o_free, kSoftThreads);
    mbar_init(&B.fin, 1);
    mbar_init(&B.s_full[0], 1);
    mbar_init(&B.s_full[1], 1);
    for (int i = 0; i < kMaxRopes; ++i) {
      mbar_init(&B.r_full[i], 1);
      mbar_init(&B.r_free[i], 1);
    }
    for (int i = 0; i < kMaxPairs; ++i) {
      mbar_init(&B.e_full[i], 1);
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
  if (C::kOwn && a.own_list) build_list<C::kThreads, kOwnTiles, kTree>(a, N, own.off, own.before, own, blockIdx.x == 0);
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = __shfl_sync(kFull, *reinterpret_cast<volatile uint32_t*>(&B.tmem), 0);
  // a warp's lanes wait together; false: give up
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(kFull, phase_wait(bar, parity & 1u, a.wait_ns, abort_flag));
  };

  grid_wait();
  Walk<N, C::kOwn, kTree> walk;
  walk.begin(a, own);
  Seg s;
  int g = 0;   // blocks so far
  int tc = 0;  // segments with blocks so far
  const int64_t block_bytes = (int64_t)a.B * kRowBytesF8;

  if (warp == kCopyWarp) {
    // ---- copies: lane l < 16 (and l + 16) holds the cache block and row of a block's run l (-1: not read): of this block,
    // and of the next one --------------------------------------------------------------------------
    const int run = maps.run, runs = kBlk / run;
    int pairs = 0, ropes = 0;  // filled, or being filled
    bool ok = true;
    while (ok && walk.next(a, own, s)) {
      if (s.b0 >= s.b1) continue;
      const int32_t* table = a.table + (int64_t)s.r * a.M;
      auto find = [&](int b, int& in) -> int {
        const int t = s.block(b) * kBlk + (lane & 15) * run;
        if (b >= s.b1 || (lane & 15) >= runs || t > s.pmax || (t + run - 1 < s.lo && t >= a.sinks)) return -1;
        const int j = entry_of(a, t);
        in = t - j * a.B;
        const int32_t blk = __ldg(table + j);
        return blk < 0 || (int64_t)blk >= a.n_blocks ? -1 : blk;
      };
      if (lane == 0 && tc > 0)  // the softmax warps read the tile's queries when the last tile's scores are done
        prefetch_l2(a.q + (int64_t)s.grow * kRow, (uint32_t)s.nrows * (kRow * 2));
      ++tc;
      int in_next = 0, next = find(s.b0, in_next);
      for (int b = s.b0; b < s.b1; ++b, ++g) {
        const int blk = next, in = in_next;
        next = find(b + 1, in_next);
        // The next block into L2, with its scales, which the softmax warps load one by one.  Runs of 8 rows keep the copy
        // unit busy with boxes (three a run) as it is.  32 requests of 32k, 16 heads, us with none, the scales, all in one or
        // two requests, all in two or three: blocks of 8 tokens 143, 154, 154, 191; of 24 145, 157, 177, 196; of 16 130, 136,
        // 117, 128; of 64 126, 126, 109, 110.
        if (run > 8 && next >= 0 && lane < 16) {
          const uint8_t* block = a.pool + next * block_bytes;
          const bool joint = run == a.B;  // they lie behind the run
          prefetch_l2(block + (int64_t)in_next * kRow, (uint32_t)run * (joint ? kRowBytesF8 : kRow));
          if (!joint) prefetch_l2(block + (int64_t)a.B * kRow + 4 * in_next, (uint32_t)run * 4);
        }
        const uint32_t got = __popc(__ballot_sync(kFull, blk >= 0)) >> 1;  // runs
        const uint32_t off = (uint32_t)((lane & 15) * run);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          if (i == 1) {  // the rope keys, which the products take between the pairs
            const int slot = g % C::kRopes, use = g / C::kRopes;
            if (use >= 1 && !wait(&B.r_free[slot], (uint32_t)(use - 1))) { ok = false; break; }
            // N = 64: the last codes of the weights lie there from the next block's S^T (a tile's last block: its own) to
            // their part of O^T
            const int under = b == s.b0 ? g - 1 : g - 2;
            if (!C::kApart && under >= 0 && !wait(&B.l_free, (uint32_t)under)) { ok = false; break; }
            if (lane == 0) mbar_arrive_expect_tx(&B.r_full[slot], got * (uint32_t)run * 64u);
            __syncwarp();
            ropes = g + 1;
            if (blk >= 0 && lane < 16)
              tma_rope(sb + C::kRopeOff + (uint32_t)slot * kRopeF8 + off * 64u, &maps.rope, in, blk, &B.r_full[slot]);
          }
          const int x = kPairs * g + i, slot = x % C::kRing, use = x / C::kRing;
          if (use >= 1 && !wait(&B.e_free[slot], (uint32_t)(use - 1))) { ok = false; break; }
          if (lane == 0) mbar_arrive_expect_tx(&B.e_full[slot], got * (uint32_t)run * 256u);
          __syncwarp();
          pairs = x + 1;
          if (blk >= 0 && lane < 16)
            tma_codes(sb + C::kRingOff + (uint32_t)slot * kPairF8 + off * 256u, &maps.codes, 2 * i, in >> 3, blk, &B.e_full[slot]);
        }
        if (!ok) break;
      }
    }
    if (!ok) fail();
    // the CTA may not end before its copies have landed (they have, unless a role gave up)
    bool landed = true;
    for (int x = max(0, pairs - C::kRing); x < pairs; ++x)
      landed = phase_wait(&B.e_full[x % C::kRing], (uint32_t)(x / C::kRing) & 1u, a.wait_ns) && landed;
    for (int x = max(0, ropes - C::kRopes); x < ropes; ++x)
      landed = phase_wait(&B.r_full[x % C::kRopes], (uint32_t)(x / C::kRopes) & 1u, a.wait_ns) && landed;
    if (!landed) fail();
  } else if (warp == kMmaWarp) {
    // ---- MMA issue: S^T of a block, then O^T of the one before it; a tile's last O^T at once, since the next tile's
    // queries come behind its last weights ----------------------------------------------------------
    // The proxy fences stand here, behind the waits, for the bytes that other threads wrote with ordinary stores.
    const uint32_t el = elect();
    constexpr uint32_t kIdS = idesc8(false, 2 * N, false, false);
    constexpr bool kMnP = N >= 32;  // P^T of a code: [token][N rows], else [row][128 tokens]
    constexpr uint32_t kIdO = idesc8(true, (int)C::kSums, true, kMnP);
    constexpr uint32_t kHighP = N == 64 ? kHigh64 : N == 32 ? kHigh32 : kHigh128;
    constexpr uint32_t kStepP = (kMnP ? 32u * N : 32u) >> 4;  // 32 tokens further
    const uint32_t ring = sdesc(sb + C::kRingOff, 16), rope = sdesc(sb + C::kRopeOff, 16);
    const uint32_t qd = sdesc(sb, 16), qr = sdesc(sb + C::kQRopeOff, 16), ld = sdesc(sb + C::kLastOff, 16);
    const uint32_t pd = sdesc(sb + C::kPOff, kMnP ? C::kPPart : 16);  // (N = 32: the three codes' columns, that far apart)
    bool ok = true, open = false, first = false, last = false;  // of the block whose O^T is to come
    int og = 0, otc = 0;
    auto value = [&]() -> bool {
      if (!wait(&B.p_full, (uint32_t)og)) return false;
      if (first && otc >= 1 && !wait(&B.o_free, (uint32_t)(otc - 1))) return false;
      fence_proxy_async_smem();
      tc_after();
      // chunk x (128 value elements) of the block's codes; 32 tokens kk of them
      auto codes = [&](int x, int kk) -> uint32_t {
        return ring + (((uint32_t)((kPairs * og + (x >> 1)) % C::kRing) * kPairF8 + (uint32_t)(x & 1) * kAtom +
                        (uint32_t)kk * 8 * kAtom) >> 4);
      };
#pragma unroll
      for (int x = 0; x < 4; ++x) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint32_t d = tmem + (uint32_t)x * C::kSums, at = codes(x, kk);
          mma8<kHighPair, kHighP>(d, at, pd + kk * kStepP, kIdO, (!first || kk > 0 || (!C::kApart && x >= 2)) ? 1u : 0u, el);
          if (!C::kApart) mma8<kHighPair, kHighP>(d, at, pd + (C::kPPart >> 4) + kk * kStepP, kIdO, 1u, el);
        }
        if (!C::kApart && x == 1) {
          // the last codes come while these products run, and all their products before the other pair's: the next rope
          // keys wait for their place
          if (!wait(&B.l_full, (uint32_t)og)) return false;
          fence_proxy_async_smem();
          tc_after();
#pragma unroll
          for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma8<kHighPair, kHighP>(tmem + (uint32_t)y * C::kSums, codes(y, kk), ld + kk * kStepP, kIdO,
                                      (!first || y < 2 || kk > 0) ? 1u : 0u, el);
          mma_commit(&B.l_free, el);
        }
        if (x & 1) mma_commit(&B.e_free[(kPairs * og + (x >> 1)) % C::kRing], el);
      }
      mma_commit(&B.o_step, el);
      if (last) mma_commit(&B.o_done, el);
      return true;
    };
    while (ok && walk.next(a, own, s)) {
      if (s.b0 >= s.b1) continue;
      if (!wait(&B.q_full, (uint32_t)tc)) { ok = false; break; }
      for (int b = s.b0; b < s.b1; ++b, ++g) {
        const uint32_t dS = tmem + C::kColS + (uint32_t)(g & 1) * (2 * N);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          if (i == 1) {
            const int slot = g % C::kRopes;
            if (!wait(&B.r_full[slot], (uint32_t)(g / C::kRopes))) { ok = false; break; }
            tc_after();
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
              mma8<kHigh64, kHigh64>(dS, rope + ((uint32_t)slot * kRopeF8 >> 4) + (uint32_t)(kk * 2), qr + (uint32_t)(kk * 2), kIdS, 1u, el);
            mma_commit(&B.r_free[slot], el);
          }
          const int x = kPairs * g + i, slot = x % C::kRing, use = x / C::kRing;
          if (!wait(&B.e_full[slot], (uint32_t)use)) { ok = false; break; }
          fence_proxy_async_smem();
          tc_after();
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma8<kHighPair, kHigh128>(
                dS, ring + (((uint32_t)slot * kPairF8 + (uint32_t)(kk >> 2) * kAtom) >> 4) + (uint32_t)((kk & 3) * 2),
                qd + (((uint32_t)(2 * i + (kk >> 2)) * C::kQSlab) >> 4) + (uint32_t)((kk & 3) * 2), kIdS, (i | kk) ? 1u : 0u, el);
        }
        if (!ok) break;
        mma_commit(&B.s_full[g & 1], el);
        if (open && !value()) { ok = false; break; }
        open = true;
        first = b == s.b0;
        last = b + 1 == s.b1;
        og = g;
        otc = tc;
      }
      if (ok) ok = value();
      open = false;
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
    // A tile's queries: 2^-e brings a row's largest magnitude to at most 448.  A warp has N / 8 rows side by side, up to
    // four at a time: their 16-byte pieces in a line, 72 a row.  Called when this warp has seen the last tile's last scores,
    // so no product reads the queries any more.
    auto convert = [&](const Seg& q, float* mul) {
      constexpr int kRows = N / kSoftWarps, kAt = kRows < 4 ? kRows : 4, kSteps = (kAt * 72 + 31) / 32, kTurns = kRows / kAt;
#pragma unroll 1
      for (int turn = 0; turn < kTurns; ++turn) {
        const int r0 = warp * kRows + turn * kAt, pieces = min(max(q.nrows - r0, 0), kAt) * 72;  // (rows behind the tile's: zeros)
        const uint4* src = reinterpret_cast<const uint4*>(a.q + (int64_t)(q.grow + r0) * kRow);
        uint4 v[kSteps];
#pragma unroll
        for (int m = 0; m < kSteps; ++m) {
          v[m] = make_uint4(0u, 0u, 0u, 0u);
          if (32 * m + lane < pieces) v[m] = __ldg(src + 32 * m + lane);
        }
        uint32_t top[kAt];
#pragma unroll
        for (int k = 0; k < kAt; ++k) top[k] = 0u;
#pragma unroll
        for (int m = 0; m < kSteps; ++m) {
          const uint32_t most = __vmaxu2(__vmaxu2(v[m].x & 0x7fff7fffu, v[m].y & 0x7fff7fffu),
                                         __vmaxu2(v[m].z & 0x7fff7fffu, v[m].w & 0x7fff7fffu));
          const int first = 32 * m / 72, last = (32 * m + 31) / 72;  // the step's rows, one or two
          const bool second = 32 * m + lane >= 72 * last;
          if (first == last) {
            if (first < kAt) top[first] = __vmaxu2(top[first], most);
          } else {
            top[first] = __vmaxu2(top[first], second ? 0u : most);
            if (last < kAt) top[last] = __vmaxu2(top[last], second ? most : 0u);
          }
        }
        float down[kAt];
#pragma unroll
        for (int k = 0; k < kAt; ++k) {
          const uint32_t most = __reduce_max_sync(kFull, max(top[k] & 0xffffu, top[k] >> 16));
          const int e = min(max((int)(most >> 7) - 127 - 8 + ((most & 127u) > 96u ? 1 : 0), -112), 120);
          down[k] = __uint_as_float((uint32_t)(127 - e) << 23);
          // a query that is not finite has no finite score
          if (lane == 0)
            mul[r0 + k] = most < 0x7f80u ? a.scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23) : __int_as_float(0x7fffffff);
        }
#pragma unroll
        for (int m = 0; m < kSteps; ++m) {
          const int i = 32 * m + lane, first = 32 * m / 72, last = (32 * m + 31) / 72;
          const bool second = first != last && i >= 72 * last;
          if (second && last >= kAt) continue;
          const float by = second && last < kAt ? down[last < kAt ? last : 0] : down[first];
          const int row = second ? last : first, c = i - 72 * row, r = r0 + row;
          const uint32_t w[4] = {v[m].x, v[m].y, v[m].z, v[m].w};
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            // (8 bits up to 448 are exact in fp16, down to where they pass the codes' range)
            const __half2 h = __floats2half2_rn(bf_lo(w[x]) * by, bf_hi(w[x]) * by);
            hi[x] = (uint32_t)__nv_cvt_halfraw2_to_fp8x2(__half2_raw(h), __NV_SATFINITE, __NV_E4M3);
            const __half2 rest = __hsub2(h, __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)hi[x], __NV_E4M3)));
            lo[x] = (uint32_t)__nv_cvt_halfraw2_to_fp8x2(__half2_raw(__hmul2(rest, __float2half2_rn(16.f))), __NV_SATFINITE, __NV_E4M3);
          }
          const uint32_t in = (uint32_t)(c & 1) * 8u;
          const uint32_t to = c < 64 ? swz(sb + (uint32_t)(c >> 4) * C::kQSlab, r, (c & 15) >> 1)
                                     : swz64(sb + C::kQRopeOff, r, (c - 64) >> 1);
          st_v2(to + in, hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
          // N rows further on the swizzle is the same
          st_v2(to + in + (c < 64 ? N * 128u : N * 64u), lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
        }
      }
      mbar_arrive(&B.q_full);
    };
    Seg after;
    bool more;
    auto advance = [&]() {  // to the next tile that sees something; the others get their zeros
      while ((more = walk.next(a, own, after)) && after.b0 >= after.b1) {
        for (int i = st; i < after.nrows * (kVal / 8); i += kSoftThreads)
          reinterpret_cast<uint4*>(a.out + (int64_t)after.grow * kVal)[i] = make_uint4(0u, 0u, 0u, 0u);
        if (a.lse && st < after.nrows) a.lse[after.grow + st] = -INFINITY;
      }
    };
    advance();
    if (more) convert(after, q_mul);
    while (ok && more) {
      s = after;
      const float* qm = q_mul + (tc & 1) * N;
      const int32_t* table = a.table + (int64_t)s.r * a.M;
      // the cache block of this thread's token of block b (-1: no position's), and its row's scale
      auto entry = [&](int b) -> int32_t {
        const int t = s.block(b) * kBlk + tok;
        return (int32_t)load_if(b < s.b1 && s.any_sees(a, t), table + entry_of(a, t), 0xffffffffu);
      };
      auto there = [&](int32_t blk) -> bool { return blk >= 0 && (int64_t)blk < a.n_blocks; };
      auto scale_of = [&](int b, int32_t blk) -> uint32_t {
        const int t = s.block(b) * kBlk + tok;
        return load_if(there(blk), a.pool + blk * block_bytes + (int64_t)a.B * kRow + 4 * (t - entry_of(a, t) * a.B), 0x3f800000u);
      };
      int32_t blk_next = entry(s.b0), blk_far = entry(s.b0 + 1);
      uint32_t bits_next;
      if (quad == 0 && lane < NC) {
        less_max[c0 + lane] = C::kBias - kNone;
        const int i = (s.row0 + min(c0 + lane, s.nrows - 1)) / a.H;  // the row's query token
        row_pos[c0 + lane] = s.pos0 + (kTree && a.depths ? node_depth(a, s, i) : i);
        if (kTree) row_node[c0 + lane] = i;
      }
      dead = dead || !wait(&B.q_full, (uint32_t)tc);  // the factors
      if (!meet(false, any)) { ok = false; break; }
      float l[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) l[c] = 0.f;
      bits_next = scale_of(s.b0, blk_next);
      for (int b = s.b0; b < s.b1; ++b, ++g) {
        // the scale 2^x, or NaN, which then is the score's; x and 2^-x are finite either way
        const bool here = there(blk_next);
        const uint32_t bits = bits_next;
        const bool fine = row_scale_valid(bits);
        const float scale = fine ? __uint_as_float(bits) : __int_as_float(0x7fffffff);
        const float x = fine ? (float)((int)(bits >> 23) - 127) : 0.f;
        const float unscale = fine ? __uint_as_float((254u << 23) - bits) : 1.f;
        asm volatile("" ::"f"(scale), "f"(x), "f"(unscale));  // before the loads, or their arrival is waited for too
        // loads run ahead: the next block's scale, the table's entry of the one behind it
        blk_next = blk_far;
        bits_next = scale_of(b + 1, blk_next);
        blk_far = entry(b + 2);
        const int t = s.block(b) * kBlk + tok;
        // the token is seen by every position of the tile, or by some
        const bool all = here && t <= s.pmin && (a.window == 0 || t > s.pmax - a.window || t < a.sinks);
        const bool plain = __all_sync(kFull, all);
        // bit c: row c0 + c sees the token.  Position p sees token t when p - t is in [0, span).
        uint32_t vis = kFull;
        if (kTree && !plain) {
          vis = here ? tree_sees<NC>(a, s, t, row_pos + c0, row_node + c0) : 0u;
        } else if (!plain) {
          const uint32_t span = !here ? 0u : (a.window == 0 || t < a.sinks) ? 0x7fffffffu : (uint32_t)a.window;
          vis = 0u;
#pragma unroll
          for (int c = 0; c < NC; c += 4) {
            const int4 p = *reinterpret_cast<const int4*>(row_pos + c0 + c);
            vis |= (uint32_t)((uint32_t)(p.x - t) < span) << c;
            vis |= (uint32_t)((uint32_t)(p.y - t) < span) << (c + 1);
            vis |= (uint32_t)((uint32_t)(p.z - t) < span) << (c + 2);
            vis |= (uint32_t)((uint32_t)(p.w - t) < span) << (c + 3);
          }
        }
        dead = dead || !wait(&B.s_full[g & 1], (uint32_t)(g >> 1));
        tc_after();
        const uint32_t sS = tmem + lane_addr + C::kColS + (uint32_t)(g & 1) * (2 * N) + (uint32_t)c0;
        float v[NC];
        bool odd = false;  // the row has a code that is not a number
        // v: the raw scores
        auto raw = [&]() {
          float lo[NC];
          tmem_ld<NC>(sS, v);
          tmem_ld<NC>(sS + N, lo);
          tmem_wait_ld();
          odd = !(fabsf(v[0]) < INFINITY);
#pragma unroll
          for (int c = 0; c < NC; c += 2) {
            const float2 y = __ffma2_rn(make_float2(lo[c], lo[c + 1]), make_float2(0.0625f, 0.0625f), make_float2(v[c], v[c + 1]));
            v[c] = y.x;
            v[c + 1] = y.y;
          }
        };
        raw();
        // log2 of the weights: v times the row's scale, in log2 units, plus x, less the running maximum (plus kBias); -inf
        // where hidden
#pragma unroll
        for (int c = 0; c < NC; c += 4) {
          const float4 y = *reinterpret_cast<const float4*>(qm + c0 + c), m = *reinterpret_cast<const float4*>(less_max + c0 + c);
          const float2 by = make_float2(scale, scale), more_x = make_float2(x, x);
          const float2 p = __ffma2_rn(make_float2(v[c], v[c + 1]), __fmul2_rn(make_float2(y.x, y.y), by),
                                      __fadd2_rn(make_float2(m.x, m.y), more_x));
          const float2 q = __ffma2_rn(make_float2(v[c + 2], v[c + 3]), __fmul2_rn(make_float2(y.z, y.w), by),
                                      __fadd2_rn(make_float2(m.z, m.w), more_x));
          v[c] = p.x;
          v[c + 1] = p.y;
          v[c + 2] = q.x;
          v[c + 3] = q.y;
        }
        if (!plain) {
#pragma unroll
          for (int c = 0; c < NC; ++c) v[c] = (vis >> c) & 1u ? v[c] : -INFINITY;
        }
        float top = v[0];
#pragma unroll
        for (int c = 1; c < NC; ++c) top = fmaxf(top, v[c]);
        if (!meet(b == s.b0 || top > C::kRescale + C::kBias, any)) { ok = false; break; }
        // O^T of the block before: its weights have been read, and O^T is at rest
        if (g >= 1) dead = dead || !wait(&B.o_step, (uint32_t)(g - 1));
        if (any) {
          tc_after();
          // the tokens' maximum of each row; then the running maximum, the sums and O^T move to it
          raw();
          int32_t mine = 0;
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            v[c] = (vis >> c) & 1u ? __fadd_rn(__fmul_rn(v[c], qm[c0 + c] * scale), x) : -INFINITY;
            const int32_t w = __reduce_max_sync(kFull, as_ordered(v[c]));
            if (lane == c) mine = w;
          }
          if (lane < NC) warp_red[warp * NC + lane] = __int_as_float(as_ordered(__int_as_float(mine)));
          named_sync(bar_half, 128);
          if (quad == 0 && lane < NC) {
            const float* wm = warp_red + 4 * hw * NC + lane;
            const float top = fmaxf(fmaxf(wm[0], wm[NC]), fmaxf(wm[2 * NC], wm[3 * NC])), old = less_max[c0 + lane];
            // (far from 0, kBias - top may round to 16 - top, and 2^16 is past the weights' range)
            float less = fminf(old, C::kBias - top);
            if (less + top > C::kBias + C::kRescale) less = -top;
            less_max[c0 + lane] = less;
            row_f[c0 + lane] = ex2(less - old);
          }
          named_sync(bar_half, 128);
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            l[c] *= row_f[c0 + c];
            v[c] = __fadd_rn(v[c], less_max[c0 + c]);  // (the largest's own is no less than 0 however large it is)
          }
          if (b > s.b0) {
#pragma unroll 1
            for (int i = 0; i < 4 * (int)C::kSums / N && !dead; ++i) {
#pragma unroll
              for (int c = 0; c < NC; c += 8) {
                float o[8];
                tmem_ld8(tmem + lane_addr + (uint32_t)(i * N + c0 + c), o);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 8; ++k) o[k] *= row_f[c0 + c + k];
                tmem_st8(tmem + lane_addr + (uint32_t)(i * N + c0 + c), o);
              }
            }
            tmem_wait_st();
          }
          named_sync(bar_half, 128);  // row_f is free
        }
        // weights
#pragma unroll
        for (int c = 0; c < NC; ++c) v[c] = ex2(v[c]);
        constexpr int kBy = C::kApart ? 16 : 1;
        uint4 last[(NC + 15) / 16];  // lo codes
        if constexpr (N == 16) {  // [row][128 tokens]
#pragma unroll
          for (int c = 0; c < NC; c += 2) {
            uint32_t hi, mid, lo;
            split_weights<kBy>(v[c], v[c + 1], hi, mid, lo);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t to = swz(sb + C::kPOff, c0 + c + k, tok >> 4) + (uint32_t)(tok & 15);
              st_u8(to, hi >> (16 * k + 8));
              st_u8(to + C::kPPart, mid >> (16 * k + 8));
              st_u8(to + 2 * C::kPPart, lo >> (8 * k));
            }
          }
        } else {  // [token][N rows]
#pragma unroll
          for (int c = 0; c < NC; c += 16) {
            uint32_t h[4], m[4], w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t hi[2], mid[2], lo[2];
#pragma unroll
              for (int x = 0; x < 2; ++x)
                split_weights<kBy>(v[c + 4 * k + 2 * x], v[c + 4 * k + 2 * x + 1], hi[x], mid[x], lo[x]);
              h[k] = __byte_perm(hi[0], hi[1], 0x7531);
              m[k] = __byte_perm(mid[0], mid[1], 0x7531);
              w[k] = __byte_perm(lo[0], lo[1], 0x5410);
            }
            const int chunk = (c0 + c) / 16;
            const uint32_t to = N == 64 ? swz64(sb + C::kPOff, tok, chunk) : swz32(sb + C::kPOff, tok, chunk);
            st_v4(to, make_uint4(h[0], h[1], h[2], h[3]));
            st_v4(to + C::kPPart, make_uint4(m[0], m[1], m[2], m[3]));
            last[c / 16] = make_uint4(w[0], w[1], w[2], w[3]);
          }
          if (C::kApart) st_v4(swz32(sb + C::kLastOff, tok, hw), last[0]);
        }
        if (!plain) {
          // A weight of 0 times a code that is NaN would be NaN: such codes of rows that a position of the tile does not
          // see (another position's, or what lies in an unread place) become 0.  The score of any one query tells, and a
          // position that sees the row is not misled: its score, and so its weight, is NaN.
          uint32_t edge = __ballot_sync(kFull, !all && odd);
          const int x4 = kPairs * g + hw;  // this half's pair: two slabs of 8 chunks
          if (edge && !phase_wait(&B.e_full[x4 % C::kRing], (uint32_t)(x4 / C::kRing) & 1u, a.wait_ns)) fail();  // (S^T has read it)
          const uint32_t pair = sb + C::kRingOff + (uint32_t)(x4 % C::kRing) * kPairF8;
          while (edge) {
            const int r = 32 * quad + __ffs(edge) - 1;
            edge &= edge - 1u;
            if (lane < 16) {
              const uint32_t at = swz_pair(pair, lane >> 3, r, lane & 7);
              const uint4 y = ld_v4(at);
              uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) w[k] &= ~__vcmpeq4(w[k] & 0x7f7f7f7fu, 0x7f7f7f7fu);
              st_v4(at, make_uint4(w[0], w[1], w[2], w[3]));
            }
          }
        }
        tc_before();
        mbar_arrive(&B.p_full);
        // the sums keep the weights, without the rows' scales, in fp32; behind the arrival, while the MMAs run
#pragma unroll
        for (int c = 0; c < NC; c += 2) {
          const float2 y = __ffma2_rn(make_float2(v[c], v[c + 1]), make_float2(unscale, unscale), make_float2(l[c], l[c + 1]));
          l[c] = y.x;
          l[c + 1] = y.y;
        }
        if constexpr (!C::kApart) {
          // over the rope keys: behind the next block's S^T if it is of this tile (the next tile's are not asked for before
          // this block's O^T)
          if (b + 1 < s.b1) dead = dead || !wait(&B.s_full[(g + 1) & 1], (uint32_t)((g + 1) >> 1));
#pragma unroll
          for (int c = 0; c < NC; c += 16) st_v4(swz64(sb + C::kLastOff, tok, (c0 + c) / 16), last[c / 16]);
          mbar_arrive(&B.l_full);
        }
        if (b == s.b0) advance();  // (while these warps have time)
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
        if (lane < NC) warp_red[warp * NC + lane] = l[0];
      }
      named_sync(bar_half, 128);
      if (quad == 0 && lane < NC) {
        const float* ws = warp_red + 4 * hw * NC + lane;
        const float sum = (ws[0] + ws[NC]) + (ws[2 * NC] + ws[3 * NC]);
        const int row = c0 + lane;
        row_f[row] = sum == 0.f ? 0.f : 1.f / sum;
        if (s.part >= 0) {
          float* ml = a.part_ml + ((int64_t)blockIdx.x * 2 + s.part) * 2 * N;
          ml[row] = C::kBias - less_max[row];
          ml[N + row] = sum;
        } else if (a.lse && row < s.nrows) {
          a.lse[s.grow + row] = sum == 0.f ? -INFINITY : (log2f(sum) - less_max[row]) * 0.6931471805599453f;
        }
      }
      if (more) convert(after, q_mul + ((tc + 1) & 1) * N);
      named_sync(bar_half, 128);
      dead = dead || !wait(&B.o_done, (uint32_t)tc);
      tc_after();
#pragma unroll 1
      for (int i = 0; i < 4 && !dead; ++i) {
        float o[NC];
        const uint32_t from = tmem + lane_addr + (uint32_t)i * C::kSums + (uint32_t)c0;
        tmem_ld<NC>(from, o);
        if constexpr (C::kApart) {
          float mid[NC], lo[NC];
          tmem_ld<NC>(from + N, mid);
          tmem_ld<NC>(from + 2 * N, lo);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < NC; ++c) o[c] += 0.0625f * (mid[c] + 0.0625f * lo[c]);
        } else {
          tmem_wait_ld();
        }
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
            const float x0 = o[c] * row_f[c0 + c], x1 = o[c + 1] * row_f[c0 + c + 1];
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

bool encode_f8(MapsF8& m, const PagedAttendArgs& a) {
  const EncodeTiled fn = encoder();
  if (!fn) return false;
  const cuuint64_t block = (cuuint64_t)a.B * kRowBytesF8;
  uint8_t* pool = const_cast<uint8_t*>(a.pool);
  const cuuint64_t dims[5] = {128, 8, kVal / 128, (cuuint64_t)(a.B / 8), (cuuint64_t)a.n_blocks};
  const cuuint64_t strides[4] = {kRow, 128, 8 * kRow, block};
  const cuuint32_t box[5] = {128, 8, 2, (cuuint32_t)(m.run / 8), 1}, step[5] = {1, 1, 1, 1, 1};
  if (fn(&m.codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, pool, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return false;
  const cuuint64_t rdims[3] = {kRow - kVal, (cuuint64_t)a.B, (cuuint64_t)a.n_blocks}, rstrides[2] = {kRow, block};
  const cuuint32_t rbox[3] = {kRow - kVal, (cuuint32_t)m.run, 1};
  return fn(&m.rope, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, pool + kVal, rdims, rstrides, rbox, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int N, bool kTree>
cudaError_t launch(const PagedAttendArgs& a, cudaStream_t s) {
  using C = ShapeF8<N>;
  cudaError_t e;
  static std::atomic<uint64_t> ready{0};  // devices where the kernel may have its shared memory
  const uint64_t bit = a.device < 64 ? 1ull << a.device : 0ull;
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(attend_paged_f8_kernel<N, kTree>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  MapsF8 maps{};
  maps.run = a.B & -a.B;
  if (maps.run > kBlk) maps.run = kBlk;
  if (!encode_f8(maps, a)) return cudaErrorInvalidValue;
  if (a.own_list) {
    attend_paged_f8_kernel<N, kTree><<<a.workers, C::kThreads, C::kSmem, s>>>(a, maps);
    e = cudaGetLastError();
  } else {
    e = launch_paged_schedule(a, N, s);
    if (e == cudaSuccess) e = launch_after(attend_paged_f8_kernel<N, kTree>, a.workers, C::kThreads, C::kSmem, s, a, maps);
  }
  if (e == cudaSuccess) e = launch_paged_join(a, N, C::kBias, s);
  return e;
}

}  // namespace

cudaError_t launch_paged_f8(const PagedAttendArgs& a, int N, cudaStream_t s) {
  if (a.masks) return N == 16 ? launch<16, true>(a, s) : N == 32 ? launch<32, true>(a, s) : launch<64, true>(a, s);
  return N == 16 ? launch<16, false>(a, s) : N == 32 ? launch<32, false>(a, s) : launch<64, false>(a, s);
}

}  // namespace kvo
