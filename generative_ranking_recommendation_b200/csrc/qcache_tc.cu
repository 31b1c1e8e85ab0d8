// Candidate attention over the quantised history cache for many candidates, on 5th-generation
// tensor cores (sm_100a).
//
// The semantics are those of qcache_attn.cu: s_cj = scale q_c.k_j + bias, k_j = s_j c_j.  With tens
// of candidates a row of the cache is used often enough that it pays to write its values out as
// tensor-core operands once per 128 candidates: what bounds the work in the end is one exponential
// per pair (16 a clock and SM: 512 clocks for 128 x 64 pairs, the products take half of that).
// Today it is instruction issue: a tile of 128 x 64 pairs takes 3770 warp instructions (8 bits: 3490),
// of which 0.65 (0.55) a clock and scheduler are issued by the 27 warps that fit an SM.  1024 users x
// 480 rows x 256 candidates x 8 heads of 4 bits: 690 us (5.3 ns a tile over the GPU; the exponentials
// alone 240 us); 64 x 480 x 1024 x 16 heads of 8 bits: 354 us.
//
// Design: two blocks an SM, each one stream of items (a user, a head, 128 candidates, a range of
// the history), 14 warps:
//   * warp 13 runs ahead: it finds the next item and its largest scales, publishes them as a record
//     that the other warps read, and issues the TMA loads: the item's Q rows, and 64 rows at a
//     time the head's K codes, V codes, scales and times (boxes of 64 rows out of the cache's
//     row-major bytes).
//   * warps 4-7 write operands tile by tile, K by two warps and V by two, a thread a row of 64
//     codes, as fp16.  A code times its scale is exact there: the item's largest scale is taken out
//     as a power of two.  The bias of a key enters S through the MMA, as three bf16 parts of its
//     column term in a fifth K = 16 slice; the candidates' side of that slice holds the power of
//     two that S lacks.
//   * warp 12 (an elected lane) issues tcgen05.mma: S (128 x 64) into one of two TMEM buffers, the
//     next S before the current P V, and O += P V (128 x 64) with P read from TMEM.
//   * warps 0-3 run the softmax, a thread a candidate: P = 2^(x - m) in one pass, in fp16 (11
//     bits: rounding P to bf16 would double the error of the bf16 output).  m is the maximum of
//     the item's first tile, the most recent rows, which a decaying bias favours; a later tile
//     whose sum leaves fp16's range is redone with its own maximum and O rescaled.
//   * warps 8-11 do an item's beginning and end while the softmax is at another: Q (a candidate
//     scaled by a power of two into fp16's range; its own score q.k_c on the way), and the output
//     rows, joined with the candidate's own key and value in fp32.
// TMEM: S 2 x 64, P 2 x 32, O 64 columns = 256 of the 512 that two blocks share.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include <climits>
#include <cmath>

#include "common.cuh"
#include "host_util.h"
#include "kernels.h"
#include "qcache.cuh"

namespace gr {
namespace qtc {

constexpr int BM = 128;  // candidates of an item
constexpr int BN = 64;   // cached rows of a tile
constexpr int kThreads = 448;
constexpr int kStages = 2;
constexpr uint32_t kQBytes = BM * 128;        // a Q tile: rows of 64 fp16, 128-byte swizzle
constexpr uint32_t kTileBytes = BN * 128;     // a K or V tile
constexpr uint32_t kKABytes = BN * 16;        // column terms: 8 bf16 a key
constexpr uint32_t kQABytes = BM * 16;        // their candidate side

constexpr uint32_t kOffQ = 0;                                  // 2 tiles
constexpr uint32_t kOffK = kOffQ + 2 * kQBytes;                // kStages
constexpr uint32_t kOffV = kOffK + kStages * kTileBytes;       // kStages
constexpr uint32_t kOffKA = kOffV + kStages * kTileBytes;      // kStages
constexpr uint32_t kOffZero = kOffKA + kStages * kKABytes;     // the second half of their slice
constexpr uint32_t kOffQA = kOffZero + kKABytes;               // 2, and a pad that the last rows' half reaches
constexpr uint32_t kOffOut = kOffQA + 2 * kQABytes + 128;      // own values, then output rows
constexpr uint32_t kOffRow = kOffOut + BM * 128;  // 2 x 4 x 128 floats, per candidate: S's scale and later the
                                                  // maximum, own score, time term, sum
constexpr uint32_t kOffRec = kOffRow + 2 * 4 * BM * 4;
constexpr int kRecs = 4;  // records of items
// A tile of the cache as copied: the head's K codes, its V codes, 16 bytes of scales (the head's
// pair and its neighbours') and the time and position of each of the 64 rows.
template <int FMT>
struct Raw {
  static constexpr int kCb = FMT == GENRANK_QCACHE_INT4 ? 32 : 64;
  static constexpr int kSlots = FMT == GENRANK_QCACHE_INT4 ? 3 : 2;
  static constexpr uint32_t kOffScale = 2 * BN * kCb, kOffTail = kOffScale + BN * 16, kBytes = kOffTail + BN * 16;
};
constexpr int kMaxSlots = 3;
enum Bar {
  kQRaw = 0, kQFull = 2, kQEmpty = 4, kSFull = 6, kPFull = 8, kPvDone = 10, kKFull = 12,
  kKEmpty = kKFull + kStages, kVFull = kKEmpty + kStages, kVEmpty = kVFull + kStages, kRawFull = kVEmpty + kStages, kRawEmpty = kRawFull + kMaxSlots,
  kRecFull = kRawEmpty + kMaxSlots, kRecEmpty = kRecFull + kRecs, kOFull = kRecEmpty + kRecs, kOEmpty, kDone,
  kNumBars
};
constexpr uint32_t kOffBar = kOffRec + kRecs * 64;
constexpr uint32_t kOffMisc = kOffBar + kNumBars * 8;  // tmem base, abort flag
constexpr uint32_t kOffRaw = (kOffMisc + 16 + 127) / 128 * 128;
template <int FMT>
constexpr uint32_t smem_bytes() { return kOffRaw + Raw<FMT>::kSlots * Raw<FMT>::kBytes + 1024; }  // + alignment slack
static_assert(smem_bytes<GENRANK_QCACHE_INT8>() <= 113 * 1024 && smem_bytes<GENRANK_QCACHE_INT4>() <= 113 * 1024,
              "two blocks an SM");
static_assert(kOffOut % 128 == 0 && kOffKA % 128 == 0 && kKABytes % 128 == 0 && kOffQA % 128 == 0 && kOffBar % 8 == 0 && kOffRec % 16 == 0,
              "operand alignment");

constexpr uint32_t kTmemCols = 256;
constexpr uint32_t kColS = 0, kColP = 128, kColO = 192;
// kind::f16 descriptors: fp16 (format 0) operands, bf16 for the column terms
constexpr uint32_t idesc_f16(int M, int N, int b_mn) { return idesc_bf16_f32(M, N, 0, b_mn) & ~((1u << 7) | (1u << 10)); }
constexpr uint32_t kIdescS = idesc_f16(BM, BN, 0);
constexpr uint32_t kIdescBias = idesc_bf16_f32(BM, BN, 0, 0);
constexpr uint32_t kIdescPV = idesc_f16(BM, kQDh, 1);

// Operands are codes times their scale over the item's largest, times 2^kUp: as high in fp16's range
// as the constants of the unpacking allow (72 f and 1152 f below 65504), so that a row whose scale is
// far below the largest keeps its bits down to 2^-25 (4 bits) or 2^-30 (8 bits) of it.
template <int FMT>
constexpr int kUp = FMT == GENRANK_QCACHE_INT4 ? 9 : 6;
// Scores leave the MMA as x / (f 2^up): f in [1/2, 1) and a whole exponent fe make scale log2 e =
// f 2^fe, and 2^up is the candidate's, with fe in it.  A key's column term is its bias over f, down to
// kLowestBias; of a key past the end it is kPastEnd, which no sum of scores reaches.  Both are exact in
// bf16, and with the candidate's 2^26 at most finite.
constexpr float kPastEnd = -0x1p100f, kLowestBias = -0x1p98f;
constexpr int kMinUp = -26;
constexpr float kPExp = 6.f;        // P holds 2^(x - max + 6)
constexpr float kMaxSum = 65504.f;  // a tile's sum up to this leaves no term beyond fp16
constexpr float kHighest = 1e38f;   // of a candidate's time term
constexpr float kFar = 0x1p27f;     // a maximum from which on neighbouring floats are 8 and more apart

struct Params {
  CUtensorMap tq;              // q: [C] rows of H heads x 64 bf16, box of a head and 128 rows
  CUtensorMap tcodes, tsmall;  // the cache's bytes: boxes of 64 rows and a head's codes, or 16 bytes
  QcachedAttnArgs c;
  int ctiles, splits, chunk;
  unsigned items;
  float f, f_inv;  // scale log2 e = f 2^fe
  int fe;
  float* part;  // [splits][C][H][kQPart], or null
};

// An item as published: everything that its warps need of it.
struct Item {
  int h, s, cb, mt;      // head, range, first candidate row, candidates (at most 128)
  int n, rows, tiles;    // the user's rows, the item's, and their tiles (-1: no more items)
  int at;                // the item's first cache row
  int ke, ve;            // powers of two, 2^kUp of which are above every K and V scale
  long long t_min;       // earliest time of the item's candidates, the origin of the bias
  int pad[4];
};
static_assert(sizeof(Item) == 64, "a record");

// Exponent e of the power of two above x >= 0 (2^e > x), within [-126, 126].
GR_DEVICE int exp_above(float x) { return min(max((int)(__float_as_uint(x) >> 23) - 126, -126), 126); }

// The block's next item with something to do, from index w on (w moves past it), by a full warp.
// Users whose layout is broken are flagged and left out.
template <int FMT>
GR_DEVICE Item next_item(const Params& P, const QRow& L, unsigned& w) {
  const QcachedAttnArgs& c = P.c;
  const int lane = threadIdx.x & 31;
  Item it{};
  it.tiles = -1;
  for (; w < P.items; w += gridDim.x) {
    unsigned i = w;
    it.h = i % (unsigned)c.a.H;
    i /= (unsigned)c.a.H;
    it.s = i % (unsigned)P.splits;
    i /= (unsigned)P.splits;
    const int ct = i % (unsigned)P.ctiles, u = i / (unsigned)P.ctiles;
    const int b = c.a.off[u], e = c.a.off[u + 1];
    const long long at = c.rows[u];
    it.n = c.len[u];
    const bool good = b >= 0 && e >= b && e <= c.a.T && it.n >= 0 && at >= 0 && it.n <= c.R && at <= c.R - it.n;
    if (lane == 0 && it.h == 0 && it.s == 0 && (!good || e - b > c.max_cand || it.n > c.max_len))
      flag(c.a.err, GENRANK_DERR_LAYOUT);
    it.cb = b + ct * BM;
    it.mt = min(min(e - b, c.max_cand) - ct * BM, BM);
    const int lo = it.s * P.chunk;
    it.rows = max(0, min(min(it.n, c.max_len), lo + P.chunk) - lo);
    it.at = (int)(at + lo);
    if (!good || it.mt <= 0 || (it.s > 0 && it.rows == 0)) continue;
    it.tiles = (it.rows + BN - 1) / BN;
    w += gridDim.x;
    // its largest scales and its candidates' earliest time
    const uint8_t* src = c.cache + (at + lo) * L.bytes + L.scales + 4 * it.h;
    float kmax = 0.f, vmax = 0.f;
    it.t_min = LLONG_MAX;
#pragma unroll
    for (int r = 0; r < BM; r += 32) it.t_min = min(it.t_min, (long long)c.a.ts[it.cb + min(r + lane, it.mt - 1)]);
#pragma unroll 1
    for (int r = lane; r < it.rows; r += 32 * 4) {
      uint32_t s[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        s[k] = r + 32 * k < it.rows ? __ldg(reinterpret_cast<const uint32_t*>(src + (long long)(r + 32 * k) * L.bytes)) : 0u;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float x = bf16_lo(s[k]), y = bf16_hi(s[k]);
        if (x < INFINITY) kmax = fmaxf(kmax, x);
        if (y < INFINITY) vmax = fmaxf(vmax, y);
      }
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      kmax = fmaxf(kmax, __shfl_xor_sync(0xffffffffu, kmax, o));
      vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, o));
      it.t_min = min(it.t_min, __shfl_xor_sync(0xffffffffu, it.t_min, o));
    }
    it.ke = max(exp_above(kmax) - kUp<FMT>, -126);
    it.ve = max(exp_above(vmax) - kUp<FMT>, -126);
    break;
  }
  return it;
}

GR_DEVICE uint32_t par(int use) { return (uint32_t)(use & 1); }
// Waits by a whole warp for the phase of the given parity, in few instructions (the code of 14
// warps' roles shares the instruction cache): up to 2 million tries that the hardware suspends for
// a microsecond each, after which, or once another role has given up, it gives up.
GR_DEVICE bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  const uint32_t addr = smem_u32(bar);
#pragma unroll 1
  for (int i = 1 << 21; i > 0; --i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, 1000;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(addr), "r"(parity)
        : "memory");
    if (__all_sync(0xffffffffu, ok)) return true;
    if (__any_sync(0xffffffffu, *abort_flag)) return false;
  }
  *abort_flag = 1;
  return false;
}
// MMAs and commits by one elected lane of a converged warp: descriptors and addresses that the
// compiler knows to be the same in every lane sit in uniform registers.
GR_DEVICE void mma_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
GR_DEVICE void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
GR_DEVICE void commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}
GR_DEVICE uint64_t desc_plain(uint32_t saddr, uint32_t lbo_bytes, uint32_t sbo_bytes) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((lbo_bytes >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((sbo_bytes >> 4) & 0x3FFFu) << 32) | ((uint64_t)1 << 46);
}
// 16 bytes global -> shared without registers, waited for by cp_async_wait
GR_DEVICE void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
GR_DEVICE void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
GR_DEVICE void tmem_st8_nowait(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
GR_DEVICE uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
GR_DEVICE uint32_t sub_f16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
GR_DEVICE uint32_t mul_f16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
GR_DEVICE uint32_t fma_f16(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// A slope in log2 units (the largest stay finite: none times no distance is none)
GR_DEVICE float slope_log2(float s) { return fminf(s * kLog2e, 3.4e38f); }
GR_DEVICE float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // e in [-126, 127]

// ------------------------------------------------------------------------------------------
// operands
// ------------------------------------------------------------------------------------------
// 16-byte chunk c (8 values) of a row in a 128-byte swizzled tile
GR_DEVICE uint4* chunk_at(uint8_t* tile, int row, int c) {
  return reinterpret_cast<uint4*>(tile + row * 128 + ((c ^ (row & 7)) << 4));
}

// Shared-memory address of that row's chunk 0; chunk c is at it ^ 16 c (tiles start at multiples of
// 128 bytes).
GR_DEVICE uint32_t row_addr(const uint8_t* tile, int row) { return smem_u32(tile) + row * 128 + ((row & 7) << 4); }
GR_DEVICE void store16(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// A row's 64 values, code times f, as fp16 in the tile.  4 bits: the eight values
// of a word go out as 0 4 1 5 2 6 3 7, the order in which masks take them out (Q has the same
// order, and O's columns are put back when they are written).
template <int FMT>
GR_DEVICE void store_codes(const uint8_t* from, float f, uint32_t to) {  // to: row_addr
  const uint32_t f2 = pack_f16(f, f);
  if constexpr (FMT == GENRANK_QCACHE_INT4) {
    // high nibbles: (1024 + 16 u) f / 16 - 72 f = (u - 8) f, every factor exact
    const uint32_t f16th = mul_f16(f2, 0x2C002C00u), m72 = mul_f16(f2, 0xD480D480u);
#pragma unroll
    for (int c = 0; c < 8; c += 4) {
      const uint4 x = *reinterpret_cast<const uint4*>(from + 4 * c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w = i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w, v = w >> 8;
        store16(to ^ (16 * (c + i)), mul_f16(sub_f16((w & 0x000F000Fu) | 0x64006400u, 0x64086408u), f2),
                fma_f16((w & 0x00F000F0u) | 0x64006400u, f16th, m72),
                mul_f16(sub_f16((v & 0x000F000Fu) | 0x64006400u, 0x64086408u), f2),
                fma_f16((v & 0x00F000F0u) | 0x64006400u, f16th, m72));
      }
    }
  } else {
    const uint32_t m1152 = mul_f16(f2, 0xE480E480u);  // exact: the scale is a power of two
#pragma unroll
    for (int c = 0; c < 8; c += 2) {
      const uint4 x = *reinterpret_cast<const uint4*>(from + 8 * c);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t w = i ? x.z : x.x, v = i ? x.w : x.y;
        store16(to ^ (16 * (c + i)), fma_f16(__byte_perm(w, 0x64646464u, 0x4140), f2, m1152),
                fma_f16(__byte_perm(w, 0x64646464u, 0x4342), f2, m1152),
                fma_f16(__byte_perm(v, 0x64646464u, 0x4140), f2, m1152),
                fma_f16(__byte_perm(v, 0x64646464u, 0x4342), f2, m1152));
      }
    }
  }
}

// A float as three bf16 parts (they sum to it to about 2^-25 of it).
GR_DEVICE uint4 bf16_parts(float q) {
  const __nv_bfloat16 hi = __float2bfloat16_rn(q);
  const float r1 = q - __bfloat162float(hi);
  const __nv_bfloat16 mid = __float2bfloat16_rn(r1);
  const __nv_bfloat16 lo = __float2bfloat16_rn(r1 - __bfloat162float(mid));
  return make_uint4((uint32_t)__bfloat16_as_ushort(hi) | ((uint32_t)__bfloat16_as_ushort(mid) << 16),
                    (uint32_t)__bfloat16_as_ushort(lo), 0u, 0u);
}

template <int FMT>
__global__ void __launch_bounds__(kThreads, 2) k_qcached_tc(const __grid_constant__ Params P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const QcachedAttnArgs& c = P.c;
  const AttnArgs& a = c.a;
  if (P.part) grid_release();  // the join may be set up
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
  float* rowdata = reinterpret_cast<float*>(smem + kOffRow);  // [2][4][128]
  const Item* recs = reinterpret_cast<const Item*>(smem + kOffRec);
  using R = Raw<FMT>;
  // (the shuffle tells the compiler that the warp's number is the same in every lane)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  // the second half of the column-term slice is zero on the keys' side; the candidates' side, any
  // finite numbers there, starts as zeros
  for (int i = threadIdx.x; i < (int)((kKABytes + 2 * kQABytes + 128) / 16); i += kThreads)
    reinterpret_cast<uint4*>(smem + kOffZero)[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  if (threadIdx.x == 0) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars[kQRaw + b], 1);
      mbar_init(&bars[kQFull + b], 4);       // warps 8-11
      mbar_init(&bars[kQEmpty + b], 1 + 4);  // the last S of the item, the softmax warps' reads
      mbar_init(&bars[kSFull + b], 1);
      mbar_init(&bars[kPFull + b], 4);
      mbar_init(&bars[kPvDone + b], 1);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars[kKFull + s], 2);
      mbar_init(&bars[kKEmpty + s], 1);
      mbar_init(&bars[kVFull + s], 2);
      mbar_init(&bars[kVEmpty + s], 1);
    }
    for (int s = 0; s < R::kSlots; ++s) {
      mbar_init(&bars[kRawFull + s], 1);
      mbar_init(&bars[kRawEmpty + s], 4);
    }
    for (int s = 0; s < kRecs; ++s) {
      mbar_init(&bars[kRecFull + s], 1);
      mbar_init(&bars[kRecEmpty + s], 4 + 4 + 4 + 1);  // every warp but the last
    }
    mbar_init(&bars[kOFull], 1 + 4);  // the item's last P V, the softmax warps' maxima and sums
    mbar_init(&bars[kOEmpty], 4);     // warps 8-11 have read O
    mbar_init(&bars[kDone], 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 12) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const float sl2 = a.scale * kLog2e;
  // The record of a role's qi-th item, once it is there (null: no more); given back when the role is
  // done with it.  Whole warps.
  auto take = [&](int qi) -> const Item* {
    const Item* it = recs + qi % kRecs;
    if (!wait_warp(&bars[kRecFull + qi % kRecs], par(qi / kRecs), abort_flag)) return nullptr;
    return it->tiles >= 0 ? it : nullptr;
  };
  auto give_back = [&](int qi) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[kRecEmpty + qi % kRecs]);
  };

  if (warp == 13) {
    // ---------------------------------------------------------------- items and loads
    const QRow L = qrow(a.H, FMT);
    unsigned w = blockIdx.x;
    int qi = 0, g = 0;  // items published, tiles loaded
    bool ok = true;
    Item cur{}, nx{};  // the item whose tiles are loaded (none at first) and the one after it
    int j = 0;
    for (;;) {
      if (j == min(cur.tiles, R::kSlots)) {
        // the next item's record, and the load of its Q rows, while this one's first tiles are
        // worked on
        nx = next_item<FMT>(P, L, w);
        const int rs = qi % kRecs, qb = qi & 1;
        ok = wait_warp(&bars[kRecEmpty + rs], par(qi / kRecs) ^ 1u, abort_flag) &&
             (nx.tiles < 0 || wait_warp(&bars[kQEmpty + qb], par(qi >> 1) ^ 1u, abort_flag));
        if (!ok) break;
        if (lane == 0) {
          reinterpret_cast<Item*>(smem + kOffRec)[rs] = nx;
          mbar_arrive(&bars[kRecFull + rs]);
          if (nx.tiles >= 0) {
            mbar_expect_tx(&bars[kQRaw + qb], kQBytes);
            tma_load_3d(smem + kOffQ + qb * kQBytes, &P.tq, &bars[kQRaw + qb], 0, nx.h, nx.cb);
          }
        }
        ++qi;
      }
      if (j == cur.tiles) {
        if (nx.tiles < 0) break;
        cur = nx;
        j = 0;
        if (cur.tiles == 0) continue;
      }
      // tile j of the item, from the most recent rows back
      const int sl = g % R::kSlots;
      ok = wait_warp(&bars[kRawEmpty + sl], par(g / R::kSlots) ^ 1u, abort_flag);
      if (!ok) break;
      if (lane == 0) {
        uint8_t* to = smem + kOffRaw + sl * R::kBytes;
        const int row = cur.at + (cur.tiles - 1 - j) * BN;
        mbar_expect_tx(&bars[kRawFull + sl], R::kBytes);
        tma_load_2d(to, &P.tcodes, &bars[kRawFull + sl], cur.h * L.cb, row);
        tma_load_2d(to + BN * R::kCb, &P.tcodes, &bars[kRawFull + sl], L.scales / 2 + cur.h * L.cb, row);
        tma_load_2d(to + R::kOffScale, &P.tsmall, &bars[kRawFull + sl], L.scales + (4 * cur.h & ~15), row);
        tma_load_2d(to + R::kOffTail, &P.tsmall, &bars[kRawFull + sl], L.tail, row);
      }
      ++g;
      ++j;
    }
    // on the way out, the copies issued last land before the block exits
    if (lane == 0) {
      for (int x = max(0, g - R::kSlots); x < g; ++x) mbar_drain(&bars[kRawFull + x % R::kSlots], par(x / R::kSlots));
      const int nq = ok ? qi - 1 : qi;  // the last record holds no item
      for (int x = max(0, nq - 2); x < nq; ++x) mbar_drain(&bars[kQRaw + (x & 1)], par(x >> 1));
    }
  } else if (warp >= 4 && warp < 8) {
    // ---------------------------------------------------------------- operands
    const int d = threadIdx.x - 128;
    const int side = d >> 6, key = d & 63;  // K or V row of a tile
    const uint32_t tile0 = row_addr(smem + (side == 0 ? kOffK : kOffV), key);
    int qi = 0, g = 0;
    bool ok = true;
    while (ok) {
      const Item* rec = take(qi);
      if (!rec) break;
      const Item& it = *rec;
      const float down = pow2(-(side == 0 ? it.ke : it.ve));
      const float sp2 = slope_log2(a.slope_pos[it.h]), st2 = slope_log2(a.slope_time[it.h]);
      const float f_inv = P.f_inv;
      bool bad_time = false, bad_pos = false;
      const int tiles = it.tiles, rows = it.rows, n1 = it.n + 1, h = it.h;
      const long long t_min = it.t_min;
#pragma unroll 1
      for (int j = 0; j < tiles; ++j, ++g) {
        const int st = g % kStages, sl = g % R::kSlots;
        if (!wait_warp(&bars[kRawFull + sl], par(g / R::kSlots), abort_flag)) {
          ok = false;
          break;
        }
        const uint8_t* from = smem + kOffRaw + sl * R::kBytes;
        const bool on = (tiles - 1 - j) * BN + key < rows;  // rows past the end are another user's
        const uint32_t scale = *reinterpret_cast<const uint32_t*>(from + R::kOffScale + key * 16 + (4 * h & 15));
        const float f = on ? (side == 0 ? bf16_lo(scale) : bf16_hi(scale)) * down : 0.f;
        uint4 term4 = make_uint4(0u, 0u, 0u, 0u);
        if (side == 0) {
          const int4 tail = *reinterpret_cast<const int4*>(from + R::kOffTail + key * 16);
          const long long tj = (long long)(((uint64_t)(uint32_t)tail.y << 32) | (uint32_t)tail.x);
          bad_time |= on && tj > t_min;
          bad_pos |= on && (tail.z < 0 || tail.z > n1);
          const float dp = (float)min(tail.z - n1, 0), dt = (float)min(tj - t_min, 0ll);
          term4 = bf16_parts(on ? fmaxf(fmaf(sp2, dp, st2 * dt) * f_inv, kLowestBias) : kPastEnd);
        }
        // (a K buffer is free after its S, long before the V buffer of the same tile)
        if (!wait_warp(&bars[(side == 0 ? kKEmpty : kVEmpty) + st], par(g / kStages) ^ 1u, abort_flag)) {
          ok = false;
          break;
        }
        if (side == 0) reinterpret_cast<uint4*>(smem + kOffKA + st * kKABytes)[key] = term4;
        store_codes<FMT>(from + (side * BN + key) * R::kCb, f, tile0 + st * kTileBytes);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars[(side == 0 ? kKFull : kVFull) + st]);
          mbar_arrive(&bars[kRawEmpty + sl]);
        }
      }
      if (bad_time && h == 0) flag(a.err, GENRANK_DERR_TS_ORDER);
      if (bad_pos && h == 0) flag(a.err, GENRANK_DERR_POS_RANGE);
      give_back(qi++);
    }
  } else if (warp == 12) {
    // ---------------------------------------------------------------- MMA issuer
    const uint64_t dQ = smem_desc_sw128(smem_u32(smem + kOffQ), 16, 1024);
    const uint64_t dK = smem_desc_sw128(smem_u32(smem + kOffK), 16, 1024);
    const uint64_t dV = smem_desc_sw128(smem_u32(smem + kOffV), kTileBytes, 1024);
    const uint64_t dQA = desc_plain(smem_u32(smem + kOffQA), 128, 128);
    static_assert(kStages == 2, "a tile and the one before it use both");
    const uint64_t dKA[2] = {desc_plain(smem_u32(smem + kOffKA), 2 * kKABytes, 128),
                             desc_plain(smem_u32(smem + kOffKA + kKABytes), kKABytes, 128)};
    int qi = 0, g = 0;
    bool ok = true;
    while (ok) {
      const Item* rec = take(qi);
      if (!rec) break;
      const int qb = qi & 1;
      const int tiles = __shfl_sync(0xffffffffu, rec->tiles, 0);
      give_back(qi);
      ok = wait_warp(&bars[kQFull + qb], par(qi >> 1), abort_flag);
      // S of tile j before P V of tile j - 1, so that the softmax finds it when it is done there
#pragma unroll 1
      for (int j = 0; j <= tiles && ok; ++j) {
        const int sb = g & 1, st = g % kStages;  // of tile j; the one before it has the others
        if (j < tiles) {
          // the S buffer is free once the softmax has handed over the P of tile g - 2
          ok = (g < 2 || wait_warp(&bars[kPFull + sb], par((g - 2) >> 1), abort_flag)) &&
               wait_warp(&bars[kKFull + st], par(g / kStages), abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint64_t q = dQ + qb * (kQBytes / 16), k = dK + st * (kTileBytes / 16);
#pragma unroll
          for (int i = 0; i < kQDh / 16; ++i) mma_ss(tmem + kColS + sb * BN, q + 2 * i, k + 2 * i, kIdescS, i > 0 ? 1u : 0u);
          mma_ss(tmem + kColS + sb * BN, dQA + qb * (kQABytes / 16), st ? dKA[1] : dKA[0], kIdescBias, 1u);
          commit(&bars[kSFull + sb]);
          commit(&bars[kKEmpty + st]);
          if (j == tiles - 1) commit(&bars[kQEmpty + qb]);
        }
        if (j > 0) {
          const int pb = sb ^ 1, pst = st ^ 1, gp = g - 1;
          // the first of an item overwrites O
          ok = (j > 1 || wait_warp(&bars[kOEmpty], par(qi) ^ 1u, abort_flag)) &&
               wait_warp(&bars[kVFull + pst], par(gp / kStages), abort_flag) &&
               wait_warp(&bars[kPFull + pb], par(gp >> 1), abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint64_t v = dV + pst * (kTileBytes / 16);
#pragma unroll
          for (int i = 0; i < BN / 16; ++i)
            mma_ts(tmem + kColO, tmem + kColP + pb * (BN / 2) + i * 8, v + 128 * i, kIdescPV, (j > 1 || i > 0) ? 1u : 0u);
          commit(&bars[kVEmpty + pst]);
          commit(&bars[kPvDone + pb]);
          if (j == tiles) commit(&bars[kOFull]);
        }
        if (j < tiles) ++g;
      }
      if (tiles == 0 && ok) {
        ok = wait_warp(&bars[kOEmpty], par(qi) ^ 1u, abort_flag);
        if (lane == 0) {
          mbar_arrive(&bars[kQEmpty + qb]);
          mbar_arrive(&bars[kOFull]);
        }
      }
      ++qi;
    }
    // every MMA issued has completed before TMEM is freed
    __syncwarp();
    commit(&bars[kDone]);
    mbar_drain(&bars[kDone], 0);
  } else if (warp < 4) {
    // ---------------------------------------------------------------- softmax
    const int r = threadIdx.x;  // candidate row of the item == TMEM lane
    const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
    int qi = 0, g = 0;
    bool ok = true;
    while (ok) {
      const Item* rec = take(qi);
      if (!rec) break;
      const int qb = qi & 1, tiles = rec->tiles;
      const int mt = __shfl_sync(0xffffffffu, rec->mt, 0);
      const bool idle = warp * 32 >= mt;  // none of the item's candidates
      give_back(qi);
      if (!wait_warp(&bars[kQFull + qb], par(qi >> 1), abort_flag)) break;
      float* rd = rowdata + qb * 4 * BM + r;
      const float f = r < mt ? rd[0] : 0.f;  // x = S f (a row past the candidates moves nothing)
      ++qi;
      float m = 0.f, l = 0.f;
      uint64_t f2 = f2_pack(f, f), nm2 = 0ull;  // x - m = S f2 + nm2
      for (int j = 0; j < tiles; ++j, ++g) {
        const int sb = g & 1;
        // S_g's completion covers every MMA issued before it, P_{g-2} V_{g-2} included, so its P
        // buffer is free as well
        if (!wait_warp(&bars[kSFull + sb], par(g >> 1), abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t s_addr = lane_base + kColS + sb * BN, p_addr = lane_base + kColP + sb * (BN / 2);
        if (idle) {  // (whatever P holds there reaches those rows of O alone)
          if (lane == 0) mbar_arrive(&bars[kPFull + sb]);
          continue;
        }
        bool move = j == 0;  // the offset is set from this tile's maximum
        for (int pass = 0;; ++pass) {
          if (__any_sync(0xffffffffu, move)) {
            // every lane takes part in the .sync.aligned accesses; only rows that move change m
            float mx = -INFINITY;
#pragma unroll 1
            for (int c0 = 0; c0 < BN; c0 += 16) {
              uint32_t s[16];
              tmem_ld16_async(s_addr + c0, s);
              tmem_ld_wait(s);
#pragma unroll
              for (int e = 0; e < 16; ++e) mx = fmaxf(mx, __uint_as_float(s[e]));
            }
            float top = __fmaf_ru(mx, f, -kPExp);  // up: no x - m is above kPExp
            float fe = f, off = top;
            if (fabsf(top) >= kFar) {
              // Rounding up would leave the maximum itself no weight.  S f with a power of two for f, and
              // the maximum's, are exact, so that it weighs 1; other scores of this size are whole steps
              // of a float below, in which up to half of f changes what is rounded off anyway.
              fe = __uint_as_float(__float_as_uint(f) & 0xFF800000u);
              off = mx * fe;
              top = mx * f;
            }
            const bool take_it = move && (j == 0 ? mx > -INFINITY : top > m);
            const float al = j == 0 ? 1.f : ex2(take_it ? m - top : 0.f);
            if (take_it) {
              m = top;
              f2 = f2_pack(fe, fe);
              nm2 = f2_pack(-off, -off);
            }
            if (j > 0) {
              l *= al;
              if (!wait_warp(&bars[kPvDone + (sb ^ 1)], par((g - 1) >> 1), abort_flag)) {
                ok = false;
                break;
              }
              tc_fence_after();
#pragma unroll 1
              for (int c0 = 0; c0 < kQDh; c0 += 16) {
                uint32_t o[16];
                tmem_ld16_async(lane_base + kColO + c0, o);
                tmem_ld_wait(o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
                tmem_st16(lane_base + kColO + c0, o);
              }
            }
          }
          // P = 2^(x - m), 16 keys at a time with the next ones' load in flight
          uint64_t sum2[2] = {0ull, 0ull};
          uint32_t xa[16], xb[16];
          auto part = [&](uint32_t (&s)[16], int c0) {
            uint32_t pk[8];
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              float v0, v1;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), f2, nm2), v0, v1);
              const float p0 = ex2(v0), p1 = ex2(v1);
              sum2[(e >> 1) & 1] = f2_add(sum2[(e >> 1) & 1], f2_pack(p0, p1));
              pk[e / 2] = pack_f16(p0, p1);
            }
            tmem_st8_nowait(p_addr + c0 / 2, pk);
          };
          tmem_ld16_async(s_addr, xa);
          tmem_ld_wait(xa);
#pragma unroll 1
          for (int c0 = 0; c0 < BN; c0 += 32) {
            tmem_ld16_async(s_addr + c0 + 16, xb);
            part(xa, c0);
            tmem_ld_wait(xb);
            if (c0 + 32 < BN) tmem_ld16_async(s_addr + c0 + 32, xa);
            part(xb, c0 + 16);
            tmem_ld_wait(xa);
          }
          tmem_wait_st();
          float s0, s1, s2, s3;
          f2_unpack(sum2[0], s0, s1);
          f2_unpack(sum2[1], s2, s3);
          const float rs = (s0 + s1) + (s2 + s3);
          move = j > 0 && pass == 0 && rs > kMaxSum;  // (once is enough: then every term is 2^kPExp at most)
          if (!__any_sync(0xffffffffu, move)) {
            l += rs;
            break;
          }
        }
        if (!ok) break;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kPFull + sb]);  // P is ready and S has been read
      }
      if (!ok) break;
      rd[0] = m;
      rd[3 * BM] = l;
      // the item before this one is complete: a warp that is early (an item without tiles, or of
      // one) does not count twice for it
      if (qi > 1 && !wait_warp(&bars[kOFull], par(qi - 2), abort_flag)) break;
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bars[kOFull]);
        mbar_arrive(&bars[kQEmpty + qb]);
      }
    }
  } else {
    // ---------------------------------------------------------------- Q and output, warps 8-11
    const int w4 = warp - 8, r = 32 * w4 + lane;  // candidate row of the output == TMEM lane
    const int sub = lane >> 3, ch = lane & 7;     // of loads and stores: 8 lanes a row, 16 bytes a lane
    const uint32_t lane_base = tmem + ((uint32_t)(w4 * 32) << 16);
    uint8_t* stage = smem + kOffOut + w4 * 32 * 128;
    int qi = 0;  // items whose record was taken
    const Item *nxp = nullptr, *itp = nullptr;
    auto write_q = [&]() -> bool {  // Q of the qi-th item
      const Item& nx = *nxp;
      const int qb = qi & 1;
      const float term =
          fminf(slope_log2(a.slope_time[nx.h]) * (float)(a.ts[nx.cb + min(r, nx.mt - 1)] - nx.t_min), kHighest);
      const __nv_bfloat16* k = (const __nv_bfloat16*)a.k + nx.h * kQDh + 8 * ch;
      auto load_k = [&](int i) {
        return __ldg(reinterpret_cast<const uint4*>(
            k + (nx.cb + (long long)min(32 * w4 + 4 * i + sub, nx.mt - 1)) * a.tok_stride));
      };
      uint4 k_next[2] = {load_k(0), load_k(1)};
      if (!wait_warp(&bars[kQRaw + qb], par(qi >> 1), abort_flag)) return false;
      const int rows4 = (nx.mt - 32 * w4 + 3) >> 2;  // rows of candidates, by fours
      float own_dot = 0.f;  // of the lane's own row, and its exponent
      int own_qe = 0;
#pragma unroll 1
      for (int i = 0; i < min(rows4, 8); ++i) {
        const uint4 k4 = k_next[0];
        k_next[0] = k_next[1];
        if (i + 2 < 8) k_next[1] = load_k(i + 2);
        const int at = 4 * i + sub, row = 32 * w4 + at;
        uint4* place = chunk_at(smem + kOffQ + qb * kQBytes, row, ch);
        const uint4 q4 = *place;
        const uint32_t qw[4] = {q4.x, q4.y, q4.z, q4.w}, kw[4] = {k4.x, k4.y, k4.z, k4.w};
        uint64_t f2[4], dot2 = 0ull;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f2[e] = f2_pack(bf16_lo(qw[e]), bf16_hi(qw[e]));
          dot2 = f2_fma(f2[e], f2_pack(bf16_lo(kw[e]), bf16_hi(kw[e])), dot2);
        }
        float dot, dot_hi;
        f2_unpack(dot2, dot, dot_hi);
        dot += dot_hi;
        // the row's largest magnitude, as bf16 bits (an infinity or a NaN makes the row NaN anyhow)
        const uint32_t mk = 0x7FFF7FFFu;
        uint32_t top = __vmaxu2(__vmaxu2(q4.x & mk, q4.y & mk), __vmaxu2(q4.z & mk, q4.w & mk));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
          top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
          dot += __shfl_xor_sync(0xffffffffu, dot, o);
        }
        // q = q' 2^qe, q' below 2 (and smaller where all scores are: its 2^-25 then stands for
        // 2^-43 of a score)
        int qe = min(max((int)(max(top & 0xFFFFu, top >> 16) >> 7) - 127, -126), 126);
        qe = max(qe, kMinUp - P.fe - nx.ke);
        const float qd = qe <= 126 ? pow2(-qe) : 0.f;
        float f[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) f2_unpack(f2_mul(f2[e], f2_pack(qd, qd)), f[2 * e], f[2 * e + 1]);
        *place = FMT == GENRANK_QCACHE_INT4
                     ? make_uint4(pack_f16(f[0], f[4]), pack_f16(f[1], f[5]), pack_f16(f[2], f[6]), pack_f16(f[3], f[7]))
                     : make_uint4(pack_f16(f[0], f[1]), pack_f16(f[2], f[3]), pack_f16(f[4], f[5]), pack_f16(f[6], f[7]));
        // the row's lane is 4 i + sub
        const float d = __shfl_sync(0xffffffffu, dot, 8 * (lane & 3));
        const int e = __shfl_sync(0xffffffffu, qe, 8 * (lane & 3));
        if (i == lane >> 2) {
          own_dot = d;
          own_qe = e;
        }
      }
      if (32 * w4 < nx.mt) {
        const int up = min(max(own_qe + nx.ke + P.fe, kMinUp), 126);  // (of rows past the candidates as well)
        const uint32_t one = __float_as_uint(pow2(-up)) >> 16;
        reinterpret_cast<uint4*>(smem + kOffQA + qb * kQABytes)[r] = make_uint4(one | (one << 16), one, 0u, 0u);
        float* rd = rowdata + qb * 4 * BM + r;
        rd[0] = P.f * pow2(up);
        rd[BM] = own_dot * sl2;
        rd[2 * BM] = term;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kQFull + qb]);
      ++qi;
      return true;
    };
    for (;;) {
      if (itp && itp->s == 0) {
        const Item& it = *itp;  // the values of the candidates to finish are on their way meanwhile
#pragma unroll 1
        for (int k = 0; k < 8; ++k)
          cp_async16(chunk_at(stage, 4 * k + sub, ch),
                     (const __nv_bfloat16*)a.v + (it.cb + (long long)min(32 * w4 + 4 * k + sub, it.mt - 1)) * a.tok_stride +
                         it.h * kQDh + 8 * ch);
      }
      // the next item's Q, then the output of the one before it
      nxp = take(qi);
      const bool more = nxp != nullptr;
      if (more && !write_q()) break;
      const int done = qi - 1 - (more ? 1 : 0), qb = done & 1;
      if (!itp) {
        if (!more) break;
        itp = nxp;
        continue;
      }
      const Item& it = *itp;
      cp_async_wait();
      __syncwarp();
      if (!wait_warp(&bars[kOFull], par(done), abort_flag)) break;
      tc_fence_after();
      const float* rd = rowdata + qb * 4 * BM + r;
      const float m = rd[0] - rd[2 * BM], own = rd[BM], l = rd[3 * BM];
      const bool row_ok = r < it.mt;
      const long long ci = it.cb + min(r, it.mt - 1);
      // the candidate itself joins where the item is the first range
      const float top = it.s > 0 ? m : it.tiles > 0 ? fmaxf(m, own) : own;
      const float wa = it.tiles > 0 ? (it.s > 0 ? 1.f : ex2(m - top)) : 0.f;
      const float ws = it.s > 0 ? 0.f : ex2(own - top);
      const float total = fmaf(l, wa, ws);
      const float inv = P.part ? 1.f : 1.f / total;
      const float wo = wa * pow2(it.ve) * inv, wb = ws * inv;
      const uint64_t wo2 = f2_pack(wo, wo), wb2 = f2_pack(wb, wb);
      float* part = P.part ? P.part + (((long long)it.s * a.T + ci) * a.H + it.h) * kQPart : nullptr;
#pragma unroll 1
      for (int c0 = 0; c0 < (32 * w4 < it.mt ? kQDh : 0); c0 += 16) {
        uint32_t o[16];
        tmem_ld16_async(lane_base + kColO + c0, o);
        tmem_ld_wait(o);
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          float x[8];
          uint4* place = chunk_at(stage, lane, c0 / 8 + z);
          const uint4 v4 = *place;
          const uint32_t v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const int lo = FMT == GENRANK_QCACHE_INT4 ? (e & 3) * 2 + (e >> 2) : e;  // columns of dimensions
            const int hi = FMT == GENRANK_QCACHE_INT4 ? lo + 2 : e + 1;              // e and e + 1
            uint64_t y = 0ull;
            if (it.tiles > 0) y = f2_mul(f2_pack(__uint_as_float(o[8 * z + lo]), __uint_as_float(o[8 * z + hi])), wo2);
            if (it.s == 0) y = f2_fma(f2_pack(bf16_lo(v[e / 2]), bf16_hi(v[e / 2])), wb2, y);
            f2_unpack(y, x[e], x[e + 1]);
          }
          if (part) {
            if (row_ok)
#pragma unroll
              for (int e = 0; e < 8; e += 2)
                *reinterpret_cast<float2*>(part + c0 + 8 * z + e) = make_float2(x[e], x[e + 1]);
          } else {
            *place = Elem<__nv_bfloat16>::pack(x);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kOEmpty]);  // O may be overwritten
      if (part && row_ok) *reinterpret_cast<float2*>(part + kQDh) = make_float2(top, total);
      __syncwarp();
      if (!part) {
        __nv_bfloat16* out = (__nv_bfloat16*)a.o + (long long)it.cb * a.o_stride + it.h * kQDh + 8 * ch;
#pragma unroll 2
        for (int k = 0; k < 8; ++k) {  // whole 128-byte rows
          const int row = 32 * w4 + 4 * k + sub;
          if (row < it.mt) *reinterpret_cast<uint4*>(out + (long long)row * a.o_stride) = *chunk_at(stage, 4 * k + sub, ch);
        }
        if (row_ok && a.lse) a.lse[(long long)it.h * a.T + ci] = (top + log2f(total)) * kLn2;
      }
      give_back(done);
      if (!more) break;
      itp = nxp;
    }
    cp_async_wait();
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && *abort_flag) flag(a.err, GENRANK_DERR_TIMEOUT);
  if (warp == 12) tmem_dealloc(tmem, kTmemCols);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  return fn;
}

// [C] rows of H heads x 64 bf16; box = one head x 128 rows, 128-byte swizzle
bool map_q(CUtensorMap* m, const AttnArgs& a) {
  cuuint64_t dims[3] = {(cuuint64_t)kQDh, (cuuint64_t)a.H, (cuuint64_t)a.T};
  cuuint64_t strides[2] = {(cuuint64_t)kQDh * 2, (cuuint64_t)a.tok_stride * 2};
  cuuint32_t box[3] = {(cuuint32_t)kQDh, 1, (cuuint32_t)BM}, es[3] = {1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.q), dims, strides, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// the cache as R rows of bytes; box = 64 rows x `bytes` (every box starts at a multiple of 16 bytes)
bool map_cache(CUtensorMap* m, const QcachedAttnArgs& c, int bytes) {
  cuuint64_t dims[2] = {(cuuint64_t)qrow(c.a.H, c.format).bytes, (cuuint64_t)c.R};
  cuuint64_t strides[1] = {dims[0]};
  cuuint32_t box[2] = {(cuuint32_t)bytes, (cuuint32_t)BN}, es[2] = {1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(c.cache), dims, strides, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int FMT>
int launch(const Params& P, cudaStream_t st) {
  static DeviceOnce once;
  if (!set_smem_limit_once(once, (const void*)k_qcached_tc<FMT>, (int)smem_bytes<FMT>())) return GENRANK_ERR_CUDA;
  const int sms = sm_count_current();
  if (sms <= 0) return GENRANK_ERR_CUDA;
  const unsigned blocks = P.items < 2u * sms ? P.items : 2u * sms;
  k_qcached_tc<FMT><<<blocks, kThreads, smem_bytes<FMT>(), st>>>(P);
  return cudaGetLastError() == cudaSuccess ? GENRANK_OK : GENRANK_ERR_LAUNCH;
}

}  // namespace qtc

int launch_qcached_tc(const QcachedAttnArgs& c, int ctiles, int splits, int chunk, float* part, cudaStream_t st) {
  qtc::Params P;
  if (!qtc::encode_fn() || !qtc::map_q(&P.tq, c.a)) return GENRANK_ERR_CUDA;
  if (c.R > 0) {
    if (c.R > INT32_MAX - qtc::BN) return GENRANK_ERR_UNSUPPORTED;  // rows are 32-bit TMA coordinates
    if (!qtc::map_cache(&P.tcodes, c, c.format == GENRANK_QCACHE_INT8 ? 64 : 32) || !qtc::map_cache(&P.tsmall, c, 16))
      return GENRANK_ERR_CUDA;
  } else {  // no history anywhere: no tile is ever loaded
    P.tcodes = P.tsmall = P.tq;
  }
  P.c = c;
  P.ctiles = ctiles;
  P.splits = splits;
  P.chunk = chunk;
  P.items = (unsigned)((long long)c.a.B * ctiles * splits * c.a.H);
  P.part = part;
  P.f = (float)frexp((double)c.a.scale * (double)kLog2e, &P.fe);
  P.f_inv = 1.f / P.f;
  return c.format == GENRANK_QCACHE_INT8 ? qtc::launch<GENRANK_QCACHE_INT8>(P, st)
                                         : qtc::launch<GENRANK_QCACHE_INT4>(P, st);
}

}  // namespace gr
