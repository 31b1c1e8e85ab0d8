// Candidate attention over the quantised history cache (sm_100a).  This is the form for few
// candidates a user, and the choice between it and the one of qcache_tc.cu (plan, below).
//
// Candidate c of user u (position n + 1, time t_c) sees the user's n cached rows and itself:
//   s_cj = scale q_c.k_j - m_h |n + 1 - p_j| - m_t,h |t_c - t_j|,   s_cc = scale q_c.k_c
// With k_j = s_j c_j (whole codes c_j, one scale a token and head) the score is
// (q_c.c_j) (s_j scale log2 e) + col_j, where col_j = log2 e (m_h (p_j - n - 1) +
// m_t,h (t_j - t_0)) is the key's part of the bias against t_0, the earliest time of the block's
// candidates, and the row's part, log2 e m_t,h (t_c - t_0) >= 0, is taken off the cached rows'
// maximum when the candidate itself joins them: only a candidate whose history has no weight then
// sees large numbers cancel.  Codes of at most 7 bits
// are exact in fp16, so q.c has exact products and fp32 sums: no key is ever rounded.
//
// One pass over the rows with the running maximum and sum of an online softmax:
//   * A block takes one user, up to 8 heads (a warp each), up to 8 candidates and a range of the
//     history.  A row of the cache holds every head's keys and values next to one another,
//     so a tile of rows is one contiguous piece: one more warp copies tiles into a ring of
//     shared-memory stages with bulk copies (wider models: a few per row), and turns each row's
//     time and position into two distances, once for all heads.
//   * A warp multiplies codes as the 16-row operand of m16n8k16 (keys for S^T = K q^T, head
//     dimensions for O^T = V^T P^T), candidates in the 8 columns, so that one candidate wastes
//     7/8 of a column tile and not 15/16 of a row tile; the work per row is the unpacking: two or
//     three instructions per code pair, no conversions.  The candidate's P^T operand is S^T's
//     accumulator transposed 8 x 8 (movmatrix); the key order inside a tile is permuted so that
//     the shared-memory reads of eight lanes fall into different banks for every row length.
//   * V's scale is folded into P (p_j s_j, fp16 with a power-of-two range shift): 11 bits where
//     rounding P or V to bf16 would cost as much again as rounding the output does.
//   * The maximum moves only when a score passes it by 2^8, and the first one is the
//     candidate's own score: most tiles take one vote and no shuffles.
//   * Short of blocks, the history is cut into ranges; the ranges' (max, sum, O) in fp32 are
//     joined by a second kernel, always in the same order.
// Bound: with one candidate the copies and the unpacking, at 256 users x 4096 rows of 8 heads 152 us
// for int4 rows (587 MB, 3.9 TB/s; the copies alone take 117), and the copies for int8, 203 us (1124
// MB, 5.5 TB/s); with more the unpacking, which every 8 candidates repeat (256 users x 480 rows x 32
// candidates: 90 us).
#include <cuda_fp16.h>

#include <cfloat>

#include "common.cuh"
#include "host_util.h"
#include "kernels.h"
#include "qcache.cuh"

namespace gr {
namespace qca {

constexpr int kHeads = 8;    // heads of a block, one warp each
constexpr int kCands = 8;    // candidates of a block
constexpr int kStages = 3;   // tiles in flight
constexpr int kMaxThreads = (kHeads + 1) * 32;  // the heads' warps and the one that copies
// P s enters the second product in fp16, s over the largest V scale so far: its 11 bits are whole down
// to P s = 2^-25 of that, its smallest numbers 2^-35.  (A slack of 8 and 2^7 lost bits from 2^-21 on;
// the more frequent moves cost ragged batches of up to 33 candidates 1 to 2 %, one candidate nothing.)
constexpr float kSlack = 4.f;  // a score may pass the running maximum by this (log2)
constexpr int kVExp = 11;      // P s <= 2^(kSlack + kVExp) = 2^15 < 65504
constexpr float kLowest = -1e30f;  // a maximum to start from when the own score is -inf
constexpr float kHighest = 1e38f;  // of a candidate's time term

struct Params {
  QcachedAttnArgs c;
  int groups;  // of 8 heads
  int ctiles;  // candidate tiles of a user
  int splits;  // ranges of the history
  int chunk;   // rows of a range, a multiple of 64
  int ways;    // half-warps that join a candidate's ranges
  unsigned first;  // blocks before this one take the longer half of the histories, the others the rest
  float* part;  // [splits][C][H][kQPart], or null: one range, written in place
};

struct Work {
  int u, g, s, ct;
  bool rest;  // a block of the second pass
};
GR_DEVICE Work work_of(const Params& P, unsigned i) {
  Work w;
  w.rest = i >= P.first;
  if (w.rest) i -= P.first;
  w.ct = i % P.ctiles;
  i /= P.ctiles;
  w.s = i % P.splits;
  i /= P.splits;
  w.g = i % P.groups;
  w.u = i / P.groups;
  return w;
}

// User u's candidates [c0, c0 + m) and cache rows [at, at + n); false when they do not fit the
// arrays (flagged by the caller).
GR_DEVICE bool user_of(const QcachedAttnArgs& c, int u, int& c0, int& m, long long& at, int& n) {
  const int b = c.a.off[u], e = c.a.off[u + 1];
  n = c.len[u];
  at = c.rows[u];
  c0 = b;
  m = e - b;
  return b >= 0 && e >= b && e <= c.a.T && n >= 0 && at >= 0 && n <= c.R && at <= c.R - n;
}

GR_DEVICE void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
GR_DEVICE uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
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
GR_DEVICE uint32_t fma_f16(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// Code pairs as fp16: a field u of a word placed under the exponent of 1024 reads as 1024 + u
// (16 u when it lies four bits higher), from which one exact subtraction (fused multiply-add)
// leaves the signed code.
GR_DEVICE uint32_t low_nibbles(uint32_t w) {  // nibbles 0 and 4
  return sub_f16((w & 0x000F000Fu) | 0x64006400u, 0x64086408u);  // - 1032
}
GR_DEVICE uint32_t high_nibbles(uint32_t w) {  // nibbles 1 and 5: (1024 + 16 u) / 16 - 72
  return fma_f16((w & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD480D480u);
}
// The same of byte pairs 1024 + 16 u1 + u0, mostly on the FMA pipe: with 1 <= u0 <= 15 (a code is
// never -8) the first rounding, to whole numbers, takes u0 off.  For keys, where the bytes come out
// with one instruction each, it relieves the integer pipe (159.7 -> 155.6 us at 256 users x 4096
// rows, one candidate); for values it does not pay.
GR_DEVICE void byte_nibbles(uint32_t b, uint32_t& lo, uint32_t& hi) {
  const uint32_t t = fma_f16(b, 0x2C002C00u, 0x63FF63FFu);  // b / 16 + 1023.5 = 1088 + u1
  hi = sub_f16(t, 0x64486448u);                             // - 1096
  lo = sub_f16(fma_f16(hi, 0xCC00CC00u, b), 0x64886488u);   // b - 16 hi = 1152 + u0, - 1160
}
GR_DEVICE uint32_t byte_pair(uint32_t w, uint32_t sel) {  // two bytes chosen by sel, - 1152
  return sub_f16(__byte_perm(w, 0x64646464u, sel), 0x64806480u);
}

// Key row of a 32-row tile that a lane's index r (0..7) stands for in 16-key half kk: even rows
// for the accumulator rows 0-7, the next odd one for 8-15.  Any four consecutive r, and the even
// and the odd r, fall into different bank groups, rows being an odd number of 16 bytes.
GR_DEVICE int key_row(int r) { return 2 * ((0x57463120u >> (4 * r)) & 7); }

// The 16 head dimensions whose q a lane (t = lane % 4) holds as the B operand, in the order of
// the codes it reads of a key: k-step ks, slot s (columns 2t.. or 2t+8..), element e.
template <int FMT>
GR_DEVICE constexpr int dim_of(int t, int ks, int s, int e) {
  return FMT == GENRANK_QCACHE_INT4 ? 16 * t + 8 * (ks >> 1) + 2 * (ks & 1) + s + 4 * e
                                    : 32 * (ks >> 1) + 8 * t + 4 * (ks & 1) + 2 * s + e;
}

// A key's 16 codes of this lane as the operand's eight registers, [k-step][slot].
template <int FMT>
GR_DEVICE void key_codes(const uint8_t* p, int t, uint32_t (&r)[4][2]) {
  if constexpr (FMT == GENRANK_QCACHE_INT4) {
    const uint2 w = *reinterpret_cast<const uint2*>(p + 8 * t);
    const uint32_t ww[2] = {w.x, w.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      byte_nibbles(__byte_perm(ww[i], 0x64646464u, 0x4240), r[2 * i][0], r[2 * i][1]);
      byte_nibbles(__byte_perm(ww[i], 0x64646464u, 0x4341), r[2 * i + 1][0], r[2 * i + 1][1]);
    }
  } else {
    const uint2 a = *reinterpret_cast<const uint2*>(p + 8 * t);
    const uint2 b = *reinterpret_cast<const uint2*>(p + 32 + 8 * t);
    const uint32_t ww[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r[i][0] = byte_pair(ww[i], 0x4140);
      r[i][1] = byte_pair(ww[i], 0x4342);
    }
  }
}

// Values 8g..8g+7 of two keys, paired key by key: r[i] = (key a's, key b's) code of 8g + i.
template <int FMT>
GR_DEVICE void value_codes(const uint8_t* pa, const uint8_t* pb, int g, uint32_t (&r)[8]) {
  if constexpr (FMT == GENRANK_QCACHE_INT4) {
    const uint32_t a = *reinterpret_cast<const uint32_t*>(pa + 4 * g);
    const uint32_t b = *reinterpret_cast<const uint32_t*>(pb + 4 * g);
    const uint32_t x = __byte_perm(a, b, 0x5410), y = __byte_perm(a, b, 0x7632);
    r[0] = low_nibbles(x);
    r[1] = high_nibbles(x);
    r[2] = low_nibbles(x >> 8);
    r[3] = high_nibbles(x >> 8);
    r[4] = low_nibbles(y);
    r[5] = high_nibbles(y);
    r[6] = low_nibbles(y >> 8);
    r[7] = high_nibbles(y >> 8);
  } else {
    const uint2 a = *reinterpret_cast<const uint2*>(pa + 8 * g);
    const uint2 b = *reinterpret_cast<const uint2*>(pb + 8 * g);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t aa = i ? a.y : a.x, bb = i ? b.y : b.x;
      const uint32_t lo = __byte_perm(aa, bb, 0x5140), hi = __byte_perm(aa, bb, 0x7362);
      r[4 * i] = byte_pair(lo, 0x4140);
      r[4 * i + 1] = byte_pair(lo, 0x4342);
      r[4 * i + 2] = byte_pair(hi, 0x4140);
      r[4 * i + 3] = byte_pair(hi, 0x4342);
    }
  }
}

GR_DEVICE float group_max(float x) {  // over the eight lanes of equal lane % 4
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
GR_DEVICE float group_sum(float x) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// A tile is 32 SUB rows, whose chains of loads, products and exponentials overlap.
template <int FMT, int SUB>
__global__ void __launch_bounds__(kMaxThreads, SUB == 1 ? 3 : 2) k_qcached(const __grid_constant__ Params P) {
  constexpr int kRows = 32 * SUB;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full[kStages], ready[kStages], empty[kStages];
  __shared__ float4 gaps[kStages][kRows];  // staged rows: position and time distance, 0 or -inf past the end
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  const QcachedAttnArgs& c = P.c;
  const AttnArgs& a = c.a;
  if (P.part) grid_release();  // the join may be set up
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Work w = work_of(P, blockIdx.x);
  int c0, m, n;
  long long at;
  if (!user_of(c, w.u, c0, m, at, n)) {
    if (threadIdx.x == 0) flag(a.err, GENRANK_DERR_LAYOUT);
    return;
  }
  if (threadIdx.x == 0 && (m > c.max_cand || n > c.max_len)) flag(a.err, GENRANK_DERR_LAYOUT);
  if (P.first < gridDim.x && (n <= c.max_len / 2) != w.rest) return;
  m = min(m, c.max_cand);
  const int cb = c0 + w.ct * kCands;               // the block's first candidate row
  const int mt = min(c0 + m - cb, kCands);         // and how many
  const int lo = w.s * P.chunk, hi = min(min(n, c.max_len), lo + P.chunk);
  if (mt <= 0 || (w.s > 0 && lo >= hi)) return;
  const int tiles = hi > lo ? (hi - lo + kRows - 1) / kRows : 0;
  const int heads = min(a.H - w.g * kHeads, kHeads);
  const QRow L = qrow(a.H, FMT);
  const QRow S = qrow(min(a.H, kHeads), FMT);  // a row as staged
  const int stage_bytes = kRows * S.bytes;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&ready[i], 1);
      mbar_init(&empty[i], heads);
    }
    abort_word = 0;
    mbar_fence_init();
  }
  __syncthreads();

  if (warp == (int)blockDim.x / 32 - 1) {
    // ------------------------------------------------------------------ copies and distances
    const uint8_t* src = c.cache + (at + lo) * (long long)L.bytes;
    const int scale_bytes = (4 * heads + 15) / 16 * 16;
    auto copy = [&](int i) {
      const int st = i % kStages;
      const int rows = min(kRows, hi - lo - i * kRows);
      uint8_t* dst = smem + st * stage_bytes;
      const uint8_t* from = src + (long long)i * kRows * L.bytes;
      if (a.H <= kHeads) {
        if (lane == 0) {
          mbar_expect_tx(&full[st], rows * L.bytes);
          bulk_load(dst, from, rows * L.bytes, &full[st]);
        }
      } else {
        if (lane == 0) mbar_expect_tx(&full[st], rows * (2 * heads * L.cb + scale_bytes + 16));
        __syncwarp();
        for (int r = lane; r < rows; r += 32) {
          uint8_t* to = dst + r * S.bytes;
          const uint8_t* row = from + (long long)r * L.bytes;
          bulk_load(to, row + w.g * kHeads * L.cb, heads * L.cb, &full[st]);
          bulk_load(to + S.scales / 2, row + L.scales / 2 + w.g * kHeads * L.cb, heads * L.cb, &full[st]);
          bulk_load(to + S.scales, row + L.scales + w.g * kHeads * 4, scale_bytes, &full[st]);
          bulk_load(to + S.tail, row + L.tail, 16, &full[st]);
        }
      }
    };
    int copied = 0;
    for (; copied < min(tiles, kStages); ++copied) copy(copied);
    long long t_min = a.ts[cb + min(lane, mt - 1)];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) t_min = min(t_min, __shfl_xor_sync(0xffffffffu, t_min, o));
    bool bad_time = false, bad_pos = false;
    for (int i = 0; i < tiles; ++i) {
      // tile i's distances, a row a lane, then the copy that takes the place of tile i - 1
      const int st = i % kStages;
      if (!__all_sync(0xffffffffu, mbar_wait(&full[st], (i / kStages) & 1, abort_flag, a.err))) break;
#pragma unroll
      for (int z = 0; z < SUB; ++z) {
        const int r = 32 * z + lane;
        uint8_t* row = smem + st * stage_bytes + r * S.bytes;
        const int4 tail = *reinterpret_cast<const int4*>(row + S.tail);
        const long long tj = (long long)(((uint64_t)(uint32_t)tail.y << 32) | (uint32_t)tail.x);
        const bool on = r < hi - lo - i * kRows;
        bad_time |= on && tj > t_min;
        bad_pos |= on && (tail.z < 0 || tail.z > n + 1);
        gaps[st][r] = on ? make_float4((float)min(tail.z - (n + 1), 0), (float)min(tj - t_min, 0ll), 0.f, 0.f)
                         : make_float4(0.f, 0.f, -INFINITY, 0.f);
        // rows past the end (of the block's last tile) hold what the stage held before: any codes
        // are finite, but a scale might not be
        if (!on)
          for (int h = 0; h < heads; ++h) *reinterpret_cast<uint32_t*>(row + S.scales + 4 * h) = 0u;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ready[st]);
      if (i > 0 && copied < tiles) {
        const int pr = (i - 1) % kStages;
        if (!__all_sync(0xffffffffu, mbar_wait(&empty[pr], ((i - 1) / kStages) & 1, abort_flag, a.err))) break;
        copy(copied++);
      }
    }
    if (bad_time) flag(a.err, GENRANK_DERR_TS_ORDER);
    if (bad_pos) flag(a.err, GENRANK_DERR_POS_RANGE);
    // the copies issued last have landed before the block exits
    if (lane == 0)
      for (int x = max(0, copied - kStages); x < copied; ++x) mbar_drain(&full[x % kStages], (x / kStages) & 1);
    return;
  }
  if (warp >= heads) return;

  // -------------------------------------------------------------------- one head
  const int h = w.g * kHeads + warp;
  const int g = lane >> 2, t = lane & 3;
  // (the largest slopes stay finite: none times no distance is none)
  const float sp2 = fminf(a.slope_pos[h] * kLog2e, 3.4e38f), st2 = fminf(a.slope_time[h] * kLog2e, 3.4e38f);
  const float sc2 = a.scale * kLog2e;

  // q as the B operand (candidate g), each scaled by its own power of two into fp16's range, and
  // each candidate's own score
  uint32_t q[4][2];
  float self[2];  // of candidates 2t, 2t + 1: the lane's accumulator columns
  uint64_t qs2;   // their scales, q's power of two included
  {
    const long long ci = cb + min(g, mt - 1);
    const __nv_bfloat16* qr = (const __nv_bfloat16*)a.q + ci * a.tok_stride + h * kQDh;
    const __nv_bfloat16* kr = (const __nv_bfloat16*)a.k + ci * a.tok_stride + h * kQDh;
    const int d0 = dim_of<FMT>(t, 0, 0, 0), d1 = dim_of<FMT>(t, 2, 0, 0);
    float qf[16], kf[16];
    Elem<__nv_bfloat16>::unpack(__ldg(reinterpret_cast<const uint4*>(qr + d0)), qf);
    Elem<__nv_bfloat16>::unpack(__ldg(reinterpret_cast<const uint4*>(qr + d1)), qf + 8);
    Elem<__nv_bfloat16>::unpack(__ldg(reinterpret_cast<const uint4*>(kr + d0)), kf);
    Elem<__nv_bfloat16>::unpack(__ldg(reinterpret_cast<const uint4*>(kr + d1)), kf + 8);
    float dot = 0.f, amax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      dot = fmaf(qf[i], kf[i], dot);
      const float x = fabsf(qf[i]);
      if (x < INFINITY) amax = fmaxf(amax, x);
    }
    dot += __shfl_xor_sync(0xffffffffu, dot, 1);
    dot += __shfl_xor_sync(0xffffffffu, dot, 2);
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const int ex = min(max((int)(__float_as_uint(amax) >> 23) - 127, -126), 126);
    const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
    const float qs = __uint_as_float((uint32_t)(127 + ex) << 23) * sc2;
    qs2 = f2_pack(__shfl_sync(0xffffffffu, qs, 8 * t), __shfl_sync(0xffffffffu, qs, 8 * t + 4));
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        // elements of the 16 loaded (two runs of 8 dimensions)
        const int i0 = 8 * (ks >> 1) + dim_of<FMT>(0, ks & 1, s, 0);
        const int i1 = 8 * (ks >> 1) + dim_of<FMT>(0, ks & 1, s, 1);
        q[ks][s] = pack_f16(qf[i0] * down, qf[i1] * down);
      }
#pragma unroll
    for (int e = 0; e < 2; ++e) self[e] = __shfl_sync(0xffffffffu, dot * sc2, 4 * (2 * t + e));
  }
  float row_term[2], mx[2];
  {
    const long long t0 = a.ts[cb + min(2 * t, mt - 1)], t1 = a.ts[cb + min(2 * t + 1, mt - 1)];
    long long t_min = min(t0, t1);
    t_min = min(t_min, __shfl_xor_sync(0xffffffffu, t_min, 1));
    t_min = min(t_min, __shfl_xor_sync(0xffffffffu, t_min, 2));
    row_term[0] = fminf(st2 * (float)(t0 - t_min), kHighest);
    row_term[1] = fminf(st2 * (float)(t1 - t_min), kHighest);
    // the maximum starts where the candidate's own score is
    for (int e = 0; e < 2; ++e) mx[e] = fmaxf(self[e] + row_term[e], kLowest);
  }
  uint64_t sum2 = 0ull;  // the lane's two candidates: (+0, +0)

  float o[4][4];  // dimension 8g + 2i (and + 1: elements 2, 3) of candidates 2t, 2t + 1
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
  float v_top = 0.f, v_down = 0.f;  // power of two >= every V scale so far; 2^kVExp over it
  const int kr0 = key_row(g);                              // this lane's key row (scores)
  const int va = key_row(2 * t) * S.bytes, vb = key_row(2 * t + 1) * S.bytes;  // its pair of value rows
  const int k_at = warp * S.cb + kr0 * S.bytes, sc_at = S.scales + 4 * warp;
  const int v_at = S.scales / 2 + warp * S.cb;
  int st = 0, ph = 0;

  for (int i = 0; i < tiles; ++i) {
    // the distances are there, and with them the rows that they were computed from
    if (!__all_sync(0xffffffffu, mbar_wait(&ready[st], ph, abort_flag, a.err))) return;
    const uint8_t* base = smem + st * stage_bytes;

    // each row's key scale, bias and value scale, a row a lane
    float key_scale[SUB], key_bias[SUB], value_scale[SUB];
    float v_max = 0.f;
#pragma unroll
    for (int z = 0; z < SUB; ++z) {
      const int row = 32 * z + lane;
      const uint32_t sc = *reinterpret_cast<const uint32_t*>(base + sc_at + row * S.bytes);
      const float4 gp = gaps[st][row];
      key_scale[z] = bf16_lo(sc);
      key_bias[z] = fmaf(sp2, gp.x, fmaf(st2, gp.y, gp.z));
      value_scale[z] = bf16_hi(sc);
      v_max = fmaxf(v_max, value_scale[z]);
    }

    // S^T = K q^T, its scale and bias
    float s[2 * SUB][4];
#pragma unroll
    for (int kk = 0; kk < 2 * SUB; ++kk) {
      const uint8_t* ra = base + k_at + 16 * kk * S.bytes;
      uint32_t ka[4][2], kb[4][2];
      key_codes<FMT>(ra, t, ka);
      key_codes<FMT>(ra + S.bytes, t, kb);
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        const uint32_t frag[4] = {ka[ks][0], kb[ks][0], ka[ks][1], kb[ks][1]};
        mma(acc, frag, q[ks][0], q[ks][1]);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int of = 16 * (kk & 1) + kr0 + e;
        const float ksc = __shfl_sync(0xffffffffu, key_scale[kk / 2], of);
        const float col = __shfl_sync(0xffffffffu, key_bias[kk / 2], of);
        f2_unpack(f2_fma(f2_pack(acc[2 * e], acc[2 * e + 1]), f2_mul(f2_pack(ksc, ksc), qs2), f2_pack(col, col)), s[kk][2 * e],
                  s[kk][2 * e + 1]);
      }
    }

    // the running maxima move (rarely: a score passed one by 2^kSlack, or a V scale is the
    // largest so far)
    bool move = v_max > v_top;
    float best[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = fmaxf(s[0][e], s[0][e + 2]);
#pragma unroll
      for (int kk = 1; kk < 2 * SUB; ++kk) x = fmaxf(x, fmaxf(s[kk][e], s[kk][e + 2]));
      best[e] = x;
      move |= x > mx[e] + kSlack;
    }
    if (__any_sync(0xffffffffu, move)) {
      float vm = v_max < INFINITY ? v_max : 0.f;
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, x));
      const int ex = max((int)(__float_as_uint(vm) >> 23) - 126, -100);  // 2^ex > vm
      const float top = fmaxf(v_top, __uint_as_float((uint32_t)(ex + 127) << 23));
      const float v_al = v_top > 0.f ? v_top / top : 1.f;
      v_top = top;
      v_down = (float)(1 << kVExp) / top;
      float al[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // (a candidate's maximum is its own affair: it does not move because a neighbour's does)
        const float top_e = group_max(best[e]);
        const float next = top_e > mx[e] + kSlack ? top_e : mx[e];
        al[e] = ex2(mx[e] - next);
        mx[e] = next;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          o[d][e] *= al[e] * v_al;
          o[d][e + 2] *= al[e] * v_al;
        }
      }
      sum2 = f2_mul(sum2, f2_pack(al[0], al[1]));
    }

    // P and O^T += V^T P^T
    float vd_row[SUB];
#pragma unroll
    for (int z = 0; z < SUB; ++z) vd_row[z] = value_scale[z] * v_down;
#pragma unroll
    for (int kk = 0; kk < 2 * SUB; ++kk) {
      uint32_t p[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float vd = __shfl_sync(0xffffffffu, vd_row[kk / 2], 16 * (kk & 1) + kr0 + e);
        float x, y;
        f2_unpack(f2_sub(f2_pack(s[kk][2 * e], s[kk][2 * e + 1]), f2_pack(mx[0], mx[1])), x, y);
        const uint64_t e2 = f2_pack(ex2(x), ex2(y));
        sum2 = f2_add(sum2, e2);
        f2_unpack(f2_mul(e2, f2_pack(vd, vd)), x, y);
        p[e] = transpose8x8(pack_f16(x, y));
      }
      const uint8_t* vp = base + v_at + 16 * kk * S.bytes;
      uint32_t fa[8], fb[8];  // even and odd rows: k columns 2t.. and 2t + 8..
      value_codes<FMT>(vp + va, vp + vb, g, fa);
      value_codes<FMT>(vp + va + S.bytes, vp + vb + S.bytes, g, fb);
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const uint32_t frag[4] = {fa[2 * d], fa[2 * d + 1], fb[2 * d], fb[2 * d + 1]};
        mma(o[d], frag, p[0], p[1]);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[st]);
    if (++st == kStages) {
      st = 0;
      ph ^= 1;
    }
  }

  // ---------------------------------------------------------------------- results
  const float up = v_top * (1.f / (1 << kVExp));
  float sum[2];
  f2_unpack(sum2, sum[0], sum[1]);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float l = group_sum(sum[e]);
    const int k = 2 * t + e;
    if (k >= mt) continue;
    const long long ci = cb + k;
    float x[8];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      x[2 * d] = o[d][e] * up;
      x[2 * d + 1] = o[d][e + 2] * up;
    }
    // rows without weight (l = 0) say nothing about where their maximum is
    float top = l == 0.f ? -FLT_MAX : mx[e] - row_term[e];
    if (w.s == 0) {  // the candidate itself
      const float next = fmaxf(top, self[e]), ph = ex2(top - next), ps = ex2(self[e] - next);
      top = next;
      l *= ph;
#pragma unroll
      for (int d = 0; d < 8; ++d) x[d] *= ph;
      float vf[8];
      Elem<__nv_bfloat16>::unpack(
          __ldg(reinterpret_cast<const uint4*>((const __nv_bfloat16*)a.v + ci * a.tok_stride + h * kQDh + 8 * g)), vf);
      l += ps;
#pragma unroll
      for (int d = 0; d < 8; ++d) x[d] = fmaf(ps, vf[d], x[d]);
    }
    if (P.part) {
      float* dst = P.part + (((long long)w.s * a.T + ci) * a.H + h) * kQPart;
#pragma unroll
      for (int d = 0; d < 8; d += 2) *reinterpret_cast<float2*>(dst + 8 * g + d) = make_float2(x[d], x[d + 1]);
      if (g == 0) *reinterpret_cast<float2*>(dst + kQDh) = make_float2(top, l);
    } else {
      const float inv = 1.f / l;
#pragma unroll
      for (int d = 0; d < 8; ++d) x[d] *= inv;
      *reinterpret_cast<uint4*>((__nv_bfloat16*)a.o + ci * a.o_stride + h * kQDh + 8 * g) = Elem<__nv_bfloat16>::pack(x);
      if (a.lse && g == 0) a.lse[(long long)h * a.T + ci] = (top + log2f(l)) * kLn2;
    }
  }
}

// Joins the ranges of a candidate and head: `ways` half-warps, four dimensions a lane, each take
// every ways-th range, then the first adds up what they found.  The order of the sums depends on the
// number of ranges alone.  What it takes is latency (4 users' 8 candidates of 8 heads in 74 ranges,
// 5 MB), so it is launched while the ranges are worked on and loads four of them at once.
constexpr int kHalfWarps = 16;
__global__ void __launch_bounds__(kHalfWarps * 16) k_qcached_join(const __grid_constant__ Params P) {
  __shared__ __align__(16) float parts[kHalfWarps][kQDh];
  __shared__ float2 stats[kHalfWarps];  // maximum and sum
  const AttnArgs& a = P.c.a;
  const int hw = threadIdx.x >> 4, lane = threadIdx.x & 15, d = 4 * lane;
  const int way = hw & (P.ways - 1);
  unsigned i = blockIdx.x * (unsigned)(kHalfWarps / P.ways) + hw / P.ways;
  const int h = i % (unsigned)a.H;
  i /= (unsigned)a.H;
  const int k = i % (unsigned)P.c.max_cand, u = i / (unsigned)P.c.max_cand;
  int c0 = 0, m = 0, n = 0;
  long long at;
  const bool on = u < a.B && user_of(P.c, u, c0, m, at, n) && k < m;
  const int splits = on ? min(P.splits, max(1, (min(n, P.c.max_len) + P.chunk - 1) / P.chunk)) : 0;
  const long long ci = c0 + k;
  grid_wait();  // the ranges are there

  const float* src = P.part + (ci * a.H + h) * kQPart;
  const long long step = a.T * a.H * kQPart;
  float top = -INFINITY, l = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s = way; s < splits; s += 4 * P.ways) {
    float2 ml[4], lo[4], hi[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float* p = src + (s + j * P.ways) * step;
      const bool there = s + j * P.ways < splits;
      ml[j] = there ? *reinterpret_cast<const float2*>(p + kQDh) : make_float2(-INFINITY, 0.f);
      lo[j] = there ? *reinterpret_cast<const float2*>(p + d) : make_float2(0.f, 0.f);
      hi[j] = there ? *reinterpret_cast<const float2*>(p + d + 2) : make_float2(0.f, 0.f);
    }
    const float next = fmaxf(top, fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)));
    const float al = ex2(top - next);
    top = next;
    l *= al;
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] *= al;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float f = ex2(ml[j].x - top);
      l = fmaf(ml[j].y, f, l);
      x[0] = fmaf(lo[j].x, f, x[0]);
      x[1] = fmaf(lo[j].y, f, x[1]);
      x[2] = fmaf(hi[j].x, f, x[2]);
      x[3] = fmaf(hi[j].y, f, x[3]);
    }
  }
  *reinterpret_cast<float4*>(&parts[hw][d]) = make_float4(x[0], x[1], x[2], x[3]);
  if (lane == 0) stats[hw] = make_float2(top, l);
  __syncthreads();
  if (way > 0 || !on) return;
  const int ways = min(P.ways, splits);
  for (int w = 1; w < ways; ++w) top = fmaxf(top, stats[hw + w].x);
  l = x[0] = x[1] = x[2] = x[3] = 0.f;
  for (int w = 0; w < ways; ++w) {
    const float f = ex2(stats[hw + w].x - top);
    const float4 v = *reinterpret_cast<const float4*>(&parts[hw + w][d]);
    l = fmaf(stats[hw + w].y, f, l);
    x[0] = fmaf(v.x, f, x[0]);
    x[1] = fmaf(v.y, f, x[1]);
    x[2] = fmaf(v.z, f, x[2]);
    x[3] = fmaf(v.w, f, x[3]);
  }
  const float inv = 1.f / l;
  *reinterpret_cast<uint2*>((__nv_bfloat16*)a.o + ci * a.o_stride + h * kQDh + d) =
      make_uint2(pack_bf16(x[0] * inv, x[1] * inv), pack_bf16(x[2] * inv, x[3] * inv));
  if (a.lse && lane == 0) a.lse[(long long)h * a.T + ci] = (top + log2f(l)) * kLn2;
}

struct Plan {
  bool tc;  // the tensor-core form: items of a head and 128 candidates in place of blocks
  int groups, ctiles, splits, chunk;
  long long units;  // blocks, or items, of one range
};
// From how many candidates a user at most the tensor-core form runs, and from how many rows for all
// blocks.  The bound on candidates is all that the host knows of them, and where they are fewer the
// blocks save the tiles of 8 that are not there, items of 128 nothing.  As many for each user (256
// users x 480 rows of 8 heads, 4 / 8 bits, us): blocks 78 / 82 for 24 candidates, 90 / 94 for 32, 111 /
// 113 for 33, 112 / 116 for 40, 131 / 135 for 41, 166 / 171 for 64; tensor cores 96 / 104, 99 / 105, 100
// / 106, 101 / 107, 101 / 107, 103 / 109.  Up to as many (300 users of up to 2000 rows, 5 heads, 8
// bits): blocks 113 for 33, 125 for 40, 138 for 48, 184 for 64; tensor cores 178, 190, 190, 207 (256
// users of up to 480 rows, 4 bits: 52 for 33, 58 for 40 against 74, 80).  The former ask for 33, the
// latter for more than 64: a sixth tile of 8 lies between, with which the former lose up to a sixth
// (1024 users x 33: 389 us against 333) and the latter up to two fifths (at 48).
// But an item is a long chain (31 us alone for 480 rows), and blocks are faster while they find free
// SMs: 128 candidates x 480 rows 16 against 25 us for 1 user (7680 rows), 31 against 37 for 16 users
// (123 thousand), 53 against 31 for 32.
constexpr int kTcFrom = 41;
constexpr long long kTcRows = 1 << 17;

// Blocks are one user's 8 heads and 8 candidates.  More candidates take more blocks, which read
// the rows from L2 again: tiles of 16 and 32 candidates share the unpacking, but
// their registers cost warps (32 candidates: 139 us in one tile, 90 us in four).
// The history is cut into ranges where that fills the 148 SMs better.  In units of a row's time in
// one of the blocks that share an SM: a block takes its rows and about 100 to start, one that has
// its SM to itself an eighth longer, and the join costs about 100.  (8 heads, 8 candidates, 8 bits, the
// count taken first: 4 users x 65536 rows 70 us in 74 ranges, 71 in 37, 103 in 18, 76 in 148; 64 users
// x 4096: 70 us in 4, 113 uncut, 74 in 2, 82 in 16; 128 users x 480: 29 us uncut, 33 in 2.)
Plan plan(int B, int H, int max_cand, int max_len) {
  Plan p;
  p.groups = (H + kHeads - 1) / kHeads;
  const long long blocks = (long long)B * p.groups * ((max_cand + kCands - 1ll) / kCands);
  p.tc = max_cand >= kTcFrom && max_len > 0 && (blocks >= kTcRows || blocks * max_len >= kTcRows);
  const int tile = p.tc ? 128 : kCands, least = p.tc ? 256 : 64, slots = p.tc ? 296 : 148;
  p.ctiles = max_cand > tile ? (int)((max_cand + tile - 1ll) / tile) : 1;
  p.units = (long long)B * (p.tc ? H : p.groups) * p.ctiles;
  auto rows = [&](long long s) { return (max_len + s * 64 - 1) / (s * 64) * 64; };
  auto cost = [&](long long s) {
    const long long rounds = (p.units * s + slots - 1) / slots, time = rounds * (rows(s) + 100);
    return time + (!p.tc && rounds == 1 ? time / 8 : 0) + (s > 1 ? 100 : 0);
  };
  long long best = 1;
  for (int k = 1; k <= 16; ++k) {  // whole rounds of the SMs
    long long s = (long long)slots * k / p.units;
    const long long most = ((long long)max_len + least - 1) / least;
    if (s > most) s = most;
    if (s > 1 && cost(s) < cost(best)) best = s;
  }
  p.chunk = (int)rows(best);
  p.splits = p.chunk > 0 ? (int)(((long long)max_len + p.chunk - 1) / p.chunk) : 1;
  return p;
}

// Tiles of 64 rows of 4 bits (150 us against 165 us with 32, at 256 users x 4096 rows) or 32 of 8
// bits: about 100 KB of stages for each of two blocks an SM.  Short histories take no more stages
// than they fill, and tiles of 32 rows, whose registers allow a third block (1000 users of 10 rows,
// 41 candidates: 143 -> 96 us).
template <int FMT, int SUB>
int launch(const Params& P, unsigned blocks, cudaStream_t st) {
  static DeviceOnce once;
  constexpr int tile = 32 * SUB;
  const int heads = P.c.a.H < kHeads ? P.c.a.H : kHeads;
  const int stages = P.chunk >= kStages * tile ? kStages : (P.chunk + tile - 1) / tile;
  if (!set_smem_limit_once(once, (const void*)k_qcached<FMT, SUB>, kStages * tile * qrow(kHeads, FMT).bytes))
    return GENRANK_ERR_CUDA;
  k_qcached<FMT, SUB><<<blocks, (heads + 1) * 32, stages * tile * qrow(heads, FMT).bytes, st>>>(P);
  return cudaGetLastError() == cudaSuccess ? GENRANK_OK : GENRANK_ERR_LAUNCH;
}

}  // namespace qca

size_t attn_fwd_qcached_workspace(int B, long long C, int H, int max_cand, int max_len) {
  const qca::Plan p = qca::plan(B, H, max_cand, max_len);
  return p.splits > 1 ? (size_t)p.splits * C * H * kQPart * sizeof(float) : 0;
}

int launch_attn_fwd_qcached(const QcachedAttnArgs& c, cudaStream_t st) {
  using namespace qca;
  const Plan p = plan(c.a.B, c.a.H, c.max_cand, c.max_len);
  int ways = 2;
  while (ways < kHalfWarps && 2 * ways < p.splits) ways *= 2;
  const int pairs = kHalfWarps / ways;  // (candidate, head) of a block
  const long long joins = p.splits > 1 ? ((long long)c.a.B * c.max_cand * c.a.H + pairs - 1) / pairs : 0;
  if (p.units * p.splits > INT32_MAX / 2 || joins * pairs > INT32_MAX) return GENRANK_ERR_UNSUPPORTED;
  Params P;
  P.c = c;
  P.groups = p.groups;
  P.ctiles = p.ctiles;
  P.splits = p.splits;
  P.chunk = p.chunk;
  P.ways = ways;
  P.part = p.splits > 1 ? (float*)c.a.ws : nullptr;
  // More blocks than the SMs hold at once (3 of an SM), each a whole history: those longer than half
  // the bound go first, so that no long one begins last.  What this saves is part of a longest
  // history's time at the end, about 10 ns a row of the bound; what it costs are the blocks that have
  // nothing to do in a pass, 3 ns each, whatever the bound: hence blocks against rows.  Once and twice
  // (us): 1500 blocks of up to 2000 rows 126, 112; 1000 of 2000 202, 191; 3000 of 4000 266, 246; 500 of
  // 2000 115, 115.  Where the rule says once: 1000 of 480 73, 73; 2000 of 480 112, 116; 2000 of 1000 195,
  // 193; 3000 of 2000 181, 174.  Histories of one length take the same time either way.
  P.first = (unsigned)(p.units * p.splits);
  const bool twice = !p.tc && p.splits == 1 && p.units > 444 && p.units < c.max_len;
  const unsigned blocks = twice ? 2 * P.first : P.first;
  const int rc = p.tc ? launch_qcached_tc(c, p.ctiles, p.splits, p.chunk, P.part, st)
                 : c.format == GENRANK_QCACHE_INT8 ? launch<GENRANK_QCACHE_INT8, 1>(P, blocks, st)
                 : c.max_len <= kStages * 32 ? launch<GENRANK_QCACHE_INT4, 1>(P, blocks, st)
                                   : launch<GENRANK_QCACHE_INT4, 2>(P, blocks, st);
  if (rc != GENRANK_OK || joins == 0) return rc;
  // launched as soon as every block of the ranges has begun, it waits for them (grid_wait)
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)joins);
  cfg.blockDim = dim3(kHalfWarps * 16);
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_qcached_join, P) == cudaSuccess ? GENRANK_OK : GENRANK_ERR_LAUNCH;
}

}  // namespace gr
