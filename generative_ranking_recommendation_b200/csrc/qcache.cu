// Quantised history cache (sm_100a): writing key/value rows to it and reading them back.
//
// One head's 64 values x (bf16; fp32 is rounded to it) become whole codes c and one scale s,
// a = max |x|:
//   int8: s = the smallest power of two with a <= 127 s
//   int4: s = a / 7 to five significant bits, halves up
//   c = sign(x) floor(|x| / s + 1/2)
// A code of 7 (3) magnitude bits times a scale of 1 (5) significant bits has at most 8, so
// every value c s is a bf16 number: what is read back, what a tensor-core operand would hold
// and what a score computed from codes stands for are the same number, with no rounding
// between them.  Power-of-two and five-bit scales cost at most a bit and 3 % of the range.
//
// Both kernels move bytes and are bound by HBM.  A warp takes a run of consecutive rows; 8
// lanes hold one head (16 bytes of bf16 a lane), so the maximum is three shuffles.
#include "common.cuh"
#include "host_util.h"
#include "kernels.h"
#include "qcache.cuh"

namespace gr {
namespace {

constexpr int kWarps = 8;            // warps of a block
constexpr int kMaxStageBytes = 64 << 10;  // staged rows of a block

// The user that token row t belongs to, for ascending rows: a search for the first, then a walk.
struct Cursor {
  int u;
  long long begin, end;  // rows [begin, end) of user u
};

GR_DEVICE void seek(Cursor& c, const int32_t* __restrict__ off, int B, long long t) {
  c.u = warp_find_user(off, B, t);
  c.begin = off[c.u];
  c.end = off[c.u + 1];
}

// Whether user u's rows are usable, and where they start in the cache: offsets inside the
// token array, no more rows than the user's segment, the cache range inside the cache and (for
// a write) before the next user's, so that no two users write one row.
GR_DEVICE bool user_rows(const QcacheArgs& a, int u, long long begin, long long end, bool write,
                         int& n, long long& at) {
  if (begin < 0 || end < begin || end > a.T) return false;
  const long long seg = end - begin;
  n = a.len ? a.len[u] : (int)seg;
  at = a.rows[u];
  if (n < 0 || n > seg || at < 0 || at > a.R - n) return false;
  return !write || u + 1 >= a.B || at + n <= a.rows[u + 1];
}

// Codes of eight values as bytes 0..7 of two words: y = x inv + magic + bias lands the code,
// rounded to nearest, in the low bits of y's pattern.  inv is 2^-14 (relative) above 1/s, so
// that halves (|x| / s = k + 1/2, exact for these operands) round away from zero; every other
// quotient is more than 1e-3 from a half (x has 8 significant bits, s at most 5), far beyond
// that factor and the rounding of 1/s.
GR_DEVICE uint2 code_bytes(const float* x, float inv, float magic) {
  uint32_t z[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = __float_as_uint(fmaf(x[i], inv, magic));
  const uint32_t a = __byte_perm(z[0], z[1], 0x0040), b = __byte_perm(z[2], z[3], 0x0040);
  const uint32_t c = __byte_perm(z[4], z[5], 0x0040), d = __byte_perm(z[6], z[7], 0x0040);
  return make_uint2(__byte_perm(a, b, 0x5410), __byte_perm(c, d, 0x5410));
}

constexpr float kMagic = 12582912.f;  // 1.5 * 2^23
constexpr float kHalfUp = 1.f + 1.f / 16384.f;

// Scale s (its bf16 bits) and the factor inv of one head from its largest magnitude (bf16
// bits; 0x7F80 and above: an infinity or a NaN among the values, whose head reads back as NaN).
template <int FMT>
GR_DEVICE uint32_t head_scale(uint32_t amax, float& inv) {
  if (amax >= 0x7F80u) {
    inv = 0.f;
    return 0x7FC0u;
  }
  const uint32_t bits = amax << 16;
  if constexpr (FMT == GENRANK_QCACHE_INT8) {
    // a = m 2^E, m in [1/2, 1): s = 2^(E-7), one more when m > 127/128 (the added bits carry)
    int e = (int)((bits + 0x1FFFFu) >> 23) - 133;
    e = min(max(e, -126), 121);
    inv = __uint_as_float((uint32_t)(127 - e) << 23) * kHalfUp;
    return (uint32_t)(e + 127) << 7;
  } else {
    const float t = __fdiv_rn(__uint_as_float(bits), 7.f);
    const uint32_t r = (__float_as_uint(t) + 0x40000u) & ~0x7FFFFu;
    const float s = fminf(fmaxf(__uint_as_float(r), 0x1p-126f), 0x1.2p125f);
    inv = __fdiv_rn(1.f, s) * kHalfUp;
    return __float_as_uint(s) >> 16;
  }
}

template <typename Tin>
GR_DEVICE uint4 load_bf16x8(const Tin* p) {
  if constexpr (sizeof(Tin) == 2) {
    return __ldg(reinterpret_cast<const uint4*>(p));
  } else {
    const float4 x = __ldg(reinterpret_cast<const float4*>(p));
    const float4 y = __ldg(reinterpret_cast<const float4*>(p) + 1);
    return make_uint4(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w), pack_bf16(y.x, y.y),
                      pack_bf16(y.z, y.w));
  }
}

// Quantises eight values a lane (one head: 8 consecutive lanes) into the staged row.
template <int FMT>
GR_DEVICE void put_head(uint8_t* row, const QRow& L, int H, int vec, const uint4& w, bool on) {
  const uint32_t m = 0x7FFF7FFFu;
  uint32_t mx = __vmaxu2(__vmaxu2(w.x & m, w.y & m), __vmaxu2(w.z & m, w.w & m));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const uint32_t amax = max(mx & 0xffffu, mx >> 16);
  float inv;
  const uint32_t s = head_scale<FMT>(amax, inv);
  if (!on) return;
  float x[8];
  Elem<__nv_bfloat16>::unpack(w, x);
  constexpr float kBias = FMT == GENRANK_QCACHE_INT8 ? 128.f : 8.f;
  if (s == 0x7FC0u || s == 0x7C00u) {  // not finite: codes 0; the largest int8 scale: |c| <= 127
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = s == 0x7FC0u ? 0.f : fminf(fmaxf(x[i], -3.3762e38f), 3.3762e38f);  // 127 * 2^121
  }
  const uint2 c = code_bytes(x, inv, kMagic + kBias);
  const int head2 = vec >> 3;  // heads of K, then of V
  if constexpr (FMT == GENRANK_QCACHE_INT8) {
    *reinterpret_cast<uint2*>(row + vec * 8) = c;
  } else {
    const uint32_t a = c.x | (c.x >> 4), b = c.y | (c.y >> 4);
    *reinterpret_cast<uint32_t*>(row + vec * 4) = __byte_perm(a, b, 0x6420);
  }
  if ((vec & 7) == 0) {
    const int side = head2 >= H;
    *reinterpret_cast<uint16_t*>(row + L.scales + (head2 - side * H) * 4 + side * 2) = (uint16_t)s;
  }
}

// k, v rows -> cache rows.  Each row is built in shared memory and leaves as whole 16-byte
// vectors (pads included, so that a row's bytes are defined).
template <typename Tin, int FMT>
__global__ void __launch_bounds__(kWarps * 32) k_qcache_append(const __grid_constant__ QcacheArgs a,
                                                               int warps, long long run) {
  extern __shared__ __align__(16) uint8_t stage_all[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp >= warps) return;
  const QRow L = qrow(a.H, FMT);
  uint8_t* row = stage_all + (size_t)warp * L.bytes;
  const int nv = 8 * a.H;  // 16-byte (bf16) vectors of one side
  const long long t0 = ((long long)blockIdx.x * warps + warp) * run;
  const long long t1 = min(t0 + run, a.T);
  if (blockIdx.x == 0 && warp == 0) {  // every user's layout is checked once
    for (int u = lane; u < a.B; u += 32) {
      int n;
      long long at;
      if (!user_rows(a, u, a.off[u], a.off[u + 1], true, n, at)) flag(a.err, GENRANK_DERR_LAYOUT);
    }
    __syncwarp();
  }
  if (t0 >= t1) return;
  for (int i = lane; i < (L.bytes - L.scales) / 4; i += 32)
    *reinterpret_cast<uint32_t*>(row + L.scales + 4 * i) = 0u;
  __syncwarp();
  Cursor c{0, 0, 0};
  bool ok = false;
  int n = 0;
  long long at = 0;
  for (long long t = t0; t < t1; ++t) {
    if (t == t0 || t >= c.end) {
      seek(c, a.off, a.B, t);
      ok = t >= c.begin && t < c.end && user_rows(a, c.u, c.begin, c.end, true, n, at);
      if (c.u == a.B - 1 && t >= c.end) break;  // rows behind the last user
    }
    if (!ok || t - c.begin >= n) continue;
    const Tin* kr = reinterpret_cast<const Tin*>(a.k) + t * a.tok_stride;
    const Tin* vr = reinterpret_cast<const Tin*>(a.v) + t * a.tok_stride;
    for (int i0 = 0; i0 < 2 * nv; i0 += 128) {
      uint4 w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = i0 + 32 * j + lane;
        w[j] = make_uint4(0u, 0u, 0u, 0u);
        if (i < 2 * nv) w[j] = load_bf16x8<Tin>((i < nv ? kr + 8 * i : vr + 8 * (i - nv)));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = i0 + 32 * j + lane;
        if (i0 + 32 * j < 2 * nv) put_head<FMT>(row, L, a.H, i, w[j], i < 2 * nv);
      }
    }
    if (lane == 0) {
      *reinterpret_cast<int64_t*>(row + L.tail) = a.ts[t];
      *reinterpret_cast<int32_t*>(row + L.tail + 8) = a.pos[t];
    }
    __syncwarp();
    uint4* dst = reinterpret_cast<uint4*>(a.cache + (at + (t - c.begin)) * L.bytes);
    for (int i = lane; i < L.bytes / 16; i += 32) dst[i] = reinterpret_cast<const uint4*>(row)[i];
    __syncwarp();
  }
}

// cache rows -> k, v rows (every value exact in bf16 and fp32)
template <typename Tout, int FMT>
__global__ void __launch_bounds__(kWarps * 32) k_qcache_read(const __grid_constant__ QcacheArgs a,
                                                             int warps, long long run) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const QRow L = qrow(a.H, FMT);
  const int nv = 8 * a.H;
  const long long t0 = ((long long)blockIdx.x * warps + warp) * run;
  const long long t1 = min(t0 + run, a.T);
  if (blockIdx.x == 0 && warp == 0) {
    for (int u = lane; u < a.B; u += 32) {
      int n;
      long long at;
      if (!user_rows(a, u, a.off[u], a.off[u + 1], false, n, at)) flag(a.err, GENRANK_DERR_LAYOUT);
    }
    __syncwarp();
  }
  Cursor c{0, 0, 0};
  bool ok = false;
  int n = 0;
  long long at = 0;
  for (long long t = t0; t < t1; ++t) {
    if (t == t0 || t >= c.end) {
      seek(c, a.off, a.B, t);
      ok = t >= c.begin && t < c.end && user_rows(a, c.u, c.begin, c.end, false, n, at);
      if (c.u == a.B - 1 && t >= c.end) break;  // rows behind the last user
    }
    if (!ok || t - c.begin >= n) continue;
    const uint8_t* row = a.cache + (at + (t - c.begin)) * L.bytes;
    Tout* kr = reinterpret_cast<Tout*>(a.k_out) + t * a.tok_stride;
    Tout* vr = reinterpret_cast<Tout*>(a.v_out) + t * a.tok_stride;
#pragma unroll 4
    for (int i = lane; i < 2 * nv; i += 32) {
      const int side = i >= nv, head = (i - side * nv) >> 3;
      const float s = __uint_as_float(
          (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(row + L.scales + head * 4 + side * 2)) << 16);
      uint2 w;
      if constexpr (FMT == GENRANK_QCACHE_INT8) {
        w = __ldg(reinterpret_cast<const uint2*>(row + i * 8));
      } else {
        const uint32_t p = __ldg(reinterpret_cast<const uint32_t*>(row + i * 4));
        const uint32_t lo = p & 0x0F0F0F0Fu, hi = (p >> 4) & 0x0F0F0F0Fu;  // even, odd values
        w = make_uint2(__byte_perm(lo, hi, 0x5140), __byte_perm(lo, hi, 0x7362));
      }
      constexpr float kBias = FMT == GENRANK_QCACHE_INT8 ? 128.f : 8.f;
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t word = e < 4 ? w.x : w.y;
        // a byte under the exponent of 2^23 reads as 2^23 + byte
        const float y = __uint_as_float(__byte_perm(word, 0x4B000000u, 0x7440u | (e & 3)));
        f[e] = (y - (8388608.f + kBias)) * s;
      }
      Tout* dst = side ? vr + 8 * (i - nv) : kr + 8 * i;
      if constexpr (sizeof(Tout) == 2) {
        *reinterpret_cast<uint4*>(dst) = Elem<__nv_bfloat16>::pack(f);
      } else {
        reinterpret_cast<float4*>(dst)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4*>(dst)[1] = make_float4(f[4], f[5], f[6], f[7]);
      }
    }
    if (lane == 0) {
      const int4 tail = __ldg(reinterpret_cast<const int4*>(row + L.tail));
      if (a.ts_out) a.ts_out[t] = (int64_t)(((uint64_t)(uint32_t)tail.y << 32) | (uint32_t)tail.x);
      if (a.pos_out) a.pos_out[t] = tail.z;
    }
  }
}

template <typename T, int FMT>
int launch(const QcacheArgs& a, bool write, cudaStream_t st) {
  static DeviceOnce smem_attr;
  const int sms = sm_count_current();
  if (sms <= 0) return GENRANK_ERR_CUDA;
  const QRow L = qrow(a.H, FMT);
  int warps = kWarps;
  if (write) {
    while (warps > 1 && warps * L.bytes > kMaxStageBytes) warps /= 2;
    if (!set_smem_limit_once(smem_attr, (const void*)k_qcache_append<T, FMT>, kMaxStageBytes))
      return GENRANK_ERR_CUDA;
  }
  // a run of consecutive rows per warp once every SM has its 64 warps
  const long long most = (long long)sms * 64;
  const long long run = (a.T + most - 1) / most;
  const long long blocks = (a.T + run * warps - 1) / (run * warps);
  if (write)
    k_qcache_append<T, FMT><<<(unsigned)blocks, warps * 32, warps * L.bytes, st>>>(a, warps, run);
  else
    k_qcache_read<T, FMT><<<(unsigned)blocks, warps * 32, 0, st>>>(a, warps, run);
  return cudaGetLastError() == cudaSuccess ? GENRANK_OK : GENRANK_ERR_LAUNCH;
}

int dispatch(const QcacheArgs& a, bool write, cudaStream_t st) {
  if (a.dtype == GENRANK_BF16)
    return a.format == GENRANK_QCACHE_INT8
               ? launch<__nv_bfloat16, GENRANK_QCACHE_INT8>(a, write, st)
               : launch<__nv_bfloat16, GENRANK_QCACHE_INT4>(a, write, st);
  return a.format == GENRANK_QCACHE_INT8 ? launch<float, GENRANK_QCACHE_INT8>(a, write, st)
                                         : launch<float, GENRANK_QCACHE_INT4>(a, write, st);
}

}  // namespace

int launch_qcache_append(const QcacheArgs& a, cudaStream_t st) { return dispatch(a, true, st); }
int launch_qcache_read(const QcacheArgs& a, cudaStream_t st) { return dispatch(a, false, st); }

}  // namespace gr
