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
// lanes hold one head (16 bytes of bf16 a lane), so the maximum is three shuffles.  1024 users x
// 480 rows of 8 heads, bf16: append 244 us (5.3 TB/s) to 4 bits and 258 (6.0) to 8, read 254 (5.1) and
// 284 (5.4); with 256 rows of nobody behind each history, where whole warps have no row to copy,
// append 284 and 283, read 303 and 328.  256 users of up to 2048 rows read to fp32 230 us (5.6 TB/s).
// More than 8 heads take the pieces one after the other, with two blocks an SM: 512 x 480 rows of 16
// heads 273 us (4.7 TB/s) to 4 bits and 299 (5.1) to 8.  Of the forms for up to 8 heads, held to 64
// registers, three spill: bf16 to 4 bits 16 bytes, fp32 to 4 bits 52, fp32 to 8 bits 132.
#include "common.cuh"
#include "host_util.h"
#include "kernels.h"
#include "qcache.cuh"

namespace gr {
namespace {

constexpr int kWarps = 8;            // warps of a block
constexpr int kMaxStageBytes = 64 << 10;  // staged rows of a block

// Whether user u's rows are usable, and where they start in the cache: offsets inside the
// token array, no more rows than the user's segment, the cache range inside the cache and (for
// a write) before the next user's.
template <bool kWrite>
GR_DEVICE bool user_rows(const QcacheArgs& a, int u, int begin, int end, int& n, long long& at) {
  if (begin < 0 || end < begin || end > a.T) return false;
  n = a.len ? a.len[u] : end - begin;
  at = a.rows[u];
  if (n < 0 || n > end - begin || at < 0 || at > a.R - n) return false;
  return !kWrite || u + 1 >= a.B || at + n <= a.rows[u + 1];
}

// A user's first cache row and its rows, as one lane of a writing warp holds them for the user that
// user u is compared with there.  Where first rows do not ascend (flagged: some user does not end
// before the next), users that are each before the next may still share rows.  So that no two users
// write one row, a user is written only when it is in order with its ancestors in the in-order
// numbered binary tree of all users (k = u + 1: k's lowest bits up to a higher bit replaced by that
// bit).  Of two users one is the other's ancestor, or they have one that lies between them, with
// which both are in order.  An ancestor a lane, and no load waits for another: a
// write and read-back of one token of 2048 users takes 28 us with it and without.
struct Ancestor {
  int side = 0;  // -1: before the user, 1: behind it, 0: none
  long long at = 0, n = 0;
};
GR_DEVICE Ancestor ancestor(const QcacheArgs& a, int u) {
  const unsigned k = u + 1u, lane = threadIdx.x & 31;
  const unsigned c = ((k >> lane) | 1u) << lane;
  Ancestor r;
  if (c != k && (k & ((1u << lane) - 1u)) && c <= (unsigned)a.B) {
    const int v = (int)(c - 1u);
    r.side = v < u ? -1 : 1;
    r.at = a.rows[v];
    r.n = a.len ? a.len[v] : (long long)a.off[v + 1] - a.off[v];
  }
  return r;
}
// (at and at + n lie inside the cache)
GR_DEVICE bool in_order(const Ancestor& r, long long at, int n) {
  const bool ok = r.side == 0 || (r.side > 0 ? at + n <= r.at
                                             : r.at <= at && (r.n <= 0 || (uint64_t)r.n <= (uint64_t)at - (uint64_t)r.at));
  return __all_sync(0xffffffffu, ok);
}

// A warp's walk over the token rows [t, t1) that have a cache row: a search for the first row's
// user, then user by user.
template <bool kWrite>
struct Walk {
  int u = -1;
  int first = 0, last = 0, end = 0;  // the user's rows [first, last) are copied, [first, end) are its
  long long at = 0;                  // cache row of token row 0 (first's less first)

  // The first such row at or after t, or one at or behind t1.  Rows before the first user's segment
  // are nobody's; where offsets do not ascend (flagged), a row is the first user's found to hold it.
  GR_DEVICE int next(const QcacheArgs& a, int t, int t1) {
    while (t < t1) {
      if (u < 0 || t >= end) {
        u = u < 0 ? warp_find_user(a.off, a.B, t) : u + 1;
        if (u >= a.B) return t1;  // rows behind the last user
        first = a.off[u];
        end = a.off[u + 1];
        int n = 0;
        Ancestor other;
        if constexpr (kWrite) other = ancestor(a, u);
        bool good = user_rows<kWrite>(a, u, first, end, n, at);
        if constexpr (kWrite) good = good && in_order(other, at, n);
        last = good ? first + n : first;
        at -= first;
      }
      t = max(t, first);
      if (t < last) return t;
      t = max(t, end);
    }
    return t1;
  }
  GR_DEVICE long long row(int t) const { return at + t; }
};

// Every user's layout is checked by one lane of the grid.
template <bool kWrite>
GR_DEVICE void check_users(const QcacheArgs& a, int warps) {
  const int stride = gridDim.x * warps * 32;
  for (int u = blockIdx.x * warps * 32 + threadIdx.x; u < a.B; u += stride) {
    int n;
    long long at;
    if (!user_rows<kWrite>(a, u, a.off[u], a.off[u + 1], n, at)) flag(a.err, GENRANK_DERR_LAYOUT);
  }
}

constexpr float kMagic = 12582912.f;  // 1.5 * 2^23
constexpr float kHalfUp = 1.f + 1.f / 16384.f;

// Codes of eight values (a vector of bf16) as bytes: x inv + magic + bias lands the code, rounded
// to nearest, in the low bits of the sum's pattern.  inv is 2^-14 (relative) above 1/s, so that
// halves (|x| / s = k + 1/2, exact for these operands) round away from zero; every other quotient
// is more than 1e-3 from a half (x has 8 significant bits, s at most 5), far beyond that factor
// and the rounding of 1/s.
GR_DEVICE uint2 code_bytes(const uint4& w, float inv, float magic) {
  const uint64_t i2 = f2_pack(inv, inv), m2 = f2_pack(magic, magic);
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    f2_unpack(f2_fma(f2_pack(bf16_lo(v[i]), bf16_hi(v[i])), i2, m2), lo, hi);
    b[i] = __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x0040);
  }
  return make_uint2(__byte_perm(b[0], b[1], 0x5410), __byte_perm(b[2], b[3], 0x5410));
}

// Scale s and the factor inv of one head from its largest magnitude (bf16 bits, finite).
template <int FMT>
GR_DEVICE float head_scale(uint32_t amax, float& inv) {
  const uint32_t bits = amax << 16;
  if constexpr (FMT == GENRANK_QCACHE_INT8) {
    // a = m 2^E, m in [1/2, 1): s = 2^(E-7), one more when m > 127/128 (the added bits carry)
    const int e = min(max((int)((bits + 0x1FFFFu) >> 23) - 133, -126), 121);
    inv = __uint_as_float((uint32_t)(127 - e) << 23) * kHalfUp;
    return __uint_as_float((uint32_t)(e + 127) << 23);
  } else {
    // a product in place of the division: a / 7 is halfway between two scales only where it is a
    // whole number, which the product reaches (1/7 rounds up), and nowhere near otherwise
    const float t = __uint_as_float(bits) * (1.f / 7.f);
    const float s = fminf(fmaxf(__uint_as_float((__float_as_uint(t) + 0x40000u) & ~0x7FFFFu), 0x1p-126f), 0x1.2p125f);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    inv *= kHalfUp;
    return s;
  }
}

GR_DEVICE uint32_t max_magnitude(const uint4& w) {  // of 8 bf16, as bits; beyond 0x7F80 for a NaN
  const uint32_t m = 0x7FFF7FFFu;
  const uint32_t x = __vmaxu2(__vmaxu2(w.x & m, w.y & m), __vmaxu2(w.z & m, w.w & m));
  return max(x & 0xFFFFu, x >> 16);
}

constexpr uint32_t kTop = 0x7F7Fu;  // the largest finite bf16

// A vector whose head holds the largest magnitude (|c| <= 127 against the largest int8 scale) or
// is not finite (codes 0).
GR_DEVICE uint4 tame(const uint4& w, uint32_t amax) {
  uint4 r = make_uint4(0u, 0u, 0u, 0u);
  if (amax > kTop) return r;
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)  // 254 * 2^120 in place of 255 * 2^120
    o[i] = (v[i] & 0x80008000u) | __vminu2(v[i] & 0x7FFF7FFFu, 0x7F7E7F7Eu);
  return make_uint4(o[0], o[1], o[2], o[3]);
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

// Quantises vector i of the keys and of the values of a row (one head: 8 consecutive lanes, of
// which lanes past the row's vectors hold zeros) into the staged row.
template <int FMT>
GR_DEVICE void put_vectors(uint8_t* row, const QRow& L, int i, uint4 k, uint4 v, bool on) {
  uint32_t mx = max_magnitude(k) | (max_magnitude(v) << 16);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  uint32_t ak = mx & 0xFFFFu, av = mx >> 16;
  float ki, vi, ks, vs;
  if (max(ak, av) >= kTop) {
    k = tame(k, ak);
    v = tame(v, av);
    ks = ak > kTop ? __uint_as_float(0x7FC00000u) : head_scale<FMT>(ak, ki);
    vs = av > kTop ? __uint_as_float(0x7FC00000u) : head_scale<FMT>(av, vi);
    if (ak > kTop) ki = 0.f;
    if (av > kTop) vi = 0.f;
  } else {
    ks = head_scale<FMT>(ak, ki);
    vs = head_scale<FMT>(av, vi);
  }
  constexpr float kBias = FMT == GENRANK_QCACHE_INT8 ? 128.f : 8.f;
  const uint2 ck = code_bytes(k, ki, kMagic + kBias), cv = code_bytes(v, vi, kMagic + kBias);
  if (!on) return;
  if constexpr (FMT == GENRANK_QCACHE_INT8) {
    *reinterpret_cast<uint2*>(row + i * 8) = ck;
    *reinterpret_cast<uint2*>(row + L.scales / 2 + i * 8) = cv;
  } else {
    *reinterpret_cast<uint32_t*>(row + i * 4) = __byte_perm(ck.x | (ck.x >> 4), ck.y | (ck.y >> 4), 0x6420);
    *reinterpret_cast<uint32_t*>(row + L.scales / 2 + i * 4) =
        __byte_perm(cv.x | (cv.x >> 4), cv.y | (cv.y >> 4), 0x6420);
  }
  if ((i & 7) == 0)
    *reinterpret_cast<uint32_t*>(row + L.scales + i / 2) =
        __byte_perm(__float_as_uint(ks), __float_as_uint(vs), 0x7632);
}

// k, v rows -> cache rows.  A piece is 64 of the 8H eight-value vectors of a row's keys and of its
// values, two of each a lane (8 heads: the row); the next piece's loads are in flight while one
// is worked on.  Each row is built in shared memory and leaves as whole 16-byte vectors (pads
// included, so that a row's bytes are defined).  kOne: up to 8 heads, one piece a row.
template <typename Tin, int FMT, bool kOne>
__global__ void __launch_bounds__(kWarps * 32, kOne ? 4 : 1)
    k_qcache_append(const __grid_constant__ QcacheArgs a, int warps, int run) {
  extern __shared__ __align__(16) uint8_t stage_all[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const QRow L = qrow(a.H, FMT);
  uint8_t* row = stage_all + (size_t)warp * L.bytes;
  const int nv = 8 * a.H;  // vectors of one side
  const int pieces = kOne ? 1 : (nv + 63) / 64;
  const long long from = ((long long)blockIdx.x * warps + warp) * run;
  const int t0 = (int)min(from, a.T), t1 = (int)min(from + run, a.T);
  for (int i = lane; i < (L.bytes - L.scales) / 4; i += 32)
    *reinterpret_cast<uint32_t*>(row + L.scales + 4 * i) = 0u;
  __syncwarp();
  Walk<true> walk;
  uint4 k[2], v[2];
  int64_t time = 0;
  int32_t pos = 0;
  auto load = [&](int t, int piece) {
    const Tin* kr = reinterpret_cast<const Tin*>(a.k) + t * a.tok_stride;
    const Tin* vr = reinterpret_cast<const Tin*>(a.v) + t * a.tok_stride;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int i = 64 * piece + 32 * j + lane;
      k[j] = v[j] = make_uint4(0u, 0u, 0u, 0u);
      if (i < nv) {
        k[j] = load_bf16x8<Tin>(kr + 8 * i);
        v[j] = load_bf16x8<Tin>(vr + 8 * i);
      }
    }
    if (lane == 0) {
      time = a.ts[t];
      pos = a.pos[t];
    }
  };
  int t = walk.next(a, t0, t1);
  int piece = 0;  // stays 0 in the one-piece form
  if (t < t1) load(t, 0);
  while (t < t1) {
    uint4 k_now[2] = {k[0], k[1]}, v_now[2] = {v[0], v[1]};
    const int64_t time_now = time;
    const int32_t pos_now = pos;
    const int piece_now = piece;
    uint4* dst = reinterpret_cast<uint4*>(a.cache + walk.row(t) * L.bytes);
    if (kOne || ++piece == pieces) {
      piece = 0;
      t = walk.next(a, t + 1, t1);
    }
    if (t < t1) load(t, piece);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int i = 64 * piece_now + 32 * j + lane;
      if (i - lane < nv) put_vectors<FMT>(row, L, i, k_now[j], v_now[j], i < nv);
    }
    if (piece_now == pieces - 1) {
      if (lane == 0) {
        *reinterpret_cast<int64_t*>(row + L.tail) = time_now;
        *reinterpret_cast<int32_t*>(row + L.tail + 8) = pos_now;
      }
      __syncwarp();
      for (int i = lane; i < L.bytes / 16; i += 32) dst[i] = reinterpret_cast<const uint4*>(row)[i];
      __syncwarp();
    }
  }
  check_users<true>(a, warps);
}

// cache rows -> k, v rows (every value exact in bf16 and fp32); a lane writes 16 bytes at a time,
// so that a warp's stores are whole lines in either type.
template <typename Tout, int FMT, bool kOne>
__global__ void __launch_bounds__(kWarps * 32, kOne ? 4 : 1)
    k_qcache_read(const __grid_constant__ QcacheArgs a, int warps, int run) {
  constexpr int kVals = 16 / sizeof(Tout);  // values of a vector
  constexpr int kVecs = 32 / kVals;         // vectors of a lane in a piece (8 heads: the row)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const QRow L = qrow(a.H, FMT);
  const int nv = kQDh / kVals * a.H;
  const int pieces = kOne ? 1 : (2 * nv + 32 * kVecs - 1) / (32 * kVecs);
  const long long from = ((long long)blockIdx.x * warps + warp) * run;
  const int t0 = (int)min(from, a.T), t1 = (int)min(from + run, a.T);
  Walk<false> walk;
  uint2 w[kVecs];      // codes
  uint16_t sc[kVecs];  // scales
  int4 tail = make_int4(0, 0, 0, 0);
  auto load = [&](int t, int piece) {
    const uint8_t* row = a.cache + walk.row(t) * L.bytes;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int i = 32 * (kVecs * piece + j) + lane;
      w[j] = make_uint2(0u, 0u);
      sc[j] = 0;
      if (i < 2 * nv) {
        const int side = i >= nv, head = (i - side * nv) / (kQDh / kVals);
        sc[j] = __ldg(reinterpret_cast<const uint16_t*>(row + L.scales + head * 4 + side * 2));
        constexpr int bytes = FMT == GENRANK_QCACHE_INT8 ? kVals : kVals / 2;
        if constexpr (bytes == 8)
          w[j] = __ldg(reinterpret_cast<const uint2*>(row + i * 8));
        else if constexpr (bytes == 4)
          w[j].x = __ldg(reinterpret_cast<const uint32_t*>(row + i * 4));
        else
          w[j].x = __ldg(reinterpret_cast<const uint16_t*>(row + i * 2));
      }
    }
    if (lane == 0) tail = __ldg(reinterpret_cast<const int4*>(row + L.tail));
  };
  int t = walk.next(a, t0, t1);
  int piece = 0;  // stays 0 in the one-piece form
  if (t < t1) load(t, 0);
  while (t < t1) {
    uint2 x[kVecs];
    uint16_t s16[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      x[j] = w[j];
      s16[j] = sc[j];
    }
    const int4 tail_now = tail;
    const int tok = t;
    const int piece_now = piece;
    if (kOne || ++piece == pieces) {
      piece = 0;
      t = walk.next(a, t + 1, t1);
    }
    if (t < t1) load(t, piece);
    Tout* kr = reinterpret_cast<Tout*>(a.k_out) + tok * a.tok_stride;
    Tout* vr = reinterpret_cast<Tout*>(a.v_out) + tok * a.tok_stride;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int i = 32 * (kVecs * piece_now + j) + lane;
      if (i >= 2 * nv) break;
      uint2 b = x[j];  // a byte per value
      if constexpr (FMT == GENRANK_QCACHE_INT4) {
        const uint32_t lo = b.x & 0x0F0F0F0Fu, hi = (b.x >> 4) & 0x0F0F0F0Fu;  // even, odd values
        b = make_uint2(__byte_perm(lo, hi, 0x5140), __byte_perm(lo, hi, 0x7362));
      }
      constexpr float kBias = FMT == GENRANK_QCACHE_INT8 ? 128.f : 8.f;
      const float s = __uint_as_float((uint32_t)s16[j] << 16);
      float f[kVals];
#pragma unroll
      for (int e = 0; e < kVals; ++e) {
        // a byte under the exponent of 2^23 reads as 2^23 + byte
        const float y = __uint_as_float(__byte_perm(e < 4 ? b.x : b.y, 0x4B000000u, 0x7440u | (e & 3)));
        f[e] = (y - (8388608.f + kBias)) * s;
      }
      *reinterpret_cast<uint4*>(i < nv ? kr + kVals * i : vr + kVals * (i - nv)) = Elem<Tout>::pack(f);
    }
    if (lane == 0 && piece_now == 0) {
      if (a.ts_out) a.ts_out[tok] = (int64_t)(((uint64_t)(uint32_t)tail_now.y << 32) | (uint32_t)tail_now.x);
      if (a.pos_out) a.pos_out[tok] = tail_now.z;
    }
  }
  check_users<false>(a, warps);
}

template <typename T, int FMT, bool kOne>
int launch_one(const QcacheArgs& a, bool write, cudaStream_t st) {
  static DeviceOnce smem_attr;
  const int sms = sm_count_current();
  if (sms <= 0) return GENRANK_ERR_CUDA;
  const QRow L = qrow(a.H, FMT);
  int warps = kWarps;
  if (write) {
    while (warps > 1 && warps * L.bytes > kMaxStageBytes) warps /= 2;
    if (!set_smem_limit_once(smem_attr, (const void*)k_qcache_append<T, FMT, kOne>, kMaxStageBytes))
      return GENRANK_ERR_CUDA;
  }
  // a run of consecutive rows per warp once every SM has its 32 warps four times over
  const long long most = (long long)sms * 128;
  const long long run = (a.T + most - 1) / most;
  const long long blocks = (a.T + run * warps - 1) / (run * warps);
  if (write)
    k_qcache_append<T, FMT, kOne><<<(unsigned)blocks, warps * 32, warps * L.bytes, st>>>(a, warps, (int)run);
  else
    k_qcache_read<T, FMT, kOne><<<(unsigned)blocks, warps * 32, 0, st>>>(a, warps, (int)run);
  return cudaGetLastError() == cudaSuccess ? GENRANK_OK : GENRANK_ERR_LAUNCH;
}

template <typename T, int FMT>
int launch(const QcacheArgs& a, bool write, cudaStream_t st) {
  return a.H <= 8 ? launch_one<T, FMT, true>(a, write, st) : launch_one<T, FMT, false>(a, write, st);
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
