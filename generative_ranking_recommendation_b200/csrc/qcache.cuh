// The row format of the quantised history cache (see include/genrank.h).
#pragma once

#include <stdint.h>

#include "genrank.h"

namespace gr {

constexpr int kQDh = 64;          // values per head
constexpr int kQMaxLen = 1 << 30;  // rows of a history
constexpr int kQPart = kQDh + 2;  // floats of a joined range: O, then its maximum and sum

// Byte offsets inside one row of H heads:
//   [K codes H x cb][V codes H x cb][(K scale, V scale) bf16 x H][pad to 16]
//   [ts int64, pos int32, 0][pad to an odd multiple of 16]
// A row is an odd number of 16-byte units: rows of one parity then start in different
// shared-memory bank groups, so that eight lanes reading eight rows do not collide.
struct QRow {
  int cb;      // code bytes of one head
  int scales;  // offset of the scales (= 2 H cb)
  int tail;    // offset of the time and the position
  int bytes;   // bytes of a row
};

__host__ __device__ constexpr QRow qrow(int H, int format) {
  QRow r{};
  r.cb = format == GENRANK_QCACHE_INT8 ? kQDh : kQDh / 2;
  r.scales = 2 * H * r.cb;
  r.tail = (r.scales + 4 * H + 15) / 16 * 16;
  r.bytes = r.tail + 16;
  if (r.bytes / 16 % 2 == 0) r.bytes += 16;
  return r;
}

#ifdef __CUDACC__
// A kernel launched to follow another early (programmatic stream serialisation) starts once every
// block of that one has called grid_release or ended, and waits in grid_wait for its end and results.
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
#endif

}  // namespace gr
