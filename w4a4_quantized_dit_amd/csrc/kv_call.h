// What the kernels that write and read a paged cache share: their arguments, the block's part of its
// sequence and the thread's unit of a page.
#pragma once

#include "device.h"
#include "kv_layout.h"

namespace svdq {

struct KvArgs {
  const uint16_t* K;     // new rows (write) — or the outputs (read, cast below)
  const uint16_t* V;
  uint16_t* Ko;
  uint16_t* Vo;
  int64_t ldk, ldv, rows;
  const int32_t* cu;
  const int32_t* start;
  const int32_t* table;
  int64_t max_blocks, n_pages;
  uint8_t* kc;
  uint8_t* vc;
  uint8_t* ks;
  uint8_t* vs;
  int heads;
  int64_t max;           // rows of a sequence that are handled
};

// The block's part of its sequence: tokens of page-table entry p, slots [lo, hi), from packed row
// row0 on; false when it has none.
struct Where {
  int64_t row0;
  int p, lo, hi;
};

__device__ __forceinline__ bool locate(const KvArgs& a, Where& w) {
  const int b = blockIdx.z;
  const int64_t first = a.cu[b], end = a.cu[b + 1], start = a.start[b];
  const int64_t n = end - first < a.max ? end - first : a.max;
  if (n <= 0 || first < 0 || end > a.rows || start < 0) return false;
  const int64_t p = start / kPage + blockIdx.x, t0 = p * kPage;
  if (t0 >= start + n || p >= a.max_blocks) return false;
  w.p = (int)p;
  w.lo = (int)(start > t0 ? start - t0 : 0);
  w.hi = (int)(start + n - t0 < kPage ? start + n - t0 : kPage);
  w.row0 = first + (t0 + w.lo - start);
  return true;
}

// The thread's unit: tokens t .. t + 3, channels d .. d + 7.  Lanes run over the channels of a
// row first; the lanes' token groups differ in the bits that select the dword of a V piece.
template <int DIM>
__device__ __forceinline__ void unit_of(int& t, int& d) {
  const int tid = threadIdx.x;
  d = 8 * (tid % (DIM / 8));
  const int g = tid / (DIM / 8);  // 0 .. 15: bits (w1, w0, c1, c0) -> token group (w1, c1, c0, w0)
  t = 4 * ((g & 8) | (g & 3) << 1 | (g >> 2 & 1));
}

template <int DIM>
constexpr int kUnits = kPage / 4 * (DIM / 8);  // threads of a block: 128 or 256

}  // namespace svdq
