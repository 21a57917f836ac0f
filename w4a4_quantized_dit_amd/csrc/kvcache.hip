// The paged 8-bit key / value cache: new tokens quantised as they are written, and read back.
//
// Write.  Per page and head, for K and V each: a = max |new values|, e = the smallest exponent
// with a <= 448·2^e; on a page that already holds earlier tokens of the sequence e is at least
// the stored exponent, and where it grows the stored codes are rounded again to the new scale
// (a power of two, so codes that stay in the normal range keep their value exactly).
//
// Memory-bound: 4 bytes per (token, head, channel) in for K and V together, 2 out.  One block
// per (page, head, sequence): the rows are read whole, encoded into an LDS image of the page in
// its stored order, and the image is written out in contiguous pieces.
#include "device.h"
#include "kv_layout.h"
#include "launch.h"

namespace svdq {

namespace {

constexpr int kThreads = 256;

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
};

// The block's page: rows [row0 + slot) of the packed input for slots [lo, hi), or false.
struct Where {
  int64_t page;   // index into the cache
  int64_t row0;   // packed row of slot lo
  int lo, hi;
};

__device__ __forceinline__ bool locate(const KvArgs& a, Where& w) {
  const int b = blockIdx.z;
  const int64_t first = a.cu[b], start = a.start[b];
  const int64_t n = (int64_t)a.cu[b + 1] - first;
  if (n <= 0 || first < 0 || first + n > a.rows || start < 0) return false;
  const int64_t p = start / kPage + blockIdx.x;
  const int64_t t0 = p * kPage;
  if (t0 >= start + n || p >= a.max_blocks) return false;
  w.page = a.table[(int64_t)b * a.max_blocks + p];
  if (w.page < 0 || w.page >= a.n_pages) return false;
  w.lo = (int)(start > t0 ? start - t0 : 0);
  w.hi = (int)(start + n - t0 < kPage ? start + n - t0 : kPage);
  w.row0 = first + (t0 + w.lo - start);
  return true;
}

__device__ __forceinline__ float abs_max16(u32x4_t a, u32x4_t b) {
  float m = 0.0f;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    m = fmaxf(m, fmaxf(fabsf(bf16_lo(a[c])), fabsf(bf16_hi(a[c]))));
    m = fmaxf(m, fmaxf(fabsf(bf16_lo(b[c])), fabsf(bf16_hi(b[c]))));
  }
  return m;
}

// One dword of four codes, rounded again for a scale 2^down times as large.
__device__ __forceinline__ uint32_t requantise4(uint32_t w, float down) {
  return e4m3_pack4(__builtin_amdgcn_cvt_f32_fp8((int)w, 0) * down,
                    __builtin_amdgcn_cvt_f32_fp8((int)w, 1) * down,
                    __builtin_amdgcn_cvt_f32_fp8((int)w, 2) * down,
                    __builtin_amdgcn_cvt_f32_fp8((int)w, 3) * down);
}

template <int DIM>
__global__ __launch_bounds__(kThreads) void k_kv_write(KvArgs a) {
  constexpr int kPieces = kPage * DIM / 16;            // 16-channel pieces of the page
  constexpr int kPer = kPieces / kThreads;             // per thread: 1 (dim 64) or 2 (dim 128)
  constexpr int kBytes = kPage * DIM;
  __shared__ __attribute__((aligned(16))) uint8_t img[2][kBytes];
  __shared__ float s_max[2][kThreads / 64];
  Where w;
  if (!locate(a, w)) return;
  const int h = blockIdx.y, tid = threadIdx.x;
  const int64_t at = w.page * a.heads + h;
  uint8_t* page[2] = {a.kc + at * kBytes, a.vc + at * kBytes};
  uint8_t* scale[2] = {a.ks + at, a.vs + at};

  // the new rows: piece p = token slot p / (DIM/16), channels 16·(p % (DIM/16)) on
  u32x4_t x[2][kPer][2];
  float m[2] = {0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int p = tid + kThreads * i, t = p / (DIM / 16), d = 16 * (p % (DIM / 16));
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      x[kv][i][0] = x[kv][i][1] = u32x4_t{0u, 0u, 0u, 0u};
      if (t >= w.lo && t < w.hi) {
        const uint16_t* src = (kv ? a.V : a.K) + (w.row0 + t - w.lo) * (kv ? a.ldv : a.ldk) +
                              (int64_t)h * DIM + d;
        x[kv][i][0] = reinterpret_cast<const u32x4_t*>(src)[0];
        x[kv][i][1] = reinterpret_cast<const u32x4_t*>(src)[1];
        m[kv] = fmaxf(m[kv], abs_max16(x[kv][i][0], x[kv][i][1]));
      }
    }
  }
  const bool part = w.lo > 0 || w.hi < kPage;
  if (part) {  // the page's other codes are kept
    for (int o = 16 * tid; o < kBytes; o += 16 * kThreads) {
      *reinterpret_cast<u32x4_t*>(&img[0][o]) = *reinterpret_cast<const u32x4_t*>(page[0] + o);
      *reinterpret_cast<u32x4_t*>(&img[1][o]) = *reinterpret_cast<const u32x4_t*>(page[1] + o);
    }
  }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) m[kv] = fmaxf(m[kv], __shfl_xor(m[kv], d));
    if ((tid & 63) == 0) s_max[kv][tid >> 6] = m[kv];
  }
  const int old[2] = {w.lo > 0 ? (int)scale[0][0] - 127 : kExpMin,
                      w.lo > 0 ? (int)scale[1][0] - 127 : kExpMin};
  __syncthreads();
  int e[2];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const float mm = fmaxf(fmaxf(s_max[kv][0], s_max[kv][1]), fmaxf(s_max[kv][2], s_max[kv][3]));
    e[kv] = page_exponent(mm);
    const int o = old[kv] < kExpMin ? kExpMin : (old[kv] > kExpMax ? kExpMax : old[kv]);
    if (w.lo > 0 && o > e[kv]) e[kv] = o;
    if (w.lo > 0 && e[kv] > o) {
      // dword i of the image holds four codes of one token (K) or of four consecutive tokens
      // (V: slots 32·(frag%2) + 16·(i/2%2) + 8·(i%2) + 4·(lane/32) on)
      const int drop = o - e[kv];
      const float down = two_to(drop < -126 ? -126 : drop);
      for (int i = tid; i < kBytes / 4; i += kThreads) {
        uint32_t* q = reinterpret_cast<uint32_t*>(&img[kv][4 * i]);
        const int frag = i >> 8, lane = (i >> 2) & 63, dw = i & 3;
        const uint32_t word = *q, again = requantise4(word, down);
        if (kv == 0) {
          const int t = 32 * (frag / (2 * (DIM / 64))) + (lane & 31);
          if (t < w.lo) *q = again;
        } else {
          const int t = 32 * (frag & 1) + 16 * (dw >> 1) + 8 * (dw & 1) + 4 * (lane >> 5);
          const int n = w.lo - t < 0 ? 0 : (w.lo - t > 4 ? 4 : w.lo - t);
          const uint32_t mask = n == 4 ? 0xFFFFFFFFu : (1u << (8 * n)) - 1u;
          *q = (again & mask) | (word & ~mask);
        }
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int p = tid + kThreads * i, t = p / (DIM / 16), d = 16 * (p % (DIM / 16));
    if (t >= w.lo && t < w.hi) {
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const float up = two_to(-e[kv]);
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t w0 = j < 2 ? x[kv][i][0][2 * j] : x[kv][i][1][2 * j - 4];
          const uint32_t w1 = j < 2 ? x[kv][i][0][2 * j + 1] : x[kv][i][1][2 * j - 3];
          c[j] = e4m3_pack4(bf16_lo(w0) * up, bf16_hi(w0) * up, bf16_lo(w1) * up, bf16_hi(w1) * up);
        }
        if (kv == 0) {
          *reinterpret_cast<u32x4_t*>(&img[0][k_offset(t, d, DIM)]) = u32x4_t{c[0], c[1], c[2], c[3]};
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            img[1][v_offset(t, d + j)] = (uint8_t)(c[j >> 2] >> (8 * (j & 3)));
        }
      }
    }
  }
  __syncthreads();
  for (int o = 16 * tid; o < kBytes; o += 16 * kThreads) {
    *reinterpret_cast<u32x4_t*>(page[0] + o) = *reinterpret_cast<const u32x4_t*>(&img[0][o]);
    *reinterpret_cast<u32x4_t*>(page[1] + o) = *reinterpret_cast<const u32x4_t*>(&img[1][o]);
  }
  if (tid < 2) scale[tid][0] = (uint8_t)(e[tid] + 127);
}

template <int DIM>
__global__ __launch_bounds__(kThreads) void k_kv_read(KvArgs a) {
  constexpr int kPer = kPage * DIM / 16 / kThreads;
  constexpr int kBytes = kPage * DIM;
  __shared__ __attribute__((aligned(16))) uint8_t img[2][kBytes];
  Where w;
  if (!locate(a, w)) return;
  const int h = blockIdx.y, tid = threadIdx.x;
  const int64_t at = w.page * a.heads + h;
  const uint8_t* page[2] = {a.kc + at * kBytes, a.vc + at * kBytes};
  for (int o = 16 * tid; o < kBytes; o += 16 * kThreads) {
    *reinterpret_cast<u32x4_t*>(&img[0][o]) = *reinterpret_cast<const u32x4_t*>(page[0] + o);
    *reinterpret_cast<u32x4_t*>(&img[1][o]) = *reinterpret_cast<const u32x4_t*>(page[1] + o);
  }
  const float s[2] = {two_to((int)a.ks[at] - 127), two_to((int)a.vs[at] - 127)};
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int p = tid + kThreads * i, t = p / (DIM / 16), d = 16 * (p % (DIM / 16));
    if (t < w.lo || t >= w.hi) continue;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      uint32_t c[4];
      if (kv == 0) {
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(&img[0][k_offset(t, d, DIM)]);
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] = v[j];
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          c[j] = 0;
#pragma unroll
          for (int b = 0; b < 4; ++b)
            c[j] |= (uint32_t)img[1][v_offset(t, d + 4 * j + b)] << (8 * b);
        }
      }
      uint16_t* dst = (kv ? a.Vo : a.Ko) + (w.row0 + t - w.lo) * (kv ? a.ldv : a.ldk) +
                      (int64_t)h * DIM + d;
      u32x4_t o[2];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        o[j >> 1][2 * (j & 1)] = pack_bf16x2(__builtin_amdgcn_cvt_f32_fp8((int)c[j], 0) * s[kv],
                                             __builtin_amdgcn_cvt_f32_fp8((int)c[j], 1) * s[kv]);
        o[j >> 1][2 * (j & 1) + 1] = pack_bf16x2(__builtin_amdgcn_cvt_f32_fp8((int)c[j], 2) * s[kv],
                                                 __builtin_amdgcn_cvt_f32_fp8((int)c[j], 3) * s[kv]);
      }
      reinterpret_cast<u32x4_t*>(dst)[0] = o[0];
      reinterpret_cast<u32x4_t*>(dst)[1] = o[1];
    }
  }
}

}  // namespace

hipError_t launch_kv_write(const uint16_t* K, int64_t ldk, const uint16_t* V, int64_t ldv,
                           int64_t rows, int heads, int dim, const int32_t* cu,
                           const int32_t* start, int64_t B, int64_t max_new, const int32_t* table,
                           int64_t max_blocks, int64_t n_pages, uint8_t* kc, uint8_t* vc,
                           uint8_t* ks, uint8_t* vs, hipStream_t s) {
  const KvArgs a{K, V, nullptr, nullptr, ldk, ldv, rows, cu, start, table, max_blocks, n_pages,
                 kc, vc, ks, vs, heads};
  // new tokens that start inside a page reach one page more
  const dim3 grid((unsigned)((max_new + kPage - 2) / kPage + 1), (unsigned)heads, (unsigned)B);
  if (dim == 64)
    k_kv_write<64><<<grid, kThreads, 0, s>>>(a);
  else
    k_kv_write<128><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_kv_read(uint16_t* K, int64_t ldk, uint16_t* V, int64_t ldv, int64_t rows,
                          int heads, int dim, const int32_t* cu, const int32_t* start, int64_t B,
                          int64_t max_n, const int32_t* table, int64_t max_blocks,
                          int64_t n_pages, const uint8_t* kc, const uint8_t* vc,
                          const uint8_t* ks, const uint8_t* vs, hipStream_t s) {
  const KvArgs a{nullptr, nullptr, K, V, ldk, ldv, rows, cu, start, table, max_blocks, n_pages,
                 const_cast<uint8_t*>(kc), const_cast<uint8_t*>(vc), const_cast<uint8_t*>(ks),
                 const_cast<uint8_t*>(vs), heads};
  const dim3 grid((unsigned)((max_n + kPage - 2) / kPage + 1), (unsigned)heads, (unsigned)B);
  if (dim == 64)
    k_kv_read<64><<<grid, kThreads, 0, s>>>(a);
  else
    k_kv_read<128><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace svdq
