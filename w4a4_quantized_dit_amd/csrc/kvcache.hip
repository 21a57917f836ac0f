// The paged 8-bit key / value cache: new tokens quantised as they are written, and read back.
//
// Write.  Per page and head, for K and V each: a = max |new values|, e = the smallest exponent
// with a <= 448·2^e; on a page that already holds earlier tokens of the sequence e is at least
// the stored exponent, and where it grows the stored codes are rounded again to the new scale
// (a power of two, so codes that stay in the normal range keep their value exactly).
//
// Memory-bound: 4 bytes per (token, head, channel) in for K and V together, 2 out.  One block
// per (page, head, sequence); a thread owns a unit of four consecutive tokens and eight channels,
// whose V codes make whole dwords of the stored order (its token is the lowest index) and whose K
// codes make half pieces.  A whole page is gathered in an LDS image and written out in contiguous
// pieces; with units of one token and sixteen channels V went there byte by byte, all lanes on a
// few banks (1008 + 719 tokens x 40 heads of 128: 17.9 us, now 15.2).  On a page that is
// only partly new the units go straight to memory, and the page is read only where codes change.
#include "device.h"
#include "kv_layout.h"
#include "launch.h"

namespace svdq {

namespace {

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

// Bits of the largest finite magnitude that the cache holds: 448·2^119.
constexpr uint32_t kTopBits = 0x7F60;

// Two values as the cache takes them: larger finite ones become ±448·2^119, infinities and NaN
// a NaN, which converts to code 0xFF.  `most` collects the finite magnitudes.
__device__ __forceinline__ uint32_t tame(uint32_t w, uint32_t& most) {
  uint32_t o = 0;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t x = (w >> (16 * k)) & 0xFFFFu, a = x & 0x7FFFu;
    const uint32_t y = a >= kInfBits ? 0x7FFFu : (a > kTopBits ? (x & 0x8000u) | kTopBits : x);
    const uint32_t m = y & 0x7FFFu;
    if (m <= kTopBits && m > most) most = m;
    o |= y << (16 * k);
  }
  return o;
}

// Four fp32 values of at most 448, or NaN, as E4M3 codes (no clamp in front of the conversion).
__device__ __forceinline__ uint32_t fp8x4(float a, float b, float c, float d) {
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(
      c, d, __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false), true);
}

__device__ __forceinline__ float at8(u32x4_t v, int j) {
  return j & 1 ? bf16_hi(v[j >> 1]) : bf16_lo(v[j >> 1]);
}

// Four codes (value times mul, E4M3) of one dword each way: consecutive channels of a token, or
// consecutive tokens of a channel.
__device__ __forceinline__ uint32_t k_code4(u32x4_t v, int j, float mul) {
  return fp8x4(at8(v, j) * mul, at8(v, j + 1) * mul, at8(v, j + 2) * mul, at8(v, j + 3) * mul);
}
__device__ __forceinline__ uint32_t v_code4(const u32x4_t (&v)[4], int j, float mul) {
  return fp8x4(at8(v[0], j) * mul, at8(v[1], j) * mul, at8(v[2], j) * mul, at8(v[3], j) * mul);
}

// One dword of four codes, rounded again for a scale 1/down times as large.
__device__ __forceinline__ uint32_t requantise4(uint32_t w, float down) {
  return fp8x4(__builtin_amdgcn_cvt_f32_fp8((int)w, 0) * down,
               __builtin_amdgcn_cvt_f32_fp8((int)w, 1) * down,
               __builtin_amdgcn_cvt_f32_fp8((int)w, 2) * down,
               __builtin_amdgcn_cvt_f32_fp8((int)w, 3) * down);
}

// Bytes k of a dword with lo <= t + k < hi
__device__ __forceinline__ uint32_t token_bytes(int t, int lo, int hi) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) m |= (t + k >= lo && t + k < hi) ? 0xFFu << (8 * k) : 0u;
  return m;
}

template <int DIM>
__global__ __launch_bounds__(256) void k_kv_write(KvArgs a) {
  constexpr int kThreads = kUnits<DIM>, kWaves = kThreads / 64, kBytes = kPage * DIM;
  __shared__ __attribute__((aligned(16))) uint8_t img[2][kBytes];
  __shared__ uint32_t s_max[2][kWaves], s_fin[2][kWaves];
  Where w;
  if (!locate(a, w)) return;
  const int h = blockIdx.y, tid = threadIdx.x;
  int t, d;
  unit_of<DIM>(t, d);
  const int64_t entry = a.table[(int64_t)blockIdx.z * a.max_blocks + w.p];
  u32x4_t x[2][4];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[kv][i] = u32x4_t{0u, 0u, 0u, 0u};
      if (t + i >= w.lo && t + i < w.hi)
        x[kv][i] = load_nt((kv ? a.V : a.K) + (w.row0 + t + i - w.lo) * (kv ? a.ldv : a.ldk) +
                           (int64_t)h * DIM + d);
    }
  if (entry < 0 || entry >= a.n_pages) return;
  const int64_t at = entry * a.heads + h;
  uint8_t* page[2] = {a.kc + at * kBytes, a.vc + at * kBytes};
  uint8_t* scale[2] = {a.ks + at, a.vs + at};
  int old[2] = {kExpMin, kExpMin};
  if (w.lo > 0) {
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const int e = (int)scale[kv][0] - 127;
      old[kv] = e < kExpMin ? kExpMin : (e > kExpMax ? kExpMax : e);
    }
  }
  // bits of the largest magnitude, of the wave's values and then of the block's
  auto wave_max = [&](uint32_t v, uint32_t& slot) {
#pragma unroll
    for (int k = 1; k < 64; k *= 2) v = max_bf16x2(v, (uint32_t)__shfl_xor((int)v, k));
    if ((tid & 63) == 0) slot = max_bf16x2(v, v >> 16) & 0xFFFFu;
  };
  auto block_max = [&](const uint32_t (&slots)[kWaves]) {
    uint32_t v = slots[0];
#pragma unroll
    for (int k = 1; k < kWaves; ++k) v = slots[k] > v ? slots[k] : v;
    return v;
  };
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) m = max_bf16x2(m, x[kv][i][j] & 0x7FFF7FFFu);
    wave_max(m, s_max[kv][tid >> 6]);
  }
  __syncthreads();
  uint32_t top[2] = {block_max(s_max[0]), block_max(s_max[1])};
  if (top[0] > kTopBits || top[1] > kTopBits) {  // the same for the whole block
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[kv][i][j] = tame(x[kv][i][j], m);
      wave_max(m, s_fin[kv][tid >> 6]);
    }
    __syncthreads();
    top[0] = block_max(s_fin[0]);
    top[1] = block_max(s_fin[1]);
  }
  int e[2];
  float up[2];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    e[kv] = page_exponent(__uint_as_float(top[kv] << 16));
    if (w.lo > 0 && old[kv] > e[kv]) e[kv] = old[kv];
    up[kv] = two_to(-e[kv]);
  }
  if (w.lo == 0 && w.hi == kPage) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<uint2*>(&img[0][k_offset(t + i, d, DIM)]) =
          uint2{k_code4(x[0][i], 0, up[0]), k_code4(x[0][i], 4, up[0])};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      *reinterpret_cast<uint32_t*>(&img[1][v_offset(t, d + j)]) = v_code4(x[1], j, up[1]);
    __syncthreads();
    for (int o = 16 * tid; o < kBytes; o += 16 * kThreads) {
      *reinterpret_cast<u32x4_t*>(page[0] + o) = *reinterpret_cast<const u32x4_t*>(&img[0][o]);
      *reinterpret_cast<u32x4_t*>(page[1] + o) = *reinterpret_cast<const u32x4_t*>(&img[1][o]);
    }
  } else {
    // the scale has grown over the earlier tokens' (then w.lo > 0): they are rounded again
    const bool grow[2] = {w.lo > 0 && e[0] > old[0], w.lo > 0 && e[1] > old[1]};
    const float down[2] = {two_to(old[0] - e[0] < -126 ? -126 : old[0] - e[0]),
                           two_to(old[1] - e[1] < -126 ? -126 : old[1] - e[1])};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint2* dst = reinterpret_cast<uint2*>(page[0] + k_offset(t + i, d, DIM));
      if (t + i >= w.lo && t + i < w.hi) {
        *dst = uint2{k_code4(x[0][i], 0, up[0]), k_code4(x[0][i], 4, up[0])};
      } else if (grow[0] && t + i < w.lo) {
        const uint2 o = *dst;
        *dst = uint2{requantise4(o.x, down[0]), requantise4(o.y, down[0])};
      }
    }
    const uint32_t fresh = token_bytes(t, w.lo, w.hi);
    const uint32_t again = grow[1] ? token_bytes(t, 0, w.lo) : 0u;
    if (fresh | again) {
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        o[j] = fresh == 0xFFFFFFFFu ? 0u : *reinterpret_cast<const uint32_t*>(page[1] + v_offset(t, d + j));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t r = again ? (requantise4(o[j], down[1]) & again) | (o[j] & ~again) : o[j];
        *reinterpret_cast<uint32_t*>(page[1] + v_offset(t, d + j)) =
            (v_code4(x[1], j, up[1]) & fresh) | (r & ~fresh);
      }
    }
  }
  if (tid < 2) scale[tid][0] = (uint8_t)(e[tid] + 127);
}

template <int DIM, bool NT>
__global__ __launch_bounds__(256) void k_kv_read(KvArgs a) {
  constexpr int kThreads = kUnits<DIM>, kBytes = kPage * DIM;
  __shared__ __attribute__((aligned(16))) uint8_t img[2][kBytes];
  Where w;
  if (!locate(a, w)) return;
  const int64_t entry = a.table[(int64_t)blockIdx.z * a.max_blocks + w.p];
  if (entry < 0 || entry >= a.n_pages) return;
  const int h = blockIdx.y, tid = threadIdx.x;
  const int64_t at = entry * a.heads + h;
  const uint8_t* page[2] = {a.kc + at * kBytes, a.vc + at * kBytes};
  for (int o = 16 * tid; o < kBytes; o += 16 * kThreads) {
    *reinterpret_cast<u32x4_t*>(&img[0][o]) = *reinterpret_cast<const u32x4_t*>(page[0] + o);
    *reinterpret_cast<u32x4_t*>(&img[1][o]) = *reinterpret_cast<const u32x4_t*>(page[1] + o);
  }
  const float s[2] = {two_to((int)a.ks[at] - 127), two_to((int)a.vs[at] - 127)};
  __syncthreads();
  int t, d;
  unit_of<DIM>(t, d);
  uint32_t v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = *reinterpret_cast<const uint32_t*>(&img[1][v_offset(t, d + j)]);
  // byte i of a dword of codes, as a value
  auto value = [](uint32_t c, int i) {
    return i == 0 ? __builtin_amdgcn_cvt_f32_fp8((int)c, 0)
         : i == 1 ? __builtin_amdgcn_cvt_f32_fp8((int)c, 1)
         : i == 2 ? __builtin_amdgcn_cvt_f32_fp8((int)c, 2)
                  : __builtin_amdgcn_cvt_f32_fp8((int)c, 3);
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (t + i < w.lo || t + i >= w.hi) continue;
    const int64_t row = w.row0 + t + i - w.lo, col = (int64_t)h * DIM + d;
    const uint2 k = *reinterpret_cast<const uint2*>(&img[0][k_offset(t + i, d, DIM)]);
    u32x4_t ko, vo;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t c = j < 2 ? k.x : k.y;
      ko[j] = pack_bf16x2(value(c, 2 * (j & 1)) * s[0], value(c, 2 * (j & 1) + 1) * s[0]);
      vo[j] = pack_bf16x2(value(v[2 * j], i) * s[1], value(v[2 * j + 1], i) * s[1]);
    }
    store16<NT>(a.Ko + row * a.ldk + col, ko);
    store16<NT>(a.Vo + row * a.ldv + col, vo);
  }
}

}  // namespace

hipError_t launch_kv_write(const uint16_t* K, int64_t ldk, const uint16_t* V, int64_t ldv,
                           int64_t rows, int heads, int dim, const int32_t* cu,
                           const int32_t* start, int64_t B, int64_t max_new, const int32_t* table,
                           int64_t max_blocks, int64_t n_pages, uint8_t* kc, uint8_t* vc,
                           uint8_t* ks, uint8_t* vs, hipStream_t s) {
  const KvArgs a{K, V, nullptr, nullptr, ldk, ldv, rows, cu, start, table, max_blocks, n_pages,
                 kc, vc, ks, vs, heads, max_new};
  // new tokens that start inside a page reach one page more
  const dim3 grid((unsigned)((max_new + kPage - 2) / kPage + 1), (unsigned)heads, (unsigned)B);
  if (dim == 64)
    k_kv_write<64><<<grid, kUnits<64>, 0, s>>>(a);
  else
    k_kv_write<128><<<grid, kUnits<128>, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_kv_read(uint16_t* K, int64_t ldk, uint16_t* V, int64_t ldv, int64_t rows,
                          int heads, int dim, const int32_t* cu, const int32_t* start, int64_t B,
                          int64_t max_n, const int32_t* table, int64_t max_blocks,
                          int64_t n_pages, const uint8_t* kc, const uint8_t* vc,
                          const uint8_t* ks, const uint8_t* vs, hipStream_t s) {
  const KvArgs a{nullptr, nullptr, K, V, ldk, ldv, rows, cu, start, table, max_blocks, n_pages,
                 const_cast<uint8_t*>(kc), const_cast<uint8_t*>(vc), const_cast<uint8_t*>(ks),
                 const_cast<uint8_t*>(vs), heads, max_n};
  const dim3 grid((unsigned)((max_n + kPage - 2) / kPage + 1), (unsigned)heads, (unsigned)B);
  const bool nt = rows * heads * dim * 4 > kPastCaches;
  if (dim == 64)
    nt ? k_kv_read<64, true><<<grid, kUnits<64>, 0, s>>>(a)
       : k_kv_read<64, false><<<grid, kUnits<64>, 0, s>>>(a);
  else
    nt ? k_kv_read<128, true><<<grid, kUnits<128>, 0, s>>>(a)
       : k_kv_read<128, false><<<grid, kUnits<128>, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace svdq
