// The paged 4-bit key / value cache: new tokens quantised as they are written, and read back.
//
// Write.  Per token, head and 32 channels, for K and V each: a = max |x|, e = floor(log2 a) − 2 within
// [kExp4Min, kExp4Max], code = E2M1(x·2^−e), nearest even, at most ±6.  bf16's exponent field is
// floor(log2 a) + 127, so the scale byte comes from the bits of the maximum without arithmetic, and the
// conversions to and from E2M1 take bf16 pairs and the scale as they are (checked against every bf16
// value at five scales).  A block with an infinity or NaN gets the scale byte 255 and codes 0.
//
// Memory-bound: 4 bytes per (token, head, channel) in for K and V together, 1.0625 out.  One block per
// (page, head, sequence); a thread owns four consecutive tokens of eight channels: a K dword for each
// token, and a V dword (two channels of the four tokens) for each pair of channels.  A page of which
// every token is new is gathered in an LDS image and written in contiguous pieces of 16 bytes a thread;
// of the others only the new tokens' own bytes are written.  16384 tokens of 40 heads of 128 take 74 to 79 us
// to write and 65 to read back, 5.9 TB/s together; a token of each of 32 streams 4 us each way.
#include "device.h"
#include "kv4_layout.h"
#include "kv_call.h"
#include "launch.h"

namespace svdq {

namespace {

// Byte of the scale of a block whose largest magnitude has the bits m.
__device__ __forceinline__ uint32_t scale_byte(uint32_t m) {
  if (m >= kInfBits) return kNan4;
  const int b = (int)(m >> 7) - 2;
  return (uint32_t)(b < kExp4Min + 127 ? kExp4Min + 127 : (b > kExp4Max + 127 ? kExp4Max + 127 : b));
}

template <int DIM>
__global__ __launch_bounds__(256) void k_kv4_write(KvArgs a) {
  constexpr int kThreads = kUnits<DIM>, kBytes = kPage * DIM / 2, kScales = kPage * DIM / 32;
  static_assert(kBytes == 16 * kThreads, "a page's codes are 16 bytes a thread");
  __shared__ __attribute__((aligned(16))) uint8_t img[2][kBytes], img_s[2][kScales];
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
  uint8_t* scales[2] = {a.ks + at * kScales, a.vs + at * kScales};
  // scale bytes of the thread's four tokens: the four lanes side by side have a block's channels
  uint32_t s[2][4];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    uint32_t m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u32x4_t v = x[kv][i];
      m[i] = max_bf16x2(max_bf16x2(v[0] & 0x7FFF7FFFu, v[1] & 0x7FFF7FFFu),
                        max_bf16x2(v[2] & 0x7FFF7FFFu, v[3] & 0x7FFF7FFFu));
    }
#pragma unroll
    for (int i = 0; i < 4; i += 2) {  // two tokens in a dword across the lanes
      uint32_t p = max_bf16x2((m[i] & 0xFFFFu) | m[i + 1] << 16, m[i] >> 16 | (m[i + 1] & 0xFFFF0000u));
      p = max_bf16x2(p, (uint32_t)__shfl_xor((int)p, 1));
      p = max_bf16x2(p, (uint32_t)__shfl_xor((int)p, 2));
      s[kv][i] = scale_byte(p & 0xFFFFu);
      s[kv][i + 1] = scale_byte(p >> 16);
    }
  }
  uint32_t kw[4], vw[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float ku = __uint_as_float(s[0][i] << 23), vu = __uint_as_float(s[1][i] << 23);
    uint32_t c = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) c = code2(c, x[0][i][j], j, ku);
    kw[i] = s[0][i] == kNan4 ? 0u : c;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      vw[j] = s[1][i] == kNan4 ? vw[j] : code2(vw[j], x[1][i][j], i, vu);
  }
  const uint32_t v_scales = s[1][0] | s[1][1] << 8 | s[1][2] << 16 | s[1][3] << 24;
  const bool first = (tid & 3) == 0;  // of the block's four lanes
  if (w.lo == 0 && w.hi == kPage) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      *reinterpret_cast<uint32_t*>(&img[0][k4_offset(t + i, d, DIM)]) = kw[i];
      *reinterpret_cast<uint32_t*>(&img[1][v4_offset(t, d + 2 * i)]) = vw[i];
      if (first) img_s[0][k4_scale_offset(t + i, d, DIM)] = (uint8_t)s[0][i];
    }
    if (first) *reinterpret_cast<uint32_t*>(&img_s[1][v4_scale_offset(t, d)]) = v_scales;
    __syncthreads();
    const int o = 16 * tid;
    *reinterpret_cast<u32x4_t*>(page[0] + o) = *reinterpret_cast<const u32x4_t*>(&img[0][o]);
    *reinterpret_cast<u32x4_t*>(page[1] + o) = *reinterpret_cast<const u32x4_t*>(&img[1][o]);
    if (o < 2 * kScales) {
      const int which = o >= kScales, so = o - which * kScales;
      *reinterpret_cast<u32x4_t*>((which ? scales[1] : scales[0]) + so) =
          *reinterpret_cast<const u32x4_t*>(&img_s[which][so]);
    }
    return;
  }
  if (t + 3 < w.lo || t >= w.hi) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (t + i < w.lo || t + i >= w.hi) continue;
    *reinterpret_cast<uint32_t*>(page[0] + k4_offset(t + i, d, DIM)) = kw[i];
    if (first) scales[0][k4_scale_offset(t + i, d, DIM)] = (uint8_t)s[0][i];
  }
  if (t >= w.lo && t + 3 < w.hi) {
#pragma unroll
    for (int j = 0; j < 4; ++j) *reinterpret_cast<uint32_t*>(page[1] + v4_offset(t, d + 2 * j)) = vw[j];
    if (first) *reinterpret_cast<uint32_t*>(scales[1] + v4_scale_offset(t, d)) = v_scales;
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (t + i < w.lo || t + i >= w.hi) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) page[1][v4_offset(t, d + 2 * j) + i] = (uint8_t)(vw[j] >> (8 * i));
    if (first) scales[1][v4_scale_offset(t, d) + i] = (uint8_t)s[1][i];
  }
}

template <int DIM, bool NT>
__global__ __launch_bounds__(256) void k_kv4_read(KvArgs a) {
  constexpr int kBytes = kPage * DIM / 2, kScales = kPage * DIM / 32;
  __shared__ __attribute__((aligned(16))) uint8_t img[2][kBytes], img_s[2][kScales];
  Where w;
  if (!locate(a, w)) return;
  const int64_t entry = a.table[(int64_t)blockIdx.z * a.max_blocks + w.p];
  if (entry < 0 || entry >= a.n_pages) return;
  const int h = blockIdx.y, tid = threadIdx.x, o = 16 * tid;
  const int64_t at = entry * a.heads + h;
  *reinterpret_cast<u32x4_t*>(&img[0][o]) =
      *reinterpret_cast<const u32x4_t*>(a.kc + at * kBytes + o);
  *reinterpret_cast<u32x4_t*>(&img[1][o]) =
      *reinterpret_cast<const u32x4_t*>(a.vc + at * kBytes + o);
  if (o < 2 * kScales) {
    const int which = o >= kScales, so = o - which * kScales;
    *reinterpret_cast<u32x4_t*>(&img_s[which][so]) =
        *reinterpret_cast<const u32x4_t*>((which ? a.vs : a.ks) + at * kScales + so);
  }
  __syncthreads();
  int t, d;
  unit_of<DIM>(t, d);
  uint32_t v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const uint32_t*>(&img[1][v4_offset(t, d + 2 * j)]);
  const uint32_t v_scales = *reinterpret_cast<const uint32_t*>(&img_s[1][v4_scale_offset(t, d)]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (t + i < w.lo || t + i >= w.hi) continue;
    const int64_t row = w.row0 + t + i - w.lo, col = (int64_t)h * DIM + d;
    const uint32_t k = *reinterpret_cast<const uint32_t*>(&img[0][k4_offset(t + i, d, DIM)]);
    const float ks = scale4(img_s[0][k4_scale_offset(t + i, d, DIM)], 0), vs = scale4(v_scales, i);
    u32x4_t ko, vo;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      ko[j] = widen2(k, j, ks);
      vo[j] = widen2(v[j], i, vs);
    }
    store16<NT>(a.Ko + row * a.ldk + col, ko);
    store16<NT>(a.Vo + row * a.ldv + col, vo);
  }
}

}  // namespace

hipError_t launch_kv4_write(const uint16_t* K, int64_t ldk, const uint16_t* V, int64_t ldv,
                            int64_t rows, int heads, int dim, const int32_t* cu,
                            const int32_t* start, int64_t B, int64_t max_new, const int32_t* table,
                            int64_t max_blocks, int64_t n_pages, uint8_t* kc, uint8_t* vc,
                            uint8_t* ks, uint8_t* vs, hipStream_t s) {
  const KvArgs a{K, V, nullptr, nullptr, ldk, ldv, rows, cu, start, table, max_blocks, n_pages,
                 kc, vc, ks, vs, heads, max_new};
  // new tokens that start inside a page reach one page more
  const dim3 grid((unsigned)((max_new + kPage - 2) / kPage + 1), (unsigned)heads, (unsigned)B);
  if (dim == 64)
    k_kv4_write<64><<<grid, kUnits<64>, 0, s>>>(a);
  else
    k_kv4_write<128><<<grid, kUnits<128>, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_kv4_read(uint16_t* K, int64_t ldk, uint16_t* V, int64_t ldv, int64_t rows,
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
    nt ? k_kv4_read<64, true><<<grid, kUnits<64>, 0, s>>>(a)
       : k_kv4_read<64, false><<<grid, kUnits<64>, 0, s>>>(a);
  else
    nt ? k_kv4_read<128, true><<<grid, kUnits<128>, 0, s>>>(a)
       : k_kv4_read<128, false><<<grid, kUnits<128>, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace svdq
