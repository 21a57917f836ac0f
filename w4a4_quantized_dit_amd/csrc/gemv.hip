// The layer's product for a few rows with 16-bit activations (no activation quantisation):
//
//   Y[m, n] = bf16( Σ_k x̂[m, k]·w[n, k] + Σ_j D[m, j]·up[n, j] ),  x̂ = bf16(x·fl32(1/λ)),
//   D = x̂·downᵀ,  w = the weight that its codes and scales stand for
//
// Bound by the weight's bytes, and for single rows by the latency of one pass over K.  The product
// runs on the 16x16x32 bf16 MFMA with the rows padded to 16: the codes are widened to bf16 once for
// every 16 rows, which for one row costs no more than a product a lane and leaves the same kernel for
// 64.  Every product is exact in the fp32 sum: an E2M1 code times a power of two (MXFP4) or times an
// E4M3 scale (NVFP4, six significant bits) is a bf16; int4 codes are widened alone, and their group's
// scale multiplies the sum of the group's 64 products.
//
// A block takes NT·16 outputs; its waves take every eighth piece of 128 channels, 16 bytes of codes a
// lane and weight row, with the next piece's loads under way, and their sums are joined through LDS in
// the waves' order.  x̂ and D come from a kernel in front (none is launched without smoothing and
// low-rank branch), where the down factor takes the weight's place.
#include "device.h"
#include "launch.h"

namespace svdq {

namespace {

constexpr int kFmtNv = 0, kFmtInt4 = 1, kFmtMx = 2;  // svdq_format
constexpr int kPiece = 128;                          // channels of a wave's step

// The lane's channels of its step `i` (0 .. 3) of a piece: eight from here on.  The codes that a lane
// loads together lie in one scale's block (E2M1), or a quarter of each of the two groups (int4).
template <int FMT>
__device__ __forceinline__ int step_channel(int q, int i) {
  return FMT == kFmtInt4 ? 64 * (i >> 1) + 16 * q + 8 * (i & 1) : 32 * q + 8 * i;
}

// A lane's codes and scales of a piece of one weight row.
struct Codes {
  uint32_t w[4];
  uint32_t s;
};

template <int FMT>
__device__ __forceinline__ void load_codes(const uint8_t* row, const uint8_t* scales, int64_t k0, int q,
                                           Codes& c) {
  if (FMT == kFmtInt4) {
    const uint2 lo = __builtin_bit_cast(uint2, __builtin_nontemporal_load(
                         reinterpret_cast<const uint64_t*>(row + (k0 >> 1) + 8 * q)));
    const uint2 hi = __builtin_bit_cast(uint2, __builtin_nontemporal_load(
                         reinterpret_cast<const uint64_t*>(row + (k0 >> 1) + 32 + 8 * q)));
    c.w[0] = lo.x; c.w[1] = lo.y; c.w[2] = hi.x; c.w[3] = hi.y;
    c.s = *reinterpret_cast<const uint32_t*>(scales + (k0 >> 5));  // two fp16
  } else {
    const u32x4_t v = load_nt(row + (k0 >> 1) + 16 * q);
    c.w[0] = v[0]; c.w[1] = v[1]; c.w[2] = v[2]; c.w[3] = v[3];
    if (FMT == kFmtNv)
      c.s = *reinterpret_cast<const uint16_t*>(scales + (k0 >> 4) + 2 * q);  // two E4M3
    else
      c.s = scales[(k0 >> 5) + q];                                           // E8M0
  }
}

// Step i's operand of a weight row.
template <int FMT>
__device__ __forceinline__ bf16x8_t widen(const Codes& c, int i) {
  const uint32_t w = c.w[i];
  u32x4_t r;
  if (FMT == kFmtMx) {
    const float s = __uint_as_float(c.s << 23);
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
  } else if (FMT == kFmtNv) {
    const float s = i < 2 ? __builtin_amdgcn_cvt_f32_fp8((int)c.s, 0) : __builtin_amdgcn_cvt_f32_fp8((int)c.s, 1);
    const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
    const auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    const auto d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
    const auto e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
    r[0] = pack_bf16x2(a[0] * s, a[1] * s);
    r[1] = pack_bf16x2(b[0] * s, b[1] * s);
    r[2] = pack_bf16x2(d[0] * s, d[1] * s);
    r[3] = pack_bf16x2(e[0] * s, e[1] * s);
  } else {
    // the conversion takes the lowest nibble as a signed number of sixteenths
#pragma unroll
    for (int j = 0; j < 4; ++j)
      r[j] = pack_bf16x2(__builtin_amdgcn_cvt_off_f32_i4((int)(w >> (8 * j))),
                         __builtin_amdgcn_cvt_off_f32_i4((int)(w >> (8 * j + 4))));
  }
  return __builtin_bit_cast(bf16x8_t, r);
}

struct GemvArgs {
  const uint16_t* X;       // x̂ [M, K] bf16
  const uint8_t* codes;
  const uint8_t* scales;
  const float* g;          // or NULL
  const float* D;          // [M, r], or NULL
  const uint16_t* up;      // [N, r]
  uint16_t* Y;
  int64_t K, ldx, ldy;
  int M, N, r;
};

constexpr int kGemvWaves = 8;

template <int FMT, int MT, int NT>
__global__ __launch_bounds__(64 * kGemvWaves) void k_gemv(GemvArgs a) {
  __shared__ float s_sum[kGemvWaves][MT * 16][NT * 16 + 1];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int n16 = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * (NT * 16);
  constexpr int kGroup = FMT == kFmtNv ? 16 : FMT == kFmtMx ? 32 : 64;
  constexpr int kScaleBytes = FMT == kFmtInt4 ? 2 : 1;
  const uint8_t* row[NT];
  const uint8_t* srow[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int64_t n = n0 + 16 * t + n16 < a.N ? n0 + 16 * t + n16 : a.N - 1;  // (past N: not stored)
    row[t] = a.codes + n * (a.K / 2);
    srow[t] = a.scales + n * (a.K / kGroup) * kScaleBytes;
  }
  const uint16_t* x[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) x[t] = a.X + (int64_t)(16 * t + n16 < a.M ? 16 * t + n16 : a.M - 1) * a.ldx;

  f32x4_t acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[m][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int pieces = (int)(a.K / kPiece);
  Codes next[NT];
  u32x4_t xn[MT][4];
  auto load = [&](int p) {
#pragma unroll
    for (int t = 0; t < NT; ++t) load_codes<FMT>(row[t], srow[t], (int64_t)p * kPiece, q, next[t]);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        xn[m][i] = *reinterpret_cast<const u32x4_t*>(x[m] + (int64_t)p * kPiece + step_channel<FMT>(q, i));
  };
  if (wave < pieces) load(wave);
  for (int p = wave; p < pieces; p += kGemvWaves) {
    Codes c[NT];
    u32x4_t xv[MT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) c[t] = next[t];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) xv[m][i] = xn[m][i];
    if (p + kGemvWaves < pieces) load(p + kGemvWaves);
    if (FMT == kFmtInt4) {
#pragma unroll
      for (int gr = 0; gr < 2; ++gr)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const bf16x8_t w0 = widen<FMT>(c[t], 2 * gr), w1 = widen<FMT>(c[t], 2 * gr + 1);
          const uint16_t h = (uint16_t)(c[t].s >> (16 * gr));
          const float s = 16.0f * (float)__builtin_bit_cast(_Float16, h);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            f32x4_t part = {0.f, 0.f, 0.f, 0.f};
            part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, xv[m][2 * gr]), w0, part, 0, 0, 0);
            part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, xv[m][2 * gr + 1]), w1, part, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[m][t][j] = __builtin_fmaf(s, part[j], acc[m][t][j]);
          }
        }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const bf16x8_t w = widen<FMT>(c[t], i);
#pragma unroll
          for (int m = 0; m < MT; ++m)
            acc[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, xv[m][i]), w, acc[m][t], 0, 0, 0);
        }
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) s_sum[wave][16 * m + 4 * q + j][16 * t + n16] = acc[m][t][j];
  __syncthreads();
  const float g = a.g ? a.g[0] : 1.0f;
  for (int o = threadIdx.x; o < a.M * NT * 16; o += 64 * kGemvWaves) {
    const int m = o / (NT * 16), n = o % (NT * 16);
    if (n0 + n >= a.N) continue;
    float y = 0.0f;
#pragma unroll
    for (int w = 0; w < kGemvWaves; ++w) y += s_sum[w][m][n];
    y *= g;
    if (a.r) {
      const f32x4_t* d = reinterpret_cast<const f32x4_t*>(a.D + (int64_t)m * a.r);
      const u32x4_t* u = reinterpret_cast<const u32x4_t*>(a.up + (int64_t)(n0 + n) * a.r);
      float z = 0.0f;
      for (int j = 0; j < a.r / 8; ++j) {
        const u32x4_t v = u[j];
        const f32x4_t d0 = d[2 * j], d1 = d[2 * j + 1];
        z = __builtin_fmaf(d0[0], bf16_lo(v[0]), z);
        z = __builtin_fmaf(d0[1], bf16_hi(v[0]), z);
        z = __builtin_fmaf(d0[2], bf16_lo(v[1]), z);
        z = __builtin_fmaf(d0[3], bf16_hi(v[1]), z);
        z = __builtin_fmaf(d1[0], bf16_lo(v[2]), z);
        z = __builtin_fmaf(d1[1], bf16_hi(v[2]), z);
        z = __builtin_fmaf(d1[2], bf16_lo(v[3]), z);
        z = __builtin_fmaf(d1[3], bf16_hi(v[3]), z);
      }
      y += z;
    }
    a.Y[(int64_t)m * a.ldy + n0 + n] = f32_to_bf16(y);
  }
}

struct PrepArgs {
  const uint16_t* X;
  const float* lambda;     // or NULL
  const uint16_t* down;    // [r, K], or NULL
  uint16_t* xhat;          // [M, K], with lambda
  float* D;                // [M, r]
  int64_t K, ldx;
  int M, r;
};

constexpr int kPrepWaves = 16;

// x̂ and D: a block takes 16 rows (blockIdx.y) and 16 ranks (blockIdx.x; those of the first ranks store
// x̂), its waves every sixteenth piece.  A wave forms the reciprocals of its piece's λ once, two a lane.
template <bool SMOOTH>
__global__ __launch_bounds__(64 * kPrepWaves) void k_gemv_prep(PrepArgs a) {
  __shared__ float s_sum[kPrepWaves][16][17];
  __shared__ __attribute__((aligned(16))) float s_inv[kPrepWaves][kPiece];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int n16 = lane & 15, q = lane >> 4;
  const int m0 = blockIdx.y * 16, j0 = blockIdx.x * 16;
  const int m = m0 + n16 < a.M ? m0 + n16 : a.M - 1;
  const int j = j0 + n16 < a.r ? j0 + n16 : (a.r ? a.r - 1 : 0);
  const uint16_t* x = a.X + (int64_t)m * a.ldx;
  const uint16_t* d = a.down + (int64_t)j * a.K;
  const bool keep = SMOOTH && blockIdx.x == 0 && m0 + n16 < a.M;
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  const int pieces = (int)(a.K / kPiece);
  for (int p = wave; p < pieces; p += kPrepWaves) {
    const int64_t k0 = (int64_t)p * kPiece;
    u32x4_t xv[4], dv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      xv[i] = *reinterpret_cast<const u32x4_t*>(x + k0 + 32 * q + 8 * i);
      if (a.r) dv[i] = *reinterpret_cast<const u32x4_t*>(d + k0 + 32 * q + 8 * i);
    }
    if (SMOOTH) {
      const float2 l = *reinterpret_cast<const float2*>(a.lambda + k0 + 2 * lane);
      __builtin_amdgcn_wave_barrier();
      *reinterpret_cast<float2*>(&s_inv[wave][2 * lane]) = float2{1.0f / l.x, 1.0f / l.y};
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x4_t u = *reinterpret_cast<const f32x4_t*>(&s_inv[wave][32 * q + 8 * i]);
        const f32x4_t v = *reinterpret_cast<const f32x4_t*>(&s_inv[wave][32 * q + 8 * i + 4]);
        xv[i][0] = pack_bf16x2(bf16_lo(xv[i][0]) * u[0], bf16_hi(xv[i][0]) * u[1]);
        xv[i][1] = pack_bf16x2(bf16_lo(xv[i][1]) * u[2], bf16_hi(xv[i][1]) * u[3]);
        xv[i][2] = pack_bf16x2(bf16_lo(xv[i][2]) * v[0], bf16_hi(xv[i][2]) * v[1]);
        xv[i][3] = pack_bf16x2(bf16_lo(xv[i][3]) * v[2], bf16_hi(xv[i][3]) * v[3]);
        if (keep) *reinterpret_cast<u32x4_t*>(a.xhat + (int64_t)m * a.K + k0 + 32 * q + 8 * i) = xv[i];
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    if (a.r) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, xv[i]),
                                                      __builtin_bit_cast(bf16x8_t, dv[i]), acc, 0, 0, 0);
    }
  }
  if (!a.r) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) s_sum[wave][4 * q + i][n16] = acc[i];
  __syncthreads();
  const int om = threadIdx.x >> 4, oj = threadIdx.x & 15;
  if (om >= 16 || m0 + om >= a.M || j0 + oj >= a.r) return;
  float y = 0.0f;
#pragma unroll
  for (int w = 0; w < kPrepWaves; ++w) y += s_sum[w][om][oj];
  a.D[(int64_t)(m0 + om) * a.r + j0 + oj] = y;
}

template <int FMT, int MT>
void launch_tiles(const GemvArgs& a, hipStream_t s) {
  // two tiles of outputs a block where that leaves two blocks a CU: x̂ is read by half as many
  if (a.N >= 32 * 2 * 256)
    k_gemv<FMT, MT, 2><<<(unsigned)((a.N + 31) / 32), 64 * kGemvWaves, 0, s>>>(a);
  else
    k_gemv<FMT, MT, 1><<<(unsigned)((a.N + 15) / 16), 64 * kGemvWaves, 0, s>>>(a);
}

template <int FMT>
void launch_rows(const GemvArgs& a, hipStream_t s) {
  switch ((a.M + 15) / 16) {
    case 1: launch_tiles<FMT, 1>(a, s); break;
    case 2: launch_tiles<FMT, 2>(a, s); break;
    case 3: launch_tiles<FMT, 3>(a, s); break;
    default: launch_tiles<FMT, 4>(a, s); break;
  }
}

int64_t xhat_bytes(int64_t M, int64_t K, bool smooth) { return smooth ? (2 * M * K + 255) / 256 * 256 : 0; }

}  // namespace

int64_t gemv_workspace_bytes(int64_t M, int64_t K, int64_t r, bool smooth) {
  return xhat_bytes(M, K, smooth) + 4 * M * r;
}

hipError_t launch_gemv(int fmt, const uint16_t* X, int64_t M, int64_t K, int64_t ldx,
                       const float* lambda, const uint16_t* down, int64_t r, const uint8_t* codes,
                       const void* scales, const float* g, const uint16_t* up, int64_t N,
                       uint16_t* Y, int64_t ldy, void* workspace, hipStream_t s) {
  uint16_t* xhat = lambda ? (uint16_t*)workspace : nullptr;
  float* D = r ? (float*)((uint8_t*)workspace + xhat_bytes(M, K, lambda != nullptr)) : nullptr;
  if (lambda || r) {
    const PrepArgs p{X, lambda, down, xhat, D, K, ldx, (int)M, (int)r};
    const dim3 grid((unsigned)(r ? (r + 15) / 16 : 1), (unsigned)((M + 15) / 16));
    if (lambda)
      k_gemv_prep<true><<<grid, 64 * kPrepWaves, 0, s>>>(p);
    else
      k_gemv_prep<false><<<grid, 64 * kPrepWaves, 0, s>>>(p);
    if (hipError_t e = hipGetLastError()) return e;
  }
  const GemvArgs a{lambda ? xhat : X, codes, (const uint8_t*)scales, g, D, up, Y, K,
                   lambda ? K : ldx, ldy, (int)M, (int)N, (int)r};
  switch (fmt) {
    case kFmtNv: launch_rows<kFmtNv>(a, s); break;
    case kFmtInt4: launch_rows<kFmtInt4>(a, s); break;
    default: launch_rows<kFmtMx>(a, s); break;
  }
  return hipGetLastError();
}

}  // namespace svdq
