// Residual addition, root-mean-square norm, smoothing and MXFP8 quantisation of a row, with the
// low-rank down-projection:
//
//   h   = bf16(x + res)                                (h = x without a residual)
//   inv = fl32( 1 / sqrt( mean_k h² + eps ) )          (sum, mean and root in fp64)
//   x̂   = fl32( fl32( fl32(h·inv) · γ ) · fl32(1/λ) )
//   MXFP8 codes and E8M0 scales of x̂ per 32 channels, D = bf16(x̂)·L1 in fp32
//
// The sum of squares is held in fp64: bf16 squares are exact there and their sum nearly always
// is, so inv does not depend on the summation order and the codes, which sit next to rounding
// borders, are the same for every work split.
//
// Memory-bound: 7 bytes per element (x, res in; h, code out).  Each element is read once, held
// in registers between the sum and the quantisation.
#include "device.h"
#include "launch.h"

namespace svdq {

namespace {

struct NormArgs {
  const uint16_t* X;
  const uint16_t* res;   // or NULL
  uint16_t* H;           // with res
  const uint16_t* gamma; // or NULL
  const float* lambda;   // or NULL
  const uint16_t* down;
  uint8_t* codes;
  uint8_t* scales;
  float* D;
  int64_t M, K, ldx, ldr, ldh;
  double eps;
  int r;
};

__device__ __forceinline__ u32x4_t load16(const uint16_t* p) {
  return *reinterpret_cast<const u32x4_t*>(p);
}

// h = bf16(x + res) of eight elements
__device__ __forceinline__ u32x4_t add8(u32x4_t a, u32x4_t b) {
  u32x4_t o;
#pragma unroll
  for (int c = 0; c < 4; ++c)
    o[c] = pack_bf16x2(bf16_lo(a[c]) + bf16_lo(b[c]), bf16_hi(a[c]) + bf16_hi(b[c]));
  return o;
}

__device__ __forceinline__ double sq8(u32x4_t h) {
  double s = 0.0;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const double a = (double)bf16_lo(h[c]), b = (double)bf16_hi(h[c]);
    s = __builtin_fma(a, a, s);
    s = __builtin_fma(b, b, s);
  }
  return s;
}

// x̂ of eight channels from k on
__device__ __forceinline__ void xhat8(const NormArgs& a, u32x4_t h, int64_t k, float inv,
                                      float (&x)[8]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    x[2 * c] = bf16_lo(h[c]) * inv;
    x[2 * c + 1] = bf16_hi(h[c]) * inv;
  }
  if (a.gamma) {
    const u32x4_t g = load16(a.gamma + k);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      x[2 * c] *= bf16_lo(g[c]);
      x[2 * c + 1] *= bf16_hi(g[c]);
    }
  }
  if (a.lambda) {
    const f32x4_t l0 = reinterpret_cast<const f32x4_t*>(a.lambda + k)[0];
    const f32x4_t l1 = reinterpret_cast<const f32x4_t*>(a.lambda + k)[1];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      x[c] *= 1.0f / l0[c];
      x[4 + c] *= 1.0f / l1[c];
    }
  }
}

__device__ __forceinline__ float amax8(const float (&x)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(x[j]));
  return m;
}

__device__ __forceinline__ uint2 codes8(const float (&x)[8], int e) {
  float y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = __builtin_ldexpf(x[j], -e);
  return uint2{e4m3_pack4(y[0], y[1], y[2], y[3]), e4m3_pack4(y[4], y[5], y[6], y[7])};
}

// One row per TPR threads, r == 0.  Thread t of the row owns the 16-byte pieces t, t + TPR, ...;
// four neighbouring threads hold one block of 32.
template <int TPR, int NV>
__global__ __launch_bounds__(256) void k_norm_row(NormArgs a) {
  constexpr int kRows = 256 / TPR;
  __shared__ double s_part[4];
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
  const bool live = row < a.M;
  const int nv = (int)(a.K / 8);
  u32x4_t h[NV];
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = t + TPR * i;
    h[i] = u32x4_t{0u, 0u, 0u, 0u};
    if (live && v < nv) {
      h[i] = load16(a.X + row * a.ldx + 8 * v);
      if (a.res) {
        h[i] = add8(h[i], load16(a.res + row * a.ldr + 8 * v));
        *reinterpret_cast<u32x4_t*>(a.H + row * a.ldh + 8 * v) = h[i];
      }
      s += sq8(h[i]);
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) s += __shfl_xor(s, d);
  if (TPR > 64) {
    if ((threadIdx.x & 63) == 0) s_part[threadIdx.x >> 6] = s;
    __syncthreads();
    s = s_part[0] + s_part[1] + s_part[2] + s_part[3];
  }
  const float inv = (float)(1.0 / sqrt(s / (double)a.K + a.eps));
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = t + TPR * i;
    const bool on = live && v < nv;  // whole blocks: nv is a multiple of 32
    float x[8];
    if (on) xhat8(a, h[i], 8 * v, inv, x);
    float m = on ? amax8(x) : 0.0f;
    m = fmaxf(m, __shfl_xor(m, 1));
    m = fmaxf(m, __shfl_xor(m, 2));
    if (on) {
      const int e = mx_exponent(m, 8);
      *reinterpret_cast<uint2*>(a.codes + row * a.K + 8 * v) = codes8(x, e);
      if ((v & 3) == 0) a.scales[row * (a.K / 32) + v / 4] = (uint8_t)(e + 127);
    }
  }
}

// Sixteen rows per block of eight waves, any K, with the down-projection on MFMA 16x16x32: lane
// (row = lane % 16, q = lane / 16) holds 8 channels of a 32-channel step, which is the A operand
// of the step, so the quantised registers feed the product directly; the four lanes of a row
// hold one MX block.  Wave w takes the 64-channel chunks w, w + 8, ...; the partial D of the
// waves are added in wave order through LDS.
constexpr int kLrWaves = 8;

template <int NT, int NCH>
__global__ __launch_bounds__(64 * kLrWaves) void k_norm_lr(NormArgs a) {
  constexpr int NTc = NT > 0 ? NT : 1;
  __shared__ double s_sum[kLrWaves][16];
  __shared__ float s_d[NT > 0 ? kLrWaves * 16 * NT * 16 : 1];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int rl = lane & 15, q = lane >> 4;
  const int64_t row = (int64_t)blockIdx.x * 16 + rl;
  const bool live = row < a.M;
  const int64_t lrow = live ? row : a.M - 1;
  const int nch = (int)(a.K / 64);
  const uint16_t* xr = a.X + lrow * a.ldx;
  const uint16_t* rr = a.res ? a.res + lrow * a.ldr : nullptr;
  uint16_t* hr = a.res ? a.H + lrow * a.ldh : nullptr;
  u32x4_t keep[2 * NCH];
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = wave + kLrWaves * i;
    if (c < nch) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int64_t k = 64 * c + 32 * u + 8 * q;
        u32x4_t h = load16(xr + k);
        if (rr) h = add8(h, load16(rr + k));
        keep[2 * i + u] = h;
        s += sq8(h);
      }
    }
  }
  // the chunks past the registers: their h is read again below
  for (int c = wave + kLrWaves * NCH; c < nch; c += kLrWaves) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t k = 64 * c + 32 * u + 8 * q;
      u32x4_t h = load16(xr + k);
      if (rr) h = add8(h, load16(rr + k));
      s += sq8(h);
    }
  }
  s += __shfl_xor(s, 16);
  s += __shfl_xor(s, 32);
  if (q == 0) s_sum[wave][rl] = s;
  __syncthreads();
  s = 0.0;
#pragma unroll
  for (int w = 0; w < kLrWaves; ++w) s += s_sum[w][rl];
  const float inv = (float)(1.0 / sqrt(s / (double)a.K + a.eps));

  f32x4_t acc[NTc];
#pragma unroll
  for (int j = 0; j < NTc; ++j) acc[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto step = [&](u32x4_t h, int64_t k) {
    if (hr && live) *reinterpret_cast<u32x4_t*>(hr + k) = h;
    float x[8];
    xhat8(a, h, k, inv, x);
    float m = amax8(x);
    m = fmaxf(m, __shfl_xor(m, 16));
    m = fmaxf(m, __shfl_xor(m, 32));
    const int e = mx_exponent(m, 8);
    if (live) {
      *reinterpret_cast<uint2*>(a.codes + row * a.K + k) = codes8(x, e);
      if (q == 0) a.scales[row * (a.K / 32) + k / 32] = (uint8_t)(e + 127);
    }
    if (NT > 0) {
      u32x4_t av;
#pragma unroll
      for (int c = 0; c < 4; ++c) av[c] = pack_bf16x2(x[2 * c], x[2 * c + 1]);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int n = 16 * j + rl;
        u32x4_t bv = u32x4_t{0u, 0u, 0u, 0u};
        if (n < a.r) bv = load16(a.down + n * a.K + k);
        acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, av),
                                                         __builtin_bit_cast(bf16x8_t, bv), acc[j],
                                                         0, 0, 0);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = wave + kLrWaves * i;
    if (c < nch) {
      step(keep[2 * i], 64 * c + 8 * q);
      step(keep[2 * i + 1], 64 * c + 32 + 8 * q);
    }
  }
  for (int c = wave + kLrWaves * NCH; c < nch; c += kLrWaves) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t k = 64 * c + 32 * u + 8 * q;
      u32x4_t h = load16(xr + k);
      if (rr) h = add8(h, load16(rr + k));
      step(h, k);
    }
  }
  if (NT > 0) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        s_d[(wave * 16 + 4 * q + i) * (NT * 16) + 16 * j + rl] = acc[j][i];
    __syncthreads();
    for (int o = threadIdx.x; o < 16 * a.r; o += 64 * kLrWaves) {
      const int m = o / a.r, n = o % a.r;
      const int64_t rw = (int64_t)blockIdx.x * 16 + m;
      if (rw < a.M) {
        float d = 0.0f;
#pragma unroll
        for (int w = 0; w < kLrWaves; ++w) d += s_d[(w * 16 + m) * (NT * 16) + n];
        a.D[rw * a.r + n] = d;
      }
    }
  }
}

template <int NT>
hipError_t launch_lr(const NormArgs& a, hipStream_t s) {
  const unsigned grid = (unsigned)((a.M + 15) / 16);
  const int64_t per_wave = (a.K / 64 + kLrWaves - 1) / kLrWaves;
  if (per_wave <= 4)
    k_norm_lr<NT, 4><<<grid, 64 * kLrWaves, 0, s>>>(a);
  else
    k_norm_lr<NT, 10><<<grid, 64 * kLrWaves, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_quant(const uint16_t* X, int64_t M, int64_t K, int64_t ldx,
                             const uint16_t* residual, int64_t ldr, uint16_t* H, int64_t ldh,
                             const uint16_t* gamma, float eps, const float* lambda,
                             const uint16_t* down, int64_t r, uint8_t* codes, uint8_t* scales,
                             float* D, hipStream_t s) {
  const NormArgs a{X, residual, H, gamma, lambda, down, codes, scales, D, M, K, ldx, ldr, ldh,
                   (double)eps, (int)r};
  if (r == 0) {
    if (K <= 8192) {
      const unsigned grid = (unsigned)M;
      if (K <= 2048)
        k_norm_row<256, 1><<<grid, 256, 0, s>>>(a);
      else if (K <= 6144)
        k_norm_row<256, 3><<<grid, 256, 0, s>>>(a);
      else
        k_norm_row<256, 4><<<grid, 256, 0, s>>>(a);
      return hipGetLastError();
    }
    return launch_lr<0>(a, s);
  }
  switch ((r + 15) / 16) {
    case 1: return launch_lr<1>(a, s);
    case 2: return launch_lr<2>(a, s);
    case 3: return launch_lr<3>(a, s);
    case 4: return launch_lr<4>(a, s);
    case 5: return launch_lr<5>(a, s);
    case 6: return launch_lr<6>(a, s);
    case 7: return launch_lr<7>(a, s);
    default: return launch_lr<8>(a, s);
  }
}

}  // namespace svdq
