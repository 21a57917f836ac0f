// Root-mean-square norm of every query and key head with the rotary positions in the same pass:
//
//   z = x·γ / sqrt(mean x² + eps) over the channels of a head (γ of the queries or of the keys),
//   pairs (u, v) of z -> (u cos θ − v sin θ, u sin θ + v cos θ),  θ = pos[m, axis]·freq[pair]
//
// rounded to bf16 once, at the end; all in fp32 (the angle as in the rotation alone: formed and reduced
// in fp64).  A sum of squares past fp32's range is formed again in fp64.
//
// Memory-bound (4 bytes per element; 31688 rows of 80 heads of 128: 213 to 218 us, 6.0 TB/s): the norm and the rotation one after the other would move 8.  A
// block takes a row, with few rows a part of its heads, with many rows of few heads several: the cos / sin
// of the pairs are formed once, a pair a thread, and kept in LDS, while the first head's loads are on their way.  A thread owns two
// pieces of eight channels, in the same place of every head that it takes, and the 2^n threads of a head
// are neighbours in a wave, so that the sum is a few lane exchanges.
#include "device.h"
#include "launch.h"

namespace svdq {

namespace {

struct QkArgs {
  const uint16_t* X;
  uint16_t* Y;
  const uint16_t* gq;
  const uint16_t* gk;
  const int32_t* pos;
  const double* freq;
  int64_t M, ldx, ldy;
  float eps, inv_dim;
  int heads, q_heads, dim, rot, n_axes;
  int lanes;             // threads of a head: dim / 16, rounded up to a power of two
  int rows;              // of a block (ROWS)
  int end[4];            // pairs up to and including each axis
};

__device__ __forceinline__ float square_sum(u32x4_t v, float s) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    s = __builtin_fmaf(bf16_lo(v[j]), bf16_lo(v[j]), s);
    s = __builtin_fmaf(bf16_hi(v[j]), bf16_hi(v[j]), s);
  }
  return s;
}

// 1 / sqrt(mean + eps) of a head whose squares leave fp32's range: the same in fp64, the root of a
// number brought near 1 by a power of four.
__device__ __noinline__ float far_inverse(u32x4_t v0, u32x4_t v1, int lanes, float inv_dim, float eps) {
  double s = 0.0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t w = j < 4 ? v0[j & 3] : v1[j & 3];
    const double lo = (double)bf16_lo(w), hi = (double)bf16_hi(w);
    s += lo * lo + hi * hi;
  }
  for (int k = 1; k < lanes; k *= 2) s += __shfl_xor(s, k);
  s = s * (double)inv_dim + (double)eps;
  if (!(s < __builtin_inf())) return s != s ? (float)s : 0.0f;
  const int e = __builtin_amdgcn_frexp_exp(s) & ~1;
  return ldexpf(__builtin_amdgcn_rsqf((float)ldexp(s, -e)), -(e / 2));
}

constexpr int kMostPairs = 512;  // of a block's rows

template <bool INTERLEAVED, bool NT, bool ROWS>
__global__ __launch_bounds__(256) void k_qk_norm_rope(QkArgs a) {
  __shared__ __attribute__((aligned(16))) float s_cs[ROWS ? 2 * kMostPairs : 256];  // cos, sin of each pair (of each row)
  const int unit = (int)threadIdx.x % a.lanes, slot = (int)threadIdx.x / a.lanes;
  const int slots = 256 / a.lanes, step = slots * (int)gridDim.y;
  const int h0 = (int)blockIdx.y * slots + slot;
  const bool own = 16 * unit < a.dim;
  // the unit's two pieces of eight channels: in the two halves of the head (interleaved) or of the
  // rotary channels, so that a load covers whole lines
  const bool halves = !INTERLEAVED && 16 * unit < a.rot;
  const int p0 = INTERLEAVED || halves ? 8 * unit : 16 * unit;
  const int p1 = INTERLEAVED ? p0 + a.dim / 2 : halves ? p0 + a.rot / 2 : p0 + 8;
  const bool turn0 = INTERLEAVED ? p0 < a.rot : halves, turn1 = INTERLEAVED ? p1 < a.rot : halves;
  const u32x4_t ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u}, none = {0u, 0u, 0u, 0u};
  u32x4_t g[2][2] = {{ones, ones}, {ones, ones}};
  if (own) {
    if (a.gq) {
      g[0][0] = *reinterpret_cast<const u32x4_t*>(a.gq + p0);
      g[0][1] = *reinterpret_cast<const u32x4_t*>(a.gq + p1);
    }
    if (a.gk) {
      g[1][0] = *reinterpret_cast<const u32x4_t*>(a.gk + p0);
      g[1][1] = *reinterpret_cast<const u32x4_t*>(a.gk + p1);
    }
  }
  const int each = ROWS ? a.rows : 1;
  for (int64_t row = (int64_t)blockIdx.x * each; row < a.M; row += (int64_t)gridDim.x * each) {
    const uint16_t* x = a.X + row * a.ldx;
    uint16_t* y = a.Y + row * a.ldy;
    const int count = ROWS && a.M - row < each ? (int)(a.M - row) : each;
    // a head of one of the rows
    int h = h0, rr = 0;
    auto settle = [&] {
      if (ROWS)
        while (h >= a.heads) {
          h -= a.heads;
          ++rr;
        }
    };
    auto there = [&] { return ROWS ? rr < count : h < a.heads; };
    u32x4_t n0 = none, n1 = none;
    auto load = [&] {
      if (!own || !there()) return;
      const uint16_t* from = x + (ROWS ? rr * a.ldx : 0) + (int64_t)h * a.dim;
      n0 = load_nt(from + p0);
      n1 = load_nt(from + p1);
    };
    settle();
    load();
    const int pairs = a.rot / 2;
    for (int t = threadIdx.x; t < count * pairs; t += 256) {
      const int i = ROWS ? t % pairs : t, r = ROWS ? t / pairs : 0;
      int ax = 0;
#pragma unroll
      for (int k = 0; k < 3; ++k) ax += (k + 1 < a.n_axes && i >= a.end[k]) ? 1 : 0;
      const double turns = (double)a.pos[(row + r) * a.n_axes + ax] * a.freq[i] * 0.15915494309189535;
      const float f = 2.0f * (float)(turns - __builtin_rint(turns));
      float sn, cs;
      sincospif(f, &sn, &cs);
      s_cs[2 * t] = cs;
      s_cs[2 * t + 1] = sn;
    }
    __syncthreads();
    float c[8], s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c[j] = 1.0f;
      s[j] = 0.0f;
    }
    auto angles = [&] {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (own && (k ? turn1 : turn0)) {
          const int first = (INTERLEAVED ? (k ? p1 : p0) / 2 : 8 * unit + 4 * k) + (ROWS ? rr * pairs : 0);
          const f32x4_t u = *reinterpret_cast<const f32x4_t*>(&s_cs[2 * first]);
          const f32x4_t v = *reinterpret_cast<const f32x4_t*>(&s_cs[2 * first + 4]);
          c[4 * k] = u[0]; s[4 * k] = u[1]; c[4 * k + 1] = u[2]; s[4 * k + 1] = u[3];
          c[4 * k + 2] = v[0]; s[4 * k + 2] = v[1]; c[4 * k + 3] = v[2]; s[4 * k + 3] = v[3];
        }
      }
    };
    if (!ROWS) {
      angles();
      if (row + gridDim.x < a.M) __syncthreads();  // the next row's are written to the same place
    }
    while (there()) {
      u32x4_t v0 = n0, v1 = n1;
      if (ROWS) angles();
      uint16_t* const to = y + (ROWS ? rr * a.ldy : 0) + (int64_t)h * a.dim;
      const bool key = h >= a.q_heads;
      h += step;
      settle();
      load();
      float sum = square_sum(v1, square_sum(v0, 0.0f));
      for (int k = 1; k < a.lanes; k *= 2) sum += __shfl_xor(sum, k);
      float inv = __builtin_amdgcn_rsqf(__builtin_fmaf(sum, a.inv_dim, a.eps));
      if (__builtin_amdgcn_ballot_w64(!(sum < 1e37f)) != 0) {
        const float far = far_inverse(v0, v1, a.lanes, a.inv_dim, a.eps);
        if (!(sum < 1e37f)) inv = far;
      }
      const u32x4_t g0 = key ? g[1][0] : g[0][0], g1 = key ? g[1][1] : g[0][1];
      float z[16];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t w = j < 4 ? v0[j & 3] : v1[j & 3], gw = j < 4 ? g0[j & 3] : g1[j & 3];
        z[2 * j] = bf16_lo(w) * inv * bf16_lo(gw);
        z[2 * j + 1] = bf16_hi(w) * inv * bf16_hi(gw);
      }
      if (INTERLEAVED) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float u = z[2 * j], v = z[2 * j + 1];
          const bool turn = j < 4 ? turn0 : turn1;
          const uint32_t o = turn ? pack_bf16x2(__builtin_fmaf(u, c[j], -(v * s[j])),
                                                __builtin_fmaf(u, s[j], v * c[j]))
                                  : pack_bf16x2(u, v);
          if (j < 4) v0[j & 3] = o; else v1[j & 3] = o;
        }
      } else if (halves) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float u0 = z[2 * j], u1 = z[2 * j + 1], w0 = z[8 + 2 * j], w1 = z[9 + 2 * j];
          v0[j] = pack_bf16x2(__builtin_fmaf(u0, c[2 * j], -(w0 * s[2 * j])),
                              __builtin_fmaf(u1, c[2 * j + 1], -(w1 * s[2 * j + 1])));
          v1[j] = pack_bf16x2(__builtin_fmaf(u0, s[2 * j], w0 * c[2 * j]),
                              __builtin_fmaf(u1, s[2 * j + 1], w1 * c[2 * j + 1]));
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v0[j] = pack_bf16x2(z[2 * j], z[2 * j + 1]);
          v1[j] = pack_bf16x2(z[8 + 2 * j], z[9 + 2 * j]);
        }
      }
      if (own) {
        store16<NT>(to + p0, v0);
        store16<NT>(to + p1, v1);
      }
    }
    if (ROWS && row + (int64_t)gridDim.x * each < a.M) __syncthreads();
  }
}

}  // namespace

hipError_t launch_qk_norm_rope(const uint16_t* X, int64_t M, int64_t ldx, int q_heads, int k_heads,
                               int dim, const uint16_t* gamma_q, const uint16_t* gamma_k, float eps,
                               const int32_t* pos, const double* freq, int n_axes,
                               const int* pairs, int interleaved, uint16_t* Y, int64_t ldy,
                               hipStream_t s) {
  QkArgs a{X, Y, gamma_q, gamma_k, pos, freq, M, ldx, ldy, eps, 1.0f / (float)dim,
           q_heads + k_heads, q_heads, dim, 0, n_axes, 1, 1, {0, 0, 0, 0}};
  int n = 0;
  for (int i = 0; i < n_axes; ++i) a.end[i] = n += pairs[i];
  a.rot = 2 * n;
  while (16 * a.lanes < dim) a.lanes *= 2;
  const int slots = 256 / a.lanes, rounds = (a.heads + slots - 1) / slots;
  // few rows: a row's heads in blocks of their own, as long as the blocks fit the card at once
  int parts = 1;
  while (parts < rounds && M * parts < 1024) ++parts;
  // Many rows of few heads: several rows a block, as long as three blocks a CU remain and the rows are at
  // most four rounds of its threads.  Rows of 40 heads of 64: 4001 take 11.7 us, four a block, and 14.1 one a
  // block (eight 12.4), 32000 69 and 84; 32768 of nine heads of 128 34 and 69; 2048 of 18 heads of 64 5.8,
  // two a block, and 7.3 (four 6.4).  With six rounds 31688 of 48 heads of 128 take 142 us for 131.
  while (a.rows < 16 && 2 * a.rows * n <= kMostPairs && M >= 2 * a.rows * 768 &&
         2 * a.rows * a.heads * a.lanes <= 4 * 256)
    a.rows *= 2;
  const int64_t blocks = (M + a.rows - 1) / a.rows;
  const dim3 grid((unsigned)(blocks < (1 << 16) ? blocks : (1 << 16)), (unsigned)parts);
  const bool nt = M * a.heads * dim * 2 > kPastCaches;
  if (a.rows > 1) {
    if (interleaved)
      nt ? k_qk_norm_rope<true, true, true><<<grid, 256, 0, s>>>(a)
         : k_qk_norm_rope<true, false, true><<<grid, 256, 0, s>>>(a);
    else
      nt ? k_qk_norm_rope<false, true, true><<<grid, 256, 0, s>>>(a)
         : k_qk_norm_rope<false, false, true><<<grid, 256, 0, s>>>(a);
  } else if (interleaved) {
    nt ? k_qk_norm_rope<true, true, false><<<grid, 256, 0, s>>>(a)
       : k_qk_norm_rope<true, false, false><<<grid, 256, 0, s>>>(a);
  } else {
    nt ? k_qk_norm_rope<false, true, false><<<grid, 256, 0, s>>>(a)
       : k_qk_norm_rope<false, false, false><<<grid, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace svdq
