// Rotary positions with several axes.  Pair i of a head belongs to the axis whose section of
// the rotary dimensions holds it, and turns by the angle θ = pos[m, axis(i)] · freq[i]:
//
//   (u, v) -> (u cos θ − v sin θ, u sin θ + v cos θ)        (inverse: −θ)
//
// The angle is formed in fp64 and reduced there to a fraction of a turn, so positions of any
// size keep their full precision; cos and sin of the fraction are fp32.
//
// Memory-bound (4 bytes per element).  A block turns one row: the cos / sin of its pairs are
// formed once, a pair a thread, and kept in LDS (formed by every thread for its own pairs they
// held up the loads: 5 % more at 31688 rows of 80 heads of 128, which take 222 us, 5.8 TB/s); a
// thread owns two pieces of eight channels in the same place of every head that it turns.
#include "device.h"
#include "launch.h"

namespace svdq {

namespace {

struct RopeArgs {
  const uint16_t* X;
  uint16_t* Y;
  const int32_t* pos;
  const double* freq;
  int64_t M, ldx, ldy;
  int heads, dim, rot, n_axes;
  int end[4];            // pairs up to and including each axis
  int inverse;
};

template <bool INTERLEAVED, bool NT>
__global__ __launch_bounds__(256) void k_rope(RopeArgs a) {
  __shared__ __attribute__((aligned(16))) float s_cs[256];  // cos, sin of each pair
  const int units = a.dim / 16;
  const int slots = (int)blockDim.x / units;      // heads side by side
  const int unit = (int)threadIdx.x % units, slot = (int)threadIdx.x / units;
  // the unit's two pieces of eight channels: in the two halves of the head (interleaved) or of the
  // rotary channels, so that a load covers whole lines
  const bool halves = !INTERLEAVED && 16 * unit < a.rot;
  const int p0 = INTERLEAVED || halves ? 8 * unit : 16 * unit;
  const int p1 = INTERLEAVED ? p0 + a.dim / 2 : halves ? p0 + a.rot / 2 : p0 + 8;
  const bool turn0 = INTERLEAVED ? p0 < a.rot : halves, turn1 = INTERLEAVED ? p1 < a.rot : halves;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
    const int i = threadIdx.x;
    if (i < a.rot / 2) {
      int ax = 0;
#pragma unroll
      for (int k = 0; k < 3; ++k) ax += (k + 1 < a.n_axes && i >= a.end[k]) ? 1 : 0;
      const double t = (double)a.pos[row * a.n_axes + ax] * a.freq[i] * 0.15915494309189535;
      const float f = 2.0f * (float)(t - __builtin_rint(t));
      float sn, cs;
      sincospif(f, &sn, &cs);
      s_cs[2 * i] = cs;
      s_cs[2 * i + 1] = a.inverse ? -sn : sn;
    }
    __syncthreads();
    float c[8], s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c[j] = 1.0f;
      s[j] = 0.0f;
    }
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      if (g ? turn1 : turn0) {
        const int first = INTERLEAVED ? (g ? p1 : p0) / 2 : 8 * unit + 4 * g;
        const f32x4_t u = *reinterpret_cast<const f32x4_t*>(&s_cs[2 * first]);
        const f32x4_t v = *reinterpret_cast<const f32x4_t*>(&s_cs[2 * first + 4]);
        c[4 * g] = u[0]; s[4 * g] = u[1]; c[4 * g + 1] = u[2]; s[4 * g + 1] = u[3];
        c[4 * g + 2] = v[0]; s[4 * g + 2] = v[1]; c[4 * g + 3] = v[2]; s[4 * g + 3] = v[3];
      }
    }
    if (row + gridDim.x < a.M) __syncthreads();  // the next row's are written to the same place
    if (slot >= slots) continue;
    for (int h = slot; h < a.heads; h += slots) {
      const uint16_t* x = a.X + row * a.ldx + (int64_t)h * a.dim;
      uint16_t* y = a.Y + row * a.ldy + (int64_t)h * a.dim;
      u32x4_t v0 = load_nt(x + p0);
      u32x4_t v1 = load_nt(x + p1);
      if (INTERLEAVED) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (j < 4 ? turn0 : turn1) {
            const uint32_t w = j < 4 ? v0[j] : v1[j - 4];
            const float u = bf16_lo(w), v = bf16_hi(w);
            const uint32_t o = pack_bf16x2(__builtin_fmaf(u, c[j], -(v * s[j])),
                                           __builtin_fmaf(u, s[j], v * c[j]));
            if (j < 4) v0[j] = o; else v1[j - 4] = o;
          }
        }
      } else if (halves) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float u0 = bf16_lo(v0[j]), u1 = bf16_hi(v0[j]);
          const float w0 = bf16_lo(v1[j]), w1 = bf16_hi(v1[j]);
          v0[j] = pack_bf16x2(__builtin_fmaf(u0, c[2 * j], -(w0 * s[2 * j])),
                              __builtin_fmaf(u1, c[2 * j + 1], -(w1 * s[2 * j + 1])));
          v1[j] = pack_bf16x2(__builtin_fmaf(u0, s[2 * j], w0 * c[2 * j]),
                              __builtin_fmaf(u1, s[2 * j + 1], w1 * c[2 * j + 1]));
        }
      }
      store16<NT>(y + p0, v0);
      store16<NT>(y + p1, v1);
    }
  }
}

}  // namespace

hipError_t launch_rope(const uint16_t* X, int64_t M, int64_t ldx, int heads, int dim,
                       const int32_t* pos, const double* freq, int n_axes, const int* pairs,
                       int interleaved, int inverse, uint16_t* Y, int64_t ldy, hipStream_t s) {
  RopeArgs a{X, Y, pos, freq, M, ldx, ldy, heads, dim, 0, n_axes, {0, 0, 0, 0}, inverse};
  int n = 0;
  for (int i = 0; i < n_axes; ++i) a.end[i] = n += pairs[i];
  a.rot = 2 * n;
  const unsigned grid = (unsigned)(M < (1 << 21) ? M : (1 << 21));
  const bool nt = M * heads * dim * 2 > kPastCaches;
  if (interleaved)
    nt ? k_rope<true, true><<<grid, 256, 0, s>>>(a) : k_rope<true, false><<<grid, 256, 0, s>>>(a);
  else
    nt ? k_rope<false, true><<<grid, 256, 0, s>>>(a) : k_rope<false, false><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace svdq
