// Rotary positions with several axes.  Pair i of a head belongs to the axis whose section of
// the rotary dimensions holds it, and turns by the angle θ = pos[m, axis(i)] · freq[i]:
//
//   (u, v) -> (u cos θ − v sin θ, u sin θ + v cos θ)        (inverse: −θ)
//
// The angle is formed in fp64 and reduced there to a fraction of a turn, so positions of any
// size keep their full precision; cos and sin of the fraction are fp32.
//
// Memory-bound (4 bytes per element).  A thread owns the eight pairs of one 16-channel unit,
// forms their cos / sin once and applies them to every head of its row.
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

template <bool INTERLEAVED>
__global__ __launch_bounds__(256) void k_rope(RopeArgs a) {
  const int units = a.dim / 16;
  const int slots = (int)blockDim.x / units;      // heads side by side
  const int unit = (int)threadIdx.x % units, slot = (int)threadIdx.x / units;
  if (slot >= slots) return;
  const bool turn = 16 * unit < a.rot;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
    float c[8], s[8];
    if (turn) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = 8 * unit + j;
        int ax = 0;
#pragma unroll
        for (int k = 0; k < 3; ++k) ax += (k + 1 < a.n_axes && i >= a.end[k]) ? 1 : 0;
        const double t = (double)a.pos[row * a.n_axes + ax] * a.freq[i] * 0.15915494309189535;
        const float f = 2.0f * (float)(t - __builtin_rint(t));
        sincospif(f, &s[j], &c[j]);
        if (a.inverse) s[j] = -s[j];
      }
    }
    // first channels of the unit's two pieces of eight
    const int p0 = INTERLEAVED || !turn ? 16 * unit : 8 * unit;
    const int p1 = INTERLEAVED || !turn ? 16 * unit + 8 : 8 * unit + a.rot / 2;
    for (int h = slot; h < a.heads; h += slots) {
      const uint16_t* x = a.X + row * a.ldx + (int64_t)h * a.dim;
      uint16_t* y = a.Y + row * a.ldy + (int64_t)h * a.dim;
      u32x4_t v0 = *reinterpret_cast<const u32x4_t*>(x + p0);
      u32x4_t v1 = *reinterpret_cast<const u32x4_t*>(x + p1);
      if (turn) {
        if (INTERLEAVED) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t w = j < 4 ? v0[j] : v1[j - 4];
            const float u = bf16_lo(w), v = bf16_hi(w);
            const uint32_t o = pack_bf16x2(__builtin_fmaf(u, c[j], -(v * s[j])),
                                           __builtin_fmaf(u, s[j], v * c[j]));
            if (j < 4) v0[j] = o; else v1[j - 4] = o;
          }
        } else {
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
      }
      *reinterpret_cast<u32x4_t*>(y + p0) = v0;
      *reinterpret_cast<u32x4_t*>(y + p1) = v1;
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
  if (interleaved)
    k_rope<true><<<grid, 256, 0, s>>>(a);
  else
    k_rope<false><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace svdq
