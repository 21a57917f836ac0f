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
// Memory-bound: 7 bytes per element (x, res in; h, code out).  Each element is read once and held
// in registers between the sum and the quantisation (16384 x 5120: 111 us, 5.3 TB/s; a large copy
// reaches 4.9).  D is a kernel of its own over h.
#include "device.h"
#include "launch.h"

namespace svdq {

namespace {

typedef __attribute__((address_space(1))) void gvoid_t;
typedef __attribute__((address_space(3))) void lvoid_t;

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

// One row per block of TPR threads: thread t owns the 16-byte pieces t, t + TPR, ... of the row;
// four neighbouring threads hold one MX block.  With a low-rank branch the row's inv is left in
// the first element of every 4 of its D row for the product kernels below, whose blocks read
// it before they write these elements of D.
template <int TPR, int NV>
__global__ __launch_bounds__(TPR) void k_norm_row(NormArgs a, int64_t first) {
  __shared__ double s_part[TPR / 64];
  const int t = threadIdx.x;
  const int nv = (int)(a.K / 8);
  const int64_t row = first + blockIdx.x;
  u32x4_t h[NV];
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = t + TPR * i;
    h[i] = u32x4_t{0u, 0u, 0u, 0u};
    if (v < nv) {
      h[i] = load_nt(a.X + row * a.ldx + 8 * v);
      if (a.res) {
        h[i] = add8(h[i], load_nt(a.res + row * a.ldr + 8 * v));
        *reinterpret_cast<u32x4_t*>(a.H + row * a.ldh + 8 * v) = h[i];
      }
      s += sq8(h[i]);
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) s += __shfl_xor(s, d);
  if ((threadIdx.x & 63) == 0) s_part[threadIdx.x >> 6] = s;
  __syncthreads();
  s = 0.0;
#pragma unroll
  for (int w = 0; w < TPR / 64; ++w) s += s_part[w];
  const float inv = (float)(1.0 / sqrt(s / (double)a.K + a.eps));
  if (4 * t < a.r) a.D[row * a.r + 4 * t] = inv;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = t + TPR * i;
    const bool on = v < nv;  // whole blocks: nv is a multiple of 32
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

// D = bf16(x̂)·L1 on MFMA 16x16x32, from h and the inv left in D.  Fusing it into the row kernel
// was tried first: a block then holds sixteen rows of h in registers while it reads all of L1
// from L2, one block a CU, 701 us at 31688 x 5120, rank 128; reading h once more costs 2 bytes
// an element and lets 128 rows share each piece of L1.
struct DownArgs {
  const uint16_t* h;
  int64_t ldh;
};

__device__ __forceinline__ void xhat8_lds(u32x4_t h, float inv, const float* g, const float* l,
                                          float (&x)[8]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    x[2 * c] = bf16_lo(h[c]) * inv;
    x[2 * c + 1] = bf16_hi(h[c]) * inv;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = (x[j] * g[j]) * l[j];
}

// Many rows: eight waves, GROUPS of 32 rows times 8 / GROUPS parts of a chunk's channels, 32 each,
// whose sums are added at the end: 128 rows and chunks of 64 channels, or, where that leaves CUs
// idle, 64 rows and chunks of 128 in half as many steps.  Each chunk of h and of L1 goes straight
// into one of three LDS images, two chunks ahead, in whole lines: a CU makes about one request per
// four clocks, and h read by the lanes that need it is twice as many, L1 for 64 rows instead of 128
// again.  A wave of 16 rows on whole chunks would read all of L1 from the images for half as many
// rows (113 us instead of 105 at 31688 x 5120, rank 128; of these 105 about 30 wait for h behind the
// caches, 20 go to the requests, and without any load 54 are left).  The 16-byte pieces of a row lie
// at piece ^ (row % pieces), so that the sixteen rows of a fragment read are on different banks.
// γ and 1/λ follow through registers.  Every step issues the same loads (past the end the last
// chunk's again), so that one count waits for the oldest.  Rows past M and ranks past r repeat the
// last one; what comes of them is not stored.
constexpr int kDownWaves = 8, kChunk = 64, kImages = 3;

template <int NT, int GROUPS>
__global__ __launch_bounds__(64 * kDownWaves, 2) void k_norm_down(NormArgs a, DownArgs d) {
  constexpr int kRows = 32 * GROUPS, kWidth = 32 * kDownWaves / GROUPS;  // a block's, channels of a chunk
  constexpr int kLine = 2 * kWidth, kPieces = kLine / 16;                // of a row: bytes, pieces
  constexpr int kL = NT * 16 * kLine, kH = kRows * kLine;                // bytes of an image
  constexpr int kAll = kL / 1024;                                        // copies of L1
  constexpr int kCopies = (kAll + kDownWaves - 1) / kDownWaves;          // per wave
  static_assert(kH == 2 * kDownWaves * 1024, "two copies of h per wave");
  constexpr int kLoads = kCopies + 4;
  __shared__ __attribute__((aligned(16))) uint8_t s_0[kL + kH], s_1[kL + kH], s_2[kL + kH];
  __shared__ __attribute__((aligned(16))) float s_g[kDownWaves][32], s_i[kDownWaves][32];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, rl = lane & 15, q = lane >> 4;
  const int group = wave % GROUPS, part = wave / GROUPS;
  const int64_t first = (int64_t)blockIdx.x * kRows;
  const int64_t row0 = first + 32 * group;
  const int nch = (int)(a.K / kWidth);
  float inv[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int64_t row = row0 + 16 * t + rl;
    inv[t] = a.D[(row < a.M ? row : a.M - 1) * a.r];
  }
  // without γ or λ something else of K elements is read in their place, and not used
  const int channel = 32 * part + (lane & 31);
  const uint16_t* gp = (a.gamma ? a.gamma : d.h) + channel;
  const float* lp = (a.lambda ? a.lambda : reinterpret_cast<const float*>(a.down)) + channel;
  // copy f of an image: 64 / kPieces rows from there on, kPieces lanes each
  constexpr int kEach = 64 / kPieces;
  auto piece = [&](int f) { return 8 * ((lane ^ (kEach * f + lane / kPieces)) & (kPieces - 1)); };
  const uint16_t *src_l[kCopies], *src_h[2];
  int f_l[kCopies];
#pragma unroll
  for (int i = 0; i < kCopies; ++i) {
    f_l[i] = wave + kDownWaves * i < kAll ? wave + kDownWaves * i : wave % kAll;  // some twice, the same bytes
    const int n = kEach * f_l[i] + lane / kPieces;
    src_l[i] = a.down + (n < a.r ? n : a.r - 1) * a.K + piece(f_l[i]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t m = first + kEach * (2 * wave + i) + lane / kPieces;
    src_h[i] = d.h + (m < a.M ? m : a.M - 1) * d.ldh + piece(2 * wave + i);
  }
  uint16_t g[kImages];
  float l[kImages];
  // part p of a chunk's loads: two pieces of h, kCopies of L1, the factors
  constexpr int kParts = kCopies + 3;
  auto load = [&](int p, int c, int slot, uint8_t* img) {
    const int64_t k = (int64_t)(c < nch ? c : nch - 1) * kWidth;
    if (p < 2) {
      __builtin_amdgcn_global_load_lds((gvoid_t*)(src_h[p] + k),
                                       (lvoid_t*)(img + kL + (2 * wave + p) * 1024), 16, 0, 0);
    } else if (p < 2 + kCopies) {
      __builtin_amdgcn_global_load_lds((gvoid_t*)(src_l[p - 2] + k),
                                       (lvoid_t*)(img + f_l[p - 2] * 1024), 16, 0, 0);
    } else {
      g[slot] = gp[k];
      l[slot] = lp[k];
    }
  };
  f32x4_t acc[2][NT];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[t][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int at = ((4 * part + q) ^ (rl & (kPieces - 1))) * 16;
  auto step = [&](int c, int slot, const uint8_t* img, uint8_t* free_img) {
    wait_vmcnt<kLoads>();  // chunk c is here; c + 1 may be on its way
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);  // no use of the chunk moves up in front of its wait
    // the wave's own copy of its channels' factors (both halves of the wave write the same)
    s_g[wave][lane & 31] = a.gamma ? bf16_to_f32(g[slot]) : 1.0f;
    s_i[wave][lane & 31] = a.lambda ? 1.0f / l[slot] : 1.0f;
    u32x4_t bv[NT], hv[2], av[2];
#pragma unroll
    for (int t = 0; t < 2; ++t)
      hv[t] = *reinterpret_cast<const u32x4_t*>(img + kL + (32 * group + 16 * t + rl) * kLine + at);
#pragma unroll
    for (int j = 0; j < NT; ++j)
      bv[j] = *reinterpret_cast<const u32x4_t*>(img + (16 * j + rl) * kLine + at);
    float gg[8], ll[8];
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      *reinterpret_cast<f32x4_t*>(gg + j) =
          *reinterpret_cast<const f32x4_t*>(&s_g[wave][8 * q + j]);
      *reinterpret_cast<f32x4_t*>(ll + j) =
          *reinterpret_cast<const f32x4_t*>(&s_i[wave][8 * q + j]);
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      float x[8];
      xhat8_lds(hv[t], c < nch ? inv[t] : 0.0f, gg, ll, x);
#pragma unroll
      for (int j = 0; j < 4; ++j) av[t][j] = pack_bf16x2(x[2 * j], x[2 * j + 1]);
    }
    // the loads of chunk c + 2 are issued between the matrix instructions: a wave waits there for
    // its turn at the one address unit
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
        acc[t][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, av[t]),
                                                            __builtin_bit_cast(bf16x8_t, bv[j]),
                                                            acc[t][j], 0, 0, 0);
#pragma unroll
      for (int p = j * kParts / NT; p < (j + 1) * kParts / NT; ++p)
        load(p, c + 2, (slot + 2) % kImages, free_img);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
#pragma unroll
  for (int p = 0; p < kParts; ++p) load(p, 0, 0, s_0);
#pragma unroll
  for (int p = 0; p < kParts; ++p) load(p, 1, 1, s_1);
  // (steps past the end add zeros: a branch around them would make the compiler drain the loads
  // where the paths meet)
  for (int c = 0; c < nch; c += 3) {
    step(c, 0, s_0, s_2);
    step(c + 1, 1, s_1, s_0);
    step(c + 2, 2, s_2, s_1);
  }
  wait_vmcnt<0>();  // no copy is left in flight when the images are taken for the sums
  __syncthreads();
  // (2·NT KB for each group and part but the first, two of them in an image)
  static_assert(2 * 2 * NT * 1024 <= kL + kH, "two groups' sums fit an image");
  auto sums = [&](int p) {
    const int n = (p - 1) * GROUPS + group;
    return reinterpret_cast<f32x4_t*>((n < 2 ? s_0 : n < 4 ? s_1 : s_2) + (n & 1) * 2 * NT * 1024);
  };
  if (part > 0) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int j = 0; j < NT; ++j) sums(part)[(t * NT + j) * 64 + lane] = acc[t][j];
  }
  __syncthreads();
  if (part > 0) return;
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int p = 1; p < kDownWaves / GROUPS; ++p) acc[t][j] += sums(p)[(t * NT + j) * 64 + lane];
      const int n = 16 * j + rl;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t m = row0 + 16 * t + 4 * q + i;
        if (m < a.M && n < a.r) a.D[m * a.r + n] = acc[t][j][i];
      }
    }
}

// Few rows: a block for each 16 rows and RT ranks, sixteen waves that take alternate 64-channel
// chunks with the loads of four chunks under way at once, the partial sums added in wave order
// (one block for all ranks, eight waves and a chunk at a time took 24 us for one row of 5120 at
// rank 32 instead of 13).  A CU fetches L1 in half lines here, about one in four clocks, so
// where 16 ranks a block leave CUs idle a block takes 4 of them (the other columns of its matrix
// instructions repeat the last one and are not stored).
constexpr int kFewWaves = 16, kFewBatch = 4;

template <int RT>
__global__ __launch_bounds__(64 * kFewWaves) void k_norm_down_few(NormArgs a, DownArgs d) {
  __shared__ float s_d[kFewWaves][16][16];
  __shared__ __attribute__((aligned(16))) float s_g[kFewWaves][kChunk], s_i[kFewWaves][kChunk];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, rl = lane & 15, q = lane >> 4;
  const int64_t row = (int64_t)blockIdx.x * 16 + rl, lrow = row < a.M ? row : a.M - 1;
  const int n0 = RT * blockIdx.y, nr = a.r - n0 < RT ? a.r - n0 : RT;
  const float inv = a.D[lrow * a.r + n0];
  const uint16_t* hr = d.h + lrow * d.ldh + 8 * q;
  const uint16_t* dr = a.down + (n0 + (rl < nr ? rl : nr - 1)) * a.K + 8 * q;
  const int nch = (int)(a.K / kChunk);
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  for (int c0 = wave; c0 < nch; c0 += kFewWaves * kFewBatch) {
    u32x4_t h[kFewBatch][2], l1[kFewBatch][2];
    float g[kFewBatch], l[kFewBatch];
#pragma unroll
    for (int i = 0; i < kFewBatch; ++i) {
      const int c = c0 + kFewWaves * i;
      if (c < nch) {
        const int64_t k = (int64_t)c * kChunk;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          h[i][s] = load16(hr + k + 32 * s);
          l1[i][s] = load16(dr + k + 32 * s);
        }
        g[i] = a.gamma ? bf16_to_f32(a.gamma[k + lane]) : 1.0f;
        l[i] = a.lambda ? a.lambda[k + lane] : 1.0f;
      }
    }
#pragma unroll
    for (int i = 0; i < kFewBatch; ++i) {
      if (c0 + kFewWaves * i < nch) {
        s_g[wave][lane] = g[i];  // the wave's own: LDS accesses of a wave keep their order
        s_i[wave][lane] = 1.0f / l[i];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          float x[8], gg[8], ll[8];
#pragma unroll
          for (int j = 0; j < 8; j += 4) {
            *reinterpret_cast<f32x4_t*>(gg + j) =
                *reinterpret_cast<const f32x4_t*>(&s_g[wave][32 * s + 8 * q + j]);
            *reinterpret_cast<f32x4_t*>(ll + j) =
                *reinterpret_cast<const f32x4_t*>(&s_i[wave][32 * s + 8 * q + j]);
          }
          xhat8_lds(h[i][s], inv, gg, ll, x);
          u32x4_t av;
#pragma unroll
          for (int j = 0; j < 4; ++j) av[j] = pack_bf16x2(x[2 * j], x[2 * j + 1]);
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, av),
                                                        __builtin_bit_cast(bf16x8_t, l1[i][s]), acc,
                                                        0, 0, 0);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) s_d[wave][4 * q + i][rl] = acc[i];
  __syncthreads();
  const int m = threadIdx.x >> 4, n = threadIdx.x & 15;
  const int64_t rw = (int64_t)blockIdx.x * 16 + m;
  if (m < 16 && n < nr && rw < a.M) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) v += s_d[w][m][n];
    a.D[rw * a.r + n0 + n] = v;
  }
}

// Which of the three (K = 5120, no residual, whole call in us; few, many with 64 rows, many with 128):
//   rank 128  M 1024: 34, 57, 73   2048: 61, 62, 78   8192: 234, 88, 103   16384: -, 131, 143
//                  20480: -, 197, 165   31688: -, 252, 231
//   rank 32   M 4096: 49, 50, 74   8192: 93, 68, 91   16384: 180, 112, 131   20480: -, 156, 154
// The kernel for few rows takes about as long as it has blocks of 16 rows and 16 ranks; the other
// one a fixed time while its blocks fit the 256 CUs, longer with more ranks, so its larger blocks
// come in where the smaller ones need a second round.
template <int NT>
void launch_down(const NormArgs& a, hipStream_t s) {
  const DownArgs d = a.res ? DownArgs{a.H, a.ldh} : DownArgs{a.X, a.ldx};
  const int64_t rows = (a.M + 15) / 16;
  if (rows * NT < 256)
    k_norm_down_few<4><<<dim3((unsigned)rows, (unsigned)a.r / 4), 64 * kFewWaves, 0, s>>>(a, d);
  else if (rows * NT <= 448 + 72 * NT)
    k_norm_down_few<16><<<dim3((unsigned)rows, NT), 64 * kFewWaves, 0, s>>>(a, d);
  else if (a.M <= 64 * 256)
    k_norm_down<NT, 2><<<(unsigned)((a.M + 63) / 64), 64 * kDownWaves, 0, s>>>(a, d);
  else
    k_norm_down<NT, 4><<<(unsigned)((a.M + 127) / 128), 64 * kDownWaves, 0, s>>>(a, d);
}

}  // namespace

hipError_t launch_norm_quant(const uint16_t* X, int64_t M, int64_t K, int64_t ldx,
                             const uint16_t* residual, int64_t ldr, uint16_t* H, int64_t ldh,
                             const uint16_t* gamma, float eps, const float* lambda,
                             const uint16_t* down, int64_t r, uint8_t* codes, uint8_t* scales,
                             float* D, hipStream_t s) {
  const NormArgs a{X, residual, H, gamma, lambda, down, codes, scales, D, M, K, ldx, ldr, ldh,
                   (double)eps, (int)r};
  // a launch has fewer than 2^32 threads
  for (int64_t first = 0; first < M; first += 1 << 21) {
    const unsigned grid = (unsigned)(M - first < (1 << 21) ? M - first : (1 << 21));
    if (K <= 2048)
      k_norm_row<256, 1><<<grid, 256, 0, s>>>(a, first);
    else if (K <= 6144)
      k_norm_row<256, 3><<<grid, 256, 0, s>>>(a, first);
    else if (K <= 8192)
      k_norm_row<256, 4><<<grid, 256, 0, s>>>(a, first);
    else
      k_norm_row<1024, 4><<<grid, 1024, 0, s>>>(a, first);
  }
  if (hipError_t e = hipGetLastError()) return e;
  switch ((r + 15) / 16) {
    case 0: break;
    case 1: launch_down<1>(a, s); break;
    case 2: launch_down<2>(a, s); break;
    case 3: launch_down<3>(a, s); break;
    case 4: launch_down<4>(a, s); break;
    case 5: launch_down<5>(a, s); break;
    case 6: launch_down<6>(a, s); break;
    case 7: launch_down<7>(a, s); break;
    default: launch_down<8>(a, s); break;
  }
  return hipGetLastError();
}

}  // namespace svdq
