// The layer's product for a few rows with 16-bit activations (no activation quantisation):
//
//   Y[m, n] = bf16( Σ_k x̂[m, k]·w[n, k] + Σ_j D[m, j]·up[n, j] ),  x̂ = bf16(x·fl32(1/λ)),
//   D = x̂·downᵀ,  w = the weight that its codes and scales stand for
//
// Bound by the weight's bytes, and for single rows by the latency of the loads.  The product runs on the
// 16x16x32 MFMA with the rows padded to 16: the codes are widened once for all rows, which for one row costs
// little more than a product a lane and leaves the same kernel for 64.  Every product is exact in the fp32
// sum.  MXFP4: an E2M1 code times its power of two is a bf16, like x̂.  NVFP4 and int4 are widened to fp16
// in packed arithmetic (half the instructions of the way through fp32, which bounded the kernel): an E2M1
// code times an E4M3 scale has six significant bits and lies in fp16's range, int4 codes go without their
// scale, which multiplies the sum of a group's 64 products.  x̂ then is an fp16 too: its rows are
// scaled by a power of two for every 256 channels so that the largest lies below 2^15, and the sums of
// those are scaled back; what is 2^29 times smaller than the largest of its 256 loses bits of its eight.  NVFP4's
// tensor scale g is about 2^-16 of the weight, and sums without it would pass fp32's range long before the result:
// they are scaled back with g's power of two, exactly, and the join multiplies by the rest of g, in [1, 2).
//
// Measured, here and below (both kernels, in graphs over 600 MB of weights in turn, which no cache holds: a
// token's step reads each weight once): one row of 5120x5120 NVFP4, rank 32, 14.4 us, five of 5120x13824 MXFP4,
// rank 128, 19.5 (without it 14.8, 2.5 TB/s), 32 of 13824x5120 int4, rank 32, 28.6; two rows of 13824x13824 NVFP4
// 33 us, 3.2 TB/s.  The 32 rows are bound by the vector instructions (widening the codes, forming x̂ in every
// block; 0.40 of the SIMDs' time) and by the loads that these wait for, a third of the waves' time: with two tiles
// of rows one chunk is on its way while the one before it is computed.
//
// Two kernels.  The first splits N among waves and K among blocks, so that even one row's weight is
// asked for all at once, and writes fp32 sums of each part of K; x̂ is formed on the way into LDS, a part
// of it for each block.  One more block for each part does the same with the down factor in the
// weight's place.  The second adds the parts in their order and the up factor's product.  (The parts do not
// depend on the rows: a row's result is the same bits alone and among others.)
#include <type_traits>

#include "device.h"
#include "kv_layout.h"
#include "launch.h"

namespace svdq {

namespace {

constexpr int kFmtNv = 0, kFmtInt4 = 1, kFmtMx = 2;  // svdq_format
constexpr int kPiece = 128;                          // channels of a lane group's load
constexpr int kWaves = 8;

// Dwords of a weight row's scales of one piece: eight E4M3, two fp16 or four E8M0.
constexpr int scale_words(int fmt) { return fmt == kFmtNv ? 2 : 1; }

// A buffer that the whole wave shares (the compiler loses sight of that and would loop over the lanes).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t shared_rsrc(const void* base, uint32_t bytes) {
  const uint64_t b = (uint64_t)base;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)b), hi = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32));
  return raw_rsrc((const void*)((uint64_t)hi << 32 | lo), __builtin_amdgcn_readfirstlane(bytes));
}

// Buffer loads: an offset of kNoLoad gives zeros without a request, so that every step issues the same
// loads and the compiler's wait counts stay exact.
__device__ __forceinline__ u32x4_t load16(__amdgpu_buffer_rsrc_t r, uint32_t at, uint32_t uniform) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, at, uniform, 0);
}

// Of a lane group q (16 lanes) the dwords 2 and 3 of its first half (q < 2) change places with the dwords 0 and
// 1 of the second: dwords 0 and 1 are then of the piece's first 64 channels in every lane, an int4 group.
__device__ __forceinline__ void split_groups(u32x4_t& w) {
  const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  w = u32x4_t{a[0], b[0], a[1], b[1]};
}

// Channel of a piece from which on a lane has eight in dword i.
template <int FMT>
__device__ __forceinline__ int channel_of(int q, int i) {
  if (FMT != kFmtInt4) return 32 * q + 8 * i;
  // dword i of group i / 2: the lane's own (i / 2 == q / 2) or its partner's
  return 64 * (i >> 1) + 32 * (q & 1) + 16 * (q >> 1) + 8 * (i & 1);
}

// The weight's two widened forms, by the bits of an operand.
__device__ __forceinline__ f32x4_t product(u32x4_t x, u32x4_t w, f32x4_t sum, std::false_type) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, x), __builtin_bit_cast(bf16x8_t, w), sum, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t product(u32x4_t x, u32x4_t w, f32x4_t sum, std::true_type) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, x), __builtin_bit_cast(f16x8_t, w), sum, 0, 0, 0);
}

__device__ __forceinline__ uint32_t bits_of(f16x2_t v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ uint32_t bits_of(bf16x2_t v) { return __builtin_bit_cast(uint32_t, v); }

// Eight codes of a weight row as an operand.  MXFP4 and NVFP4: times the block's scale (`s`: a power of two,
// an fp16 twice).  int4: without a scale, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ u32x4_t widen_mx(uint32_t w, float s) {
  return u32x4_t{bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0)),
                 bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1)),
                 bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2)),
                 bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3))};
}
__device__ __forceinline__ u32x4_t widen_int4(uint32_t w) {
  const uint32_t u = w ^ 0x88888888u;   // code + 8; as bits of an fp16: 0x6400 + u = 1024 + u, 0x5400 + 16 u = 64 + u
  const f16x2_t low = {(_Float16)-1032.0f, (_Float16)-1032.0f}, high = {(_Float16)-72.0f, (_Float16)-72.0f};
  u32x4_t r;
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    const uint32_t v = u >> (4 * j);
    r[j] = bits_of(__builtin_bit_cast(f16x2_t, (v & 0x000F000Fu) | 0x64006400u) + low);
    r[j + 1] = bits_of(__builtin_bit_cast(f16x2_t, (v & 0x00F000F0u) | 0x54005400u) + high);
  }
  return r;
}

struct GemvArgs {
  const uint16_t* X;       // [M, K] bf16
  const float* lambda;     // or NULL
  const uint8_t* codes;
  const uint8_t* scales;
  const float* g;          // or NULL
  const uint16_t* down;    // [r, K]
  const uint16_t* up;      // [N, r]
  float* sums;             // [parts, quads of rows, N, 4]
  float* D;                // [down_parts, M, r]
  uint16_t* Y;
  int64_t K, ldx, ldy;
  int M, N, r;
  int groups, parts, each; // blocks of outputs, parts of K, pieces of one
  int down_parts, down_each;
};

// The power of two of the tensor's scale (any number for zero, infinity and NaN, which stay what they are).
__device__ __forceinline__ int exponent_of(float g) { return __builtin_amdgcn_frexp_expf(g) - 1; }

// Bytes of a row of x̂ in LDS, CH pieces: rows start in banks of their own.
template <int CH>
constexpr int kRowBytes = CH * kPiece * 2 + 16;

// x̂ of a chunk of CH pieces on its way into LDS: a thread brings eight channels of every kStep-th row.
// NVFP4 and int4: as fp16 with a power of two for each row and pair of pieces, of which the exponent of the way
// back goes to s_back (with g's, g_exp); int4's order of the channels.
template <int FMT, int MT, int CH, int SETS, bool SMOOTH>
struct Activations {
  static constexpr bool kHalf = FMT == kFmtNv || FMT == kFmtInt4;
  static constexpr int kCols = 16 * CH, kStep = 64 * kWaves / kCols, kRows = 16 * MT / kStep;
  static_assert(kRows >= 1, "a chunk of 16 rows takes every thread");
  static_assert(kCols == 64 || kCols == 32, "a row's threads are a wave or half of one");
  __amdgpu_buffer_rsrc_t rx, rl;
  int col, row0, last;
  u32x4_t xr[SETS][kRows], lam[SETS][2];

  __device__ __forceinline__ Activations(const GemvArgs& a, int last)
      : rx(raw_rsrc(a.X, (uint32_t)(2 * ((a.M - 1) * a.ldx + a.K)))),
        rl(raw_rsrc(a.lambda, SMOOTH ? (uint32_t)(4 * a.K) : 0u)),
        col(threadIdx.x % kCols), row0(threadIdx.x / kCols), last(last) {}
  __device__ __forceinline__ void load(const GemvArgs& a, int p, int set) {
    const bool there = p * kPiece + 8 * col < last * kPiece;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int m = row0 + kStep * i;
      xr[set][i] = load16(rx, there && m < a.M ? (uint32_t)(m * (int)(2 * a.ldx) + 16 * col) : kNoLoad,
                     (uint32_t)p * (2 * kPiece));
    }
    if (SMOOTH) {
      lam[set][0] = load16(rl, there ? 32 * col : kNoLoad, (uint32_t)p * (4 * kPiece));
      lam[set][1] = load16(rl, there ? 32 * col + 16 : kNoLoad, (uint32_t)p * (4 * kPiece));
    }
  }
  // The largest magnitude (its bf16 bits) of the 32 lanes' channels, a pair of pieces of a row.
  static __device__ __forceinline__ uint32_t row_max(u32x4_t v) {
    uint32_t m = max_bf16x2(max_bf16x2(v[0] & 0x7FFF7FFFu, v[1] & 0x7FFF7FFFu),
                            max_bf16x2(v[2] & 0x7FFF7FFFu, v[3] & 0x7FFF7FFFu));
    m = max_bf16x2(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x121, 0xF, 0xF, true));  // row_ror:1, 2, 4, 8
    m = max_bf16x2(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x122, 0xF, 0xF, true));
    m = max_bf16x2(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x124, 0xF, 0xF, true));
    m = max_bf16x2(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x128, 0xF, 0xF, true));
    const auto a = __builtin_amdgcn_permlane16_swap(m, m, false, false);
    m = max_bf16x2(a[0], a[1]);
    return max_bf16x2(m, m >> 16) & 0xFFFFu;
  }
  // (rows past M and channels past the last piece become zeros)
  __device__ __forceinline__ void store(int p, int set, uint8_t* buf, int* s_back, int g_exp) {
    float inv[8];
    if (SMOOTH) {
      const bool there = p * kPiece + 8 * col < last * kPiece;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        inv[j] = there ? 1.0f / __uint_as_float(lam[set][j >> 2][j & 3]) : 0.0f;
        asm volatile("" : "+v"(inv[j]));  // one division after the other: side by side they take too many registers
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      u32x4_t v = xr[set][i];
      if (SMOOTH) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[j] = pack_bf16x2(bf16_lo(v[j]) * inv[2 * j], bf16_hi(v[j]) * inv[2 * j + 1]);
      }
      if constexpr (kHalf) {
        // 2^(14 − floor(log2 max)); an infinity or NaN, which makes the row one, leaves the others as they are
        const uint32_t top = row_max(v);
        const int f = 268 - (int)(top >> 7);
        const uint32_t field = top >= kInfBits ? 127u : (uint32_t)(f > 253 ? 253 : f);
        const float up = __uint_as_float(field << 23);
        if (col % 32 == 0) s_back[col / 32 * (16 * MT) + row0 + kStep * i] = 127 - (int)field + g_exp;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const auto h = __builtin_amdgcn_cvt_pkrtz(bf16_lo(v[j]) * up, bf16_hi(v[j]) * up);
          v[j] = __builtin_bit_cast(uint32_t, h);
        }
      }
      if constexpr (FMT == kFmtInt4)
        v = u32x4_t{__builtin_amdgcn_perm(v[2], v[0], 0x05040100u), __builtin_amdgcn_perm(v[2], v[0], 0x07060302u),
                    __builtin_amdgcn_perm(v[3], v[1], 0x05040100u), __builtin_amdgcn_perm(v[3], v[1], 0x07060302u)};
      *reinterpret_cast<u32x4_t*>(buf + (row0 + kStep * i) * kRowBytes<CH> + 16 * col) = v;
    }
  }
};

// All waves are past what stands before in LDS; loads from memory stay under way.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// A wave's 16 outputs n0 .., pieces [first, last).  x̂ goes through LDS a chunk of CH pieces at a time, in
// two buffers; AHEAD pieces of codes are under way in registers.  Loads come back in order, so what is
// waited for first is asked for first, and a register is loaded again when its last use is over, never
// while a copy of it lives: a copy of a load under way at the loop's end would wait for it.
//
// Four lanes side by side load 64 bytes of a weight row, and the operand's lane order comes from lane
// exchanges: the L1 takes a load four lanes at a time, and with neighbouring lanes on rows of their own,
// as the operand has them, each load took 50 cycles of it and those of the scales 90 (the kernel's
// bound).  The scales of a row's chunk come in one lane and go to the others through LDS.
template <int FMT, int MT, int CH, int AHEAD, bool SMOOTH>
__device__ __forceinline__ void outputs(const GemvArgs& a, int n0, int first, int last, uint8_t* s_x,
                                        int* s_back, uint8_t* s_scale, f32x4_t (&total)[MT]) {
  constexpr int kSets = AHEAD / CH, kScaleWords = scale_words(FMT), kWords = CH * kScaleWords;
  constexpr int kLanes = kWords > 4 ? kWords / 4 : 1;   // of a row's scales, 16 bytes each
  constexpr bool kHalf = FMT != kFmtMx;
  const std::integral_constant<bool, kHalf> half{};
  const int lane = threadIdx.x & 63, n16 = lane & 15, q = lane >> 4;
  // the wave's rows of the weight: at most 32 MB of codes
  const int rows = a.N - n0 < 16 ? (a.N - n0 > 0 ? a.N - n0 : 0) : 16;
  const uint32_t pitch = (uint32_t)(a.K / 2), spitch = (uint32_t)(a.K / kPiece * 4 * kScaleWords);
  const __amdgpu_buffer_rsrc_t rc = shared_rsrc(a.codes + (int64_t)(rows ? n0 : 0) * pitch, rows * pitch);
  const __amdgpu_buffer_rsrc_t rs = shared_rsrc(a.scales + (int64_t)(rows ? n0 : 0) * spitch, rows * spitch);
  const uint32_t at = (lane >> 2) < rows ? (lane >> 2) * pitch + 16 * (lane & 3) : kNoLoad;
  const uint32_t sat = lane / kLanes < rows ? (lane / kLanes) * spitch + 16 * (lane % kLanes) : kNoLoad;
  const int from = 4 * (4 * n16 + q);   // the lane that loaded this one's codes, for the exchange

  u32x4_t w[AHEAD], sw[kSets];
  auto load_w = [&](int p, int slot) {
    w[slot] = load16(rc, p < last ? at : kNoLoad, (uint32_t)p * (kPiece / 2));
    __builtin_amdgcn_sched_barrier(0);
  };
  auto load_s = [&](int p, int set) {
    // (the place in the lane's offset, which is checked: the last row's last chunk may be a part of one)
    sw[set] = load16(rs, p < last && lane < 16 * kLanes ? sat + (uint32_t)p * (4 * kScaleWords) : kNoLoad, 0);
    __builtin_amdgcn_sched_barrier(0);
  };
  Activations<FMT, MT, CH, kSets, SMOOTH> x(a, last);
  // the rows of x̂ that go with the lane (past M: the last one's, not stored)
  int x_off[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
    x_off[m] = (16 * m + n16 < a.M ? 16 * m + n16 : a.M - 1) * kRowBytes<CH> + 2 * channel_of<FMT>(q, 0);

#pragma unroll
  for (int k = 0; k < kSets; ++k) {
    x.load(a, first + k * CH, k);
    __builtin_amdgcn_sched_barrier(0);
    load_s(first + k * CH, k);
#pragma unroll
    for (int d = 0; d < CH; ++d) load_w(first + k * CH + d, k * CH + d);
  }
  // (behind the loads, which would wait for it)
  const int g_exp = FMT == kFmtNv ? __builtin_amdgcn_readfirstlane(exponent_of(a.g[0])) : 0;
  const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
  f32x4_t acc[MT];   // of a pair of pieces
  auto chunk = [&](int p0, int set, int buffer) {
    uint8_t* buf = s_x + buffer * (16 * MT * kRowBytes<CH>);
    int* back = s_back + buffer * (CH / 2 * 16 * MT);
    x.store(p0, set, buf, back, g_exp);
    if (kScaleWords == 1 && p0 + 2 >= last) sw[set][2] = sw[set][3] = 0u;  // (another row's, or nothing)
    if (lane < 16 * kLanes) *reinterpret_cast<u32x4_t*>(s_scale + 16 * lane) = sw[set];
    __builtin_amdgcn_sched_barrier(0);
    x.load(a, p0 + AHEAD, set);
    __builtin_amdgcn_sched_barrier(0);
    load_s(p0 + AHEAD, set);
    lds_barrier();   // (the other buffer was read before it)
    uint32_t sc[kWords];
#pragma unroll
    for (int i = 0; i < kWords; i += 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(s_scale + n16 * (16 * kLanes) + 4 * i);
      sc[i] = v.x;
      sc[i + 1] = v.y;
    }
#pragma unroll
    for (int d = 0; d < CH; ++d) {  // (pieces past the last are zeros)
      if (d % 2 == 0)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[m] = zero;
      u32x4_t now;
#pragma unroll
      for (int j = 0; j < 4; ++j) now[j] = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)w[set * CH + d][j]);
      __builtin_amdgcn_sched_barrier(0);
      load_w(p0 + AHEAD + d, set * CH + d);
      const uint8_t* xp = buf + d * (kPiece * 2);
      auto x_of = [&](int m, int i) {
        return *reinterpret_cast<const u32x4_t*>(xp + x_off[m] + 2 * (FMT == kFmtInt4 ? 64 * (i >> 1) + 8 * (i & 1) : 8 * i));
      };
      if constexpr (FMT == kFmtInt4) {
        split_groups(now);
#pragma unroll
        for (int gr = 0; gr < 2; ++gr) {
          const u32x4_t w0 = widen_int4(now[2 * gr]), w1 = widen_int4(now[2 * gr + 1]);
          const float s = (float)__builtin_bit_cast(_Float16, (uint16_t)(sc[d] >> (16 * gr)));
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const f32x4_t sum = product(x_of(m, 2 * gr + 1), w1, product(x_of(m, 2 * gr), w0, zero, half), half);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[m][j] = __builtin_fmaf(s, sum[j], acc[m][j]);
          }
        }
      } else {
        float s_mx = 0.f;
        f16x2_t s_nv = {};
        if constexpr (FMT == kFmtMx) {
          s_mx = __uint_as_float((sc[d] >> (8 * q)) << 23);  // (the conversion reads the exponent field alone)
        } else {
          const uint32_t lo = sc[2 * d], hi = sc[2 * d + 1];
          s_nv = e4m3x2_to_f16x2((q & 2 ? hi : lo) >> (16 * (q & 1)));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          u32x4_t v;
          if constexpr (FMT == kFmtMx) v = widen_mx(now[i], s_mx);
          else v = __builtin_bit_cast(u32x4_t, dequant8(now[i], f16x2_t{s_nv[i >> 1], s_nv[i >> 1]}));
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            acc[m] = product(x_of(m, i), v, acc[m], half);
          }
        }
      }
      if (d % 2 == 1)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          if constexpr (kHalf) {
            const u32x4_t e = *reinterpret_cast<const u32x4_t*>(back + (d / 2) * (16 * MT) + 16 * m + 4 * q);
#pragma unroll
            for (int j = 0; j < 4; ++j) total[m][j] += __builtin_amdgcn_ldexpf(acc[m][j], (int)e[j]);
          } else {
            total[m] += acc[m];
          }
        }
    }
  };
  int buffer = 0;
  for (int p0 = first; p0 < last; p0 += AHEAD) {
#pragma unroll
    for (int k = 0; k < kSets; ++k) {
      if (p0 + k * CH >= last) break;
      chunk(p0 + k * CH, k, buffer);
      buffer ^= 1;
    }
  }
}

// A part of D: 16 ranks a wave, and the block's pieces among the waves that have the same ranks (`turns` of
// them); their sums are joined through LDS.
template <int MT, int CH, bool SMOOTH>
__device__ __forceinline__ void down_part(const GemvArgs& a, int part, uint8_t* s_x) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int n16 = lane & 15, q = lane >> 4, pieces = (int)(a.K / kPiece);
  const int first = part * a.down_each, last = first + a.down_each < pieces ? first + a.down_each : pieces;
  const int tiles = a.r <= 16 ? 1 : a.r <= 32 ? 2 : a.r <= 64 ? 4 : 8;
  // (two turns at most, for every CH: the order of the sums does not depend on the rows)
  const int turns = kWaves / tiles < 2 ? 1 : 2, my = wave / tiles, j = 16 * (wave % tiles) + n16;
  const bool mine = my < turns;
  const __amdgpu_buffer_rsrc_t rd = raw_rsrc(a.down, (uint32_t)(2 * a.K * a.r));
  Activations<kFmtMx, MT, CH, 1, SMOOTH> x(a, last);
  f32x4_t acc[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) acc[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  int x_off[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
    x_off[m] = (16 * m + n16 < a.M ? 16 * m + n16 : a.M - 1) * kRowBytes<CH> + 16 * q;
  u32x4_t w[CH][4];
  auto load = [&](int p0) {
#pragma unroll
    for (int d = 0; d < CH; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[d][i] = load16(rd, mine && (d & (turns - 1)) == my && j < a.r && p0 + d < last
                                 ? (uint32_t)(j * (int)(2 * a.K) + 16 * q) : kNoLoad,
                         (uint32_t)(p0 + d) * (2 * kPiece) + 64 * i);
  };
  x.load(a, first, 0);
  load(first);
  for (int p0 = first; p0 < last; p0 += CH) {
    if (p0 != first) lds_barrier();
    x.store(p0, 0, s_x, nullptr, 0);
    x.load(a, p0 + CH, 0);
    lds_barrier();
#pragma unroll
    for (int d = 0; d < CH; ++d) {
      // (not the other turn's pieces: their zeros times an infinity would be NaN)
      if ((d & (turns - 1)) != my) continue;
      const uint8_t* xp = s_x + d * (kPiece * 2);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int m = 0; m < MT; ++m)
          acc[m] = product(*reinterpret_cast<const u32x4_t*>(xp + x_off[m] + 64 * i), w[d][i], acc[m], std::false_type{});
    }
    load(p0 + CH);
  }
  // [turn][row][tile][rank]
  lds_barrier();
  float* s_sum = reinterpret_cast<float*>(s_x);
  if (mine) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        s_sum[(my * (16 * MT) + 16 * m + 4 * q + i) * (16 * tiles) + j] = acc[m][i];
  }
  __syncthreads();
  for (int o = threadIdx.x; o < a.M * a.r; o += 64 * kWaves) {
    const int m = o / a.r, jj = o % a.r;
    float y = 0.0f;
    for (int t = 0; t < turns; ++t) y += s_sum[(t * (16 * MT) + m) * (16 * tiles) + jj];
    a.D[((int64_t)part * a.M + m) * a.r + jj] = y;
  }
}

// Blocks: those of the down factor's parts first, then the outputs' groups of each part.  (Two waves a SIMD:
// held to four, 33 rows and more spill, 64 of 5120x13824 MXFP4 take 40.9 us for 24.8.)
template <int FMT, int MT, int CH, bool SMOOTH>
__global__ __launch_bounds__(64 * kWaves, 2) void k_gemv_part(GemvArgs a) {
  constexpr int kScaleBytes = 16 * 4 * (CH * scale_words(FMT) > 4 ? CH * scale_words(FMT) : 4);
  __shared__ __attribute__((aligned(16))) uint8_t s_x[2 * 16 * MT * kRowBytes<CH>], s_scale[kWaves * kScaleBytes];
  __shared__ __attribute__((aligned(16))) int s_back[CH * 16 * MT];
  static_assert(sizeof(s_x) >= 8192 * MT, "the down factor's sums are joined in it");
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int block = (int)blockIdx.x - a.down_parts;
  if (block < 0) {
    down_part<MT, CH, SMOOTH>(a, blockIdx.x, s_x);
    return;
  }
  const int pieces = (int)(a.K / kPiece);
  const int p = block / a.groups, n0 = ((block % a.groups) * kWaves + wave) * 16;
  const int first = p * a.each, last = first + a.each < pieces ? first + a.each : pieces;
  f32x4_t acc[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) acc[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  constexpr int kAhead = MT == 1 ? 8 : 4;
  outputs<FMT, MT, CH, kAhead, SMOOTH>(a, n0, first, last, s_x, s_back, s_scale + wave * kScaleBytes, acc);
  const int quads = (a.M + 3) / 4, n = n0 + (lane & 15);
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int rq = 4 * m + (lane >> 4);
    if (n < a.N && rq < quads)
      *reinterpret_cast<f32x4_t*>(a.sums + (((int64_t)p * quads + rq) * a.N + n) * 4) = acc[m];
  }
}

// The parts' sums and the up factor's product.  A wave has 16 outputs of 16 rows; D, which the block's
// waves share, is cut into three bf16 of eight bits each, 32 ranks a wave, so that its products are exact in
// the fp32 sum (two would be 16 bits of it, and 0.1 us less).  Its time is a launch and the
// latency of loads, so all are on their way at once: eight parts of either, the ones past the last are
// buffer loads without a request.  (With loops that end at the last part: one row of 5120x5120 NVFP4, rank
// 32, 14.8 us for 14.3, five of 5120x13824 MXFP4, rank 128, 20.5 for 19.4, both kernels.)
constexpr int kJoinWaves = 4;

__global__ __launch_bounds__(64 * kJoinWaves) void k_gemv_join(GemvArgs a) {
  constexpr int kCuts = 3;   // of D
  __shared__ __attribute__((aligned(16))) u32x4_t s_d[kJoinWaves][kCuts][64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int n16 = lane & 15, q = lane >> 4;
  const int m0 = blockIdx.y * 16, n = (blockIdx.x * kJoinWaves + wave) * 16 + n16;
  const int quads = (a.M + 3) / 4, rq = m0 / 4 + q;
  const bool mine = n < a.N && rq < quads;
  const int j = 32 * wave + 8 * q;
  const bool ranks = j < a.r && m0 + n16 < a.M;   // (r is a multiple of 8)
  const uint32_t at_d = ranks ? (uint32_t)(((m0 + n16) * a.r + j) * 4) : kNoLoad;
  const int64_t each_s = (int64_t)quads * a.N, each_d = (int64_t)a.M * a.r;
  const f32x4_t* sums = reinterpret_cast<const f32x4_t*>(a.sums) + (mine ? (int64_t)rq * a.N + n : 0);
  f32x4_t sum = {0.f, 0.f, 0.f, 0.f}, low = sum, d0 = sum, d1 = sum;
  u32x4_t u[kJoinWaves];
#pragma unroll
  for (int s = 0; s < kJoinWaves; ++s)
    u[s] = n < a.N && 32 * s + 8 * q < a.r ? *reinterpret_cast<const u32x4_t*>(a.up + (int64_t)n * a.r + 32 * s + 8 * q)
                                           : u32x4_t{0u, 0u, 0u, 0u};
  constexpr int kAtOnce = 8;
  for (int s0 = 0; s0 < a.parts; s0 += kAtOnce) {
    f32x4_t v[kAtOnce];
#pragma unroll
    for (int s = 0; s < kAtOnce; ++s)   // (past the last: the first again, not added)
      v[s] = sums[s0 + s < a.parts ? (s0 + s) * each_s : 0];
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < kAtOnce; ++s)
      if (s0 + s < a.parts) sum += v[s];
  }
  for (int s0 = 0; s0 < a.down_parts; s0 += kAtOnce) {
    u32x4_t v0[kAtOnce], v1[kAtOnce];
#pragma unroll
    for (int s = 0; s < kAtOnce; ++s) {
      const __amdgpu_buffer_rsrc_t rd = raw_rsrc(a.D + (s0 + s) * each_d, s0 + s < a.down_parts ? (uint32_t)(4 * each_d) : 0u);
      v0[s] = load16(rd, at_d, 0);
      v1[s] = load16(rd, at_d, 16);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < kAtOnce; ++s) {
      d0 += __builtin_bit_cast(f32x4_t, v0[s]);
      d1 += __builtin_bit_cast(f32x4_t, v1[s]);
    }
  }
  if (a.r) {
    // (cut off, not rounded: a number near fp32's largest stays one; of an infinity or NaN the rest is zero)
    u32x4_t cut[kCuts];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float v0 = c < 2 ? d0[2 * (c & 1)] : d1[2 * (c & 1)], v1 = c < 2 ? d0[2 * (c & 1) + 1] : d1[2 * (c & 1) + 1];
#pragma unroll
      for (int i = 0; i < kCuts; ++i) {
        cut[i][c] = __builtin_amdgcn_perm(__float_as_uint(v1), __float_as_uint(v0), 0x07060302u);
        v0 = __builtin_isfinite(v0) ? v0 - bf16_lo(cut[i][c]) : 0.0f;
        v1 = __builtin_isfinite(v1) ? v1 - bf16_hi(cut[i][c]) : 0.0f;
      }
    }
#pragma unroll
    for (int i = 0; i < kCuts; ++i) s_d[wave][i][lane] = cut[i];
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kJoinWaves; ++s)
      if (32 * s < a.r)
#pragma unroll
        for (int i = 0; i < kCuts; ++i) low = product(s_d[s][i][lane], u[s], low, std::false_type{});
  }
  if (!mine) return;
  const float g = a.g ? __builtin_amdgcn_ldexpf(a.g[0], -exponent_of(a.g[0])) : 1.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (4 * rq + i < a.M)
      a.Y[(int64_t)(4 * rq + i) * a.ldy + n] = f32_to_bf16(__builtin_fmaf(sum[i], g, low[i]));
}

// Parts of K for about one block a CU: the least rounds of 256 blocks times the pieces of one, eight more for a
// block's ends.  One row of 5120x13824 int4 takes 18.7 us with 256 blocks a round and 21.1 with two blocks a
// CU, 32 rows 22.0 and 26.6, 64 rows of 5120x5120 NVFP4 20.0 and 23.2; one row of that 12.0 and 11.1.
struct Split {
  int groups, parts, each, down_parts, down_each;
};
Split split_of(int64_t N, int64_t K, int64_t r) {
  constexpr int64_t kSlots = 256, kStep = 4;
  const int64_t pieces = K / kPiece, groups = (N + 16 * kWaves - 1) / (16 * kWaves);
  int64_t best = 0, least = 0;
  for (int64_t each = kStep; each < pieces + kStep && each <= 1024; each += kStep) {
    const int64_t parts = (pieces + each - 1) / each;
    const int64_t cost = (groups * parts + kSlots - 1) / kSlots * (each + 8);
    if (!best || cost < least) {
      best = each;
      least = cost;
    }
  }
  const int64_t down = 4;
  return Split{(int)groups, (int)((pieces + best - 1) / best), (int)best,
               r ? (int)((pieces + down - 1) / down) : 0, (int)down};
}

template <int FMT, int MT>
void launch_part(const GemvArgs& a, hipStream_t s) {
  constexpr int CH = MT <= 2 ? 4 : 2;
  const unsigned grid = (unsigned)(a.groups * a.parts + a.down_parts);
  if (a.lambda)
    k_gemv_part<FMT, MT, CH, true><<<grid, 64 * kWaves, 0, s>>>(a);
  else
    k_gemv_part<FMT, MT, CH, false><<<grid, 64 * kWaves, 0, s>>>(a);
}

template <int FMT>
void launch_rows(const GemvArgs& a, hipStream_t s) {
  switch ((a.M + 15) / 16) {
    case 1: launch_part<FMT, 1>(a, s); break;
    case 2: launch_part<FMT, 2>(a, s); break;
    case 3: launch_part<FMT, 3>(a, s); break;
    default: launch_part<FMT, 4>(a, s); break;
  }
}

}  // namespace

int64_t gemv_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t r) {
  const Split sp = split_of(N, K, r);
  return sp.parts * ((M + 3) / 4 * N * 16) + sp.down_parts * (M * r * 4);
}

hipError_t launch_gemv(int fmt, const uint16_t* X, int64_t M, int64_t K, int64_t ldx,
                       const float* lambda, const uint16_t* down, int64_t r, const uint8_t* codes,
                       const void* scales, const float* g, const uint16_t* up, int64_t N,
                       uint16_t* Y, int64_t ldy, void* workspace, hipStream_t s) {
  const Split sp = split_of(N, K, r);
  float* sums = (float*)workspace;
  const GemvArgs a{X, lambda, codes, (const uint8_t*)scales, g, down, up, sums,
                   sums + sp.parts * ((M + 3) / 4 * N * 4), Y, K, ldx, ldy, (int)M, (int)N, (int)r,
                   sp.groups, sp.parts, sp.each, sp.down_parts, sp.down_each};
  switch (fmt) {
    case kFmtNv: launch_rows<kFmtNv>(a, s); break;
    case kFmtInt4: launch_rows<kFmtInt4>(a, s); break;
    default: launch_rows<kFmtMx>(a, s); break;
  }
  if (hipError_t e = hipGetLastError()) return e;
  const dim3 grid((unsigned)((N + 16 * kJoinWaves - 1) / (16 * kJoinWaves)), (unsigned)((M + 15) / 16));
  k_gemv_join<<<grid, 64 * kJoinWaves, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace svdq
