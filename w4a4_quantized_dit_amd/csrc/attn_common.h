// What the attention kernels of the paged caches share: arguments, a block's sequence, the query in
// operand order, the running softmax of a lane's row, and the entry that joins the splits.
#pragma once

#include "device.h"
#include "kv_layout.h"
#include "launch.h"

namespace svdq {

constexpr float kNoMax = -3.0e38f;  // running maximum before the first visible token
constexpr float kRaise = 8.0f;
constexpr float kMostSum = 4096.0f;

struct AttnArgs {
  const uint16_t* Q;
  uint16_t* O;
  float* lse;            // or NULL
  float* part;           // splits > 1: [splits][rows][heads][dim], then [splits][rows][heads][2]
  const int32_t* cu;
  const int32_t* len;
  const int32_t* table;
  const uint8_t* kc;
  const uint8_t* vc;
  const uint8_t* ks;
  const uint8_t* vs;
  int64_t ldq, ldo, rows, max_blocks, n_pages;
  int B, Hq, Hkv, G, tiles, splits, causal, max_q;
  float c;
  float to_ln, to_ln_lo;  // scale / c, in two parts: c is rounded, and lse in units of scale
  float up;               // O's sums are brought back by this
  int chunk;              // > 0: a split takes attn_chunk() pages, at least so many; 0: they share them evenly
};

// One sequence and key head of a block.  Tokens, rows and pages fit 32 bits (lengths are int32,
// and the entry point bounds rows·G); addresses are formed in 64.
struct Seq {
  int first;   // packed row of its first token
  int n, kv;   // query tokens, cached tokens
  int q;       // query tokens that are computed: at most the caller's bound
  int b, h;
};

__device__ __forceinline__ bool sequence(const AttnArgs& a, int bh, Seq& s) {
  s.b = bh / a.Hkv;
  s.h = bh % a.Hkv;
  s.first = a.cu[s.b];
  const int end = a.cu[s.b + 1];
  s.kv = a.len[s.b];   // (asked for with them)
  if (s.first < 0 || end <= s.first || end > a.rows) return false;
  s.n = end - s.first;
  s.q = s.n < a.max_q ? s.n : a.max_q;
  const int64_t room = a.max_blocks * kPage;
  s.kv = s.kv < 0 ? 0 : (s.kv > room ? (int)room : s.kv);
  return true;
}

// Tokens [0, limit) are visible to query token i.
__device__ __forceinline__ int limit_of(const AttnArgs& a, const Seq& s, int i) {
  if (!a.causal) return s.kv;
  const int v = s.kv - s.n + i + 1;
  return v < 0 ? 0 : v;
}

// Pages of a split: the longest sequence's shared by the splits.  Shorter sequences have fewer splits, of
// the same length, so that the blocks end together; lengths that the host only bounds are shared all the same.
__device__ __forceinline__ int attn_chunk(const AttnArgs& a) {
  int most = 0;
  for (int i = threadIdx.x & 63; i < a.B; i += 64) {
    const int n = a.len[i];
    most = n > most ? n : most;
  }
#pragma unroll
  for (int k = 1; k < 64; k *= 2) {
    const int n = __shfl_xor(most, k);
    most = n > most ? n : most;
  }
  int64_t pages = ((int64_t)most + kPage - 1) / kPage;
  if (pages > a.max_blocks) pages = a.max_blocks;
  const int each = (int)((pages + a.splits - 1) / a.splits);
  return each > a.chunk ? each : a.chunk;
}

// A lane's part of its row's query: channels 64s + 32·half + 8j .. + 7, the operand of step j of the
// products with the 64 channels s.
template <int DIM>
struct QueryRow {
  u32x4_t w[DIM / 64][4];
};

template <int DIM>
__device__ __forceinline__ void query_load(const uint16_t* q, int half, QueryRow<DIM>& r) {
#pragma unroll
  for (int s = 0; s < DIM / 64; ++s)
#pragma unroll
    for (int j = 0; j < 4; ++j) r.w[s][j] = reinterpret_cast<const u32x4_t*>(q + 64 * s + 32 * half)[j];
}

// An infinity or NaN in the row makes all of it NaN (and so every score).
template <int DIM>
__device__ __forceinline__ void query_check(QueryRow<DIM>& r) {
  uint32_t m = 0;
#pragma unroll
  for (int s = 0; s < DIM / 64; ++s)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) m = max_bf16x2(m, r.w[s][j][c] & 0x7FFF7FFFu);
  m = max_bf16x2(m, m >> 16) & 0xFFFFu;
  const uint32_t there = (uint32_t)__shfl_xor((int)m, 32);
  if ((there > m ? there : m) < kInfBits) return;
#pragma unroll
  for (int s = 0; s < DIM / 64; ++s)
#pragma unroll
    for (int j = 0; j < 4; ++j) r.w[s][j] = u32x4_t{0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu};
}

template <int DIM>
struct State {
  f32x16_t o[DIM / 32];  // Oᵀ: lane column = row, registers = channels 8(i/4) + 4·half + i%4
  float m, l;            // maximum (log2 units) and this half's sum
};

template <int DIM>
__device__ __forceinline__ void state_init(State<DIM>& st) {
#pragma unroll
  for (int j = 0; j < DIM / 32; ++j)
#pragma unroll
    for (int i = 0; i < 16; ++i) st.o[j][i] = 0.0f;
  st.m = kNoMax;
  st.l = 0.0f;
}

// The value of the lane's partner in the other half (the same row).
__device__ __forceinline__ float other_half(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}

// Scores of the tokens that the lane's row does not see (lim and later) become −inf.
__device__ __forceinline__ void hide(f32x16_t (&z)[2], int lim, int half) {
  lim -= 4 * half;  // the registers' tokens are then constants
#pragma unroll
  for (int tb = 0; tb < 2; ++tb)
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (32 * tb + 8 * (i >> 2) + (i & 3) >= lim) z[tb][i] = -__builtin_inff();
}

// The larger of the two halves' values.
__device__ __forceinline__ float across(float m) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(m), __float_as_uint(m), false,
                                                  false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// The page's largest score of the lane's row, in log2 units.
__device__ __forceinline__ float largest(const f32x16_t (&z)[2], float c) {
  float t[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    t[k] = fmaxf(z[k >> 1][8 * (k & 1)], z[k >> 1][8 * (k & 1) + 1]);
#pragma unroll
    for (int i = 2; i < 8; i += 2)
      t[k] = fmaxf(fmaxf(t[k], z[k >> 1][8 * (k & 1) + i]), z[k >> 1][8 * (k & 1) + i + 1]);
  }
  return across(fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]))) * c;
}

// Raises the running maximum to the page's: always, or where some row needs it.
template <int DIM>
__device__ __forceinline__ void raise_to(State<DIM>& st, float top) {
  const float m = fmaxf(st.m, top), f = __builtin_amdgcn_exp2f(st.m - m);
#pragma unroll
  for (int j = 0; j < DIM / 32; ++j)
#pragma unroll
    for (int i = 0; i < 16; ++i) st.o[j][i] *= f;
  st.l *= f;
  st.m = m;
}

template <int DIM>
__device__ __forceinline__ void raise(State<DIM>& st, float top) {
  if (__builtin_amdgcn_ballot_w64(top > st.m + kRaise) != 0) raise_to(st, top);
}

// Weights of 16 tokens (step g of token block tb) as an operand of the product with V.
template <int DIM>
__device__ __forceinline__ bf16x8_t weights(State<DIM>& st, const f32x16_t (&z)[2], int tb, int g,
                                            float c) {
  u32x4_t w;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(z[tb][8 * g + 2 * j], c, -st.m));
    const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(z[tb][8 * g + 2 * j + 1], c, -st.m));
    st.l += x + y;
    w[j] = pack_bf16x2(x, y);
  }
  return __builtin_bit_cast(bf16x8_t, w);
}

// The lane's logical page `at` (of pages [0, end), end >= 1; later ones repeat the last): its
// number in the cache, −1 outside it.
__device__ __forceinline__ int page_id(const AttnArgs& a, const Seq& s, int at, int end) {
  const int p = a.table[(int64_t)s.b * a.max_blocks + (at < end ? at : end - 1)];
  return p >= 0 && p < a.n_pages ? p : -1;
}

// lse from the maximum (c·z rounded; l makes up for that) and the sum.
__device__ __forceinline__ float lse_of(const AttnArgs& a, float m, float l) {
  if (l == 0.0f) return -__builtin_inff();
  const float rest = __builtin_fmaf(m, a.to_ln_lo, 0.6931471805599453f * __builtin_amdgcn_logf(l));
  return __builtin_fmaf(m, a.to_ln, rest);
}

// Many rows: four waves of 32 rows share a page.  Few rows: blocks of 32, whose waves share the pages.
constexpr int kTileWaves = 4;
constexpr int kTileRows = 32 * kTileWaves;
constexpr int kFewRows = 32;
constexpr int64_t kFewMost = 512;  // of a key head, in blocks of so many (measured to there)

// The kernel, its row tiles and the splits of the page range.
struct AttnPlan {
  bool few;
  int64_t tiles, splits;
  int chunk;   // AttnArgs::chunk
};

AttnPlan attn_plan(int64_t G, int64_t Hkv, int64_t dim, int64_t rows, int64_t B, int64_t max_q,
                   int64_t max_kv);

// Arguments of a call; c, to_ln from the scale.
AttnArgs attn_args(const uint16_t* Q, int64_t ldq, int64_t rows, int64_t Hq, int64_t Hkv,
                   const int32_t* cu, const int32_t* len, int64_t B, int64_t max_q,
                   const int32_t* table, int64_t max_blocks, int64_t n_pages, const uint8_t* kc,
                   const uint8_t* vc, const uint8_t* ks, const uint8_t* vs, float scale, int causal,
                   uint16_t* O, int64_t ldo, float* lse, void* workspace, const AttnPlan& p, float up);

// Joins the splits of every row.
hipError_t launch_attn_join(const AttnArgs& a, int64_t dim, hipStream_t s);

}  // namespace svdq
