// Softmax attention of bf16 query rows over the paged 8-bit cache (kv_layout.h):
//
//   z[t] = c·(q·k_t) over the tokens t the row sees,  c = scale·log2(e)
//   O = Σ_t 2^(z_t − m) v_t / l,   l = Σ_t 2^(z_t − m),   lse = ln 2·(m + log2 l)
//
// in one pass over the pages with a running maximum m (fp32 statistics and sums).  The rows of
// a key head are its query heads' rows interleaved (row = token·G + member), so grouped heads
// share every page read and single tokens still fill a matrix operand.
//
// Sᵀ = K·Qᵀ runs on the 32x32x16 bf16 MFMA: K's codes are widened exactly, with the page's exponent,
// and every product is exact in the fp32 sum.  (The FP8 MFMA on the codes themselves, the query split
// into two E4M3 codes, took 4.39 ms instead of 4.73 for 16384 rows x 16384 tokens x 40 heads of 128,
// but it aligns the products of neighbouring channels to the largest of them with 13 bits: scores
// were off by 2^-16 of Σ|q_d k_d| instead of 2^-24.)
//
// Oᵀ += Vᵀ·Pᵀ runs on the 32x32x16 bf16 MFMA: V's codes are widened exactly (with the page's
// exponent) and P is rounded to bf16 once, at most 2^-8 of each weight against l's unrounded sum
// (1.1 to 1.4e-3 of O in the root mean square, where rounding O itself to bf16 is 1.6e-3; together
// 2.0 to 2.2e-3).  fp16 would hold three bits more, but not the range of the pages' exponents, which
// bf16 takes along with the codes.  The accumulator of Sᵀ holds, per lane, one row's weights in exactly
// the token order of the stored V, so P needs no exchange between lanes.
//
// The maximum is only raised when a page exceeds it by more than 2^8 (few rows) or its weights add
// up to more than 2^12 (many rows): bf16 and fp32 hold the larger weights as well, and most pages
// skip the rescaling of O, and with many rows the maximum itself.
#include "device.h"
#include "kv_layout.h"
#include "launch.h"

namespace svdq {

namespace {

constexpr float kNoMax = -3.0e38f;  // running maximum before the first visible token
constexpr float kRaise = 8.0f;
constexpr float kMostSum = 4096.0f;

// V is widened as 2^-16 of itself and O brought back where it is stored, exact steps both: the sum of
// V over its weights is formed before the division by theirs, and cached values reach 2^128.  Sixteen
// bits are what the smallest page exponent leaves (-110 - 16 is that of fp32's smallest normal).
constexpr int kDown = 16;
constexpr float kUp = 65536.0f;

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
  if (s.first < 0 || end <= s.first || end > a.rows) return false;
  s.n = end - s.first;
  s.q = s.n < a.max_q ? s.n : a.max_q;
  s.kv = a.len[s.b];
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

// Eight codes of V, widened exactly with the page's scale: one lane's part of a 16-token step.
__device__ __forceinline__ bf16x8_t widen8(uint32_t lo, uint32_t hi, float scale) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
  const bf16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A lane's 16 bytes of a V fragment (tokens 32·tb on) without the slots past the page's n tokens,
// which may hold any byte, NaN codes among them: a weight of 0 would not hide those.
__device__ __forceinline__ u32x4_t drop_slots(u32x4_t v, int tb, int half, int n) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    int k = n - (32 * tb + 16 * (d >> 1) + 8 * (d & 1) + 4 * half);
    k = k < 0 ? 0 : (k > 4 ? 4 : k);
    v[d] &= (uint32_t)((1ull << (8 * k)) - 1ull);
  }
  return v;
}

// A lane's 16 bytes of a V fragment with its NaN codes made 0; `dirty` becomes true where a lane of
// the wave had one.  With the causal mask the rows of a block share pages of which some do not
// see every token, and a weight of 0 does not hide a NaN; those that do see it get it back from
// `restore_nan`.
__device__ __forceinline__ u32x4_t clear_nan(u32x4_t v, bool& dirty) {
  uint32_t any = 0;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const uint32_t nan = ((v[d] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
    v[d] &= ~((nan >> 7) * 0xFFu);
    any |= nan;
  }
  dirty = dirty || __builtin_amdgcn_ballot_w64(any != 0) != 0;
  return v;
}

// Scores Sᵀ of a page: token blocks of 32, lane column = row, registers = tokens
// 8(i/4) + 4·half + i%4.  kf(i): the lane's 16 bytes of K fragment i.
template <int DIM, class KF>
__device__ __forceinline__ void scores(f32x16_t (&z)[2], const QueryRow<DIM>& q, float scale, KF kf) {
#pragma unroll
  for (int tb = 0; tb < 2; ++tb) {
#pragma unroll
    for (int i = 0; i < 16; ++i) z[tb][i] = 0.0f;
#pragma unroll
    for (int s = 0; s < DIM / 64; ++s)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const u32x4_t k = kf((tb * (DIM / 64) + s) * 2 + j / 2);
        z[tb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            widen8(k[2 * (j & 1)], k[2 * (j & 1) + 1], scale), __builtin_bit_cast(bf16x8_t, q.w[s][j]),
            z[tb], 0, 0, 0);
      }
  }
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

// NaN in the channels in which a token that the lane's row sees, in pages [p0, p1), has a NaN code.
template <int DIM>
__device__ __forceinline__ void restore_nan(const AttnArgs& a, const Seq& s, State<DIM>& st, int p0,
                                            int p1, int lim_row, int half) {
  uint64_t bad = 0;  // bit 16 j + i: accumulator o[j][i]
  for (int p = p0; p < p1; ++p) {
    const int page = a.table[(int64_t)s.b * a.max_blocks + p];
    if (page < 0 || page >= a.n_pages) continue;
    const uint8_t* codes = a.vc + ((int64_t)page * a.Hkv + s.h) * (kPage * DIM);
    for (int t = 0; t < kPage; t += 4) {
      const int64_t n = lim_row - ((int64_t)p * kPage + t);
      const uint32_t seen = n >= 4 ? ~0u : (n > 0 ? (1u << (8 * n)) - 1u : 0u);
      for (int k = 0; k < DIM / 2; ++k) {
        const int d = 32 * (k >> 4) + 8 * ((k >> 2) & 3) + 4 * half + (k & 3);
        const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + v_offset(t, d)) & seen;
        if (((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) bad |= 1ull << k;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < DIM / 32; ++j)
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if ((bad >> (16 * j + i)) & 1) st.o[j][i] = __builtin_nanf("");
}

constexpr int kPresent = 1 << 16;

// The lane's logical page `at` (of pages [0, end), end >= 1; later ones repeat the last): its
// number in the cache, −1 outside it.
__device__ __forceinline__ int page_id(const AttnArgs& a, const Seq& s, int at, int end) {
  const int p = a.table[(int64_t)s.b * a.max_blocks + (at < end ? at : end - 1)];
  return p >= 0 && p < a.n_pages ? p : -1;
}

// Exponent bytes (k | v << 8 | kPresent, V's less kDown) of a page, no flag outside the cache; the
// number of a missing page becomes 0, which can be read.
__device__ __forceinline__ int page_exps(const AttnArgs& a, const Seq& s, int& page) {
  const bool there = page >= 0;
  page = there ? page : 0;
  const int64_t i = (int64_t)page * a.Hkv + s.h;
  const int v = (int)a.vs[i] - kDown;  // (below 0: only in a page that was never written)
  const int e = (int)a.ks[i] | (v < 0 ? 0 : v) << 8;
  return there ? e | kPresent : 0;
}

// lse from the maximum (c·z rounded; l makes up for that) and the sum.
__device__ __forceinline__ float lse_of(const AttnArgs& a, float m, float l) {
  if (l == 0.0f) return -__builtin_inff();
  const float rest = __builtin_fmaf(m, a.to_ln_lo, 0.6931471805599453f * __builtin_amdgcn_logf(l));
  return __builtin_fmaf(m, a.to_ln, rest);
}

// Output of one row: bf16 and lse, or the unnormalised sums of a split.
template <int DIM>
__device__ __forceinline__ void store_row(const AttnArgs& a, const State<DIM>& st, float l,
                                          int64_t token, int head, int split, int half) {
  if (a.splits > 1) {
    const int64_t at = ((int64_t)split * a.rows + token) * a.Hq + head;
    float* o = a.part + at * DIM;
#pragma unroll
    for (int j = 0; j < DIM / 32; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<f32x4_t*>(o + 32 * j + 8 * g + 4 * half) =
            f32x4_t{st.o[j][4 * g], st.o[j][4 * g + 1], st.o[j][4 * g + 2], st.o[j][4 * g + 3]};
    if (half == 0) {
      float* ml = a.part + (int64_t)a.splits * a.rows * a.Hq * DIM + at * 2;
      ml[0] = st.m;
      ml[1] = l;
    }
    return;
  }
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;
  auto value = [&](int j, int i) { return st.o[j][i] * inv * kUp; };
  uint16_t* o = a.O + token * a.ldo + (int64_t)head * DIM;
#pragma unroll
  for (int j = 0; j < DIM / 32; ++j)
#pragma unroll
    for (int g = 0; g < 4; ++g)
      *reinterpret_cast<uint2*>(o + 32 * j + 8 * g + 4 * half) =
          uint2{pack_bf16x2(value(j, 4 * g), value(j, 4 * g + 1)),
                pack_bf16x2(value(j, 4 * g + 2), value(j, 4 * g + 3))};
  if (a.lse && half == 0)
    a.lse[token * a.Hq + head] = lse_of(a, st.m, l);
}

// Many rows: four waves of 32 rows share each page through LDS.  Its codes go through registers, V's
// two pages ahead and K's three, and are widened to bf16 on the way, once for the four waves (each
// wave widening all of V for itself took a third of its vector instructions, all of K 3 % of the
// time of 16384 x 16384 x 40 heads of 128).  Two images of each, one barrier a page.
constexpr int kTileWaves = 4;
constexpr int kTileRows = 32 * kTileWaves;

template <int DIM>
__global__ __launch_bounds__(64 * kTileWaves, 2) void k_attn_tile(AttnArgs a) {
  constexpr int kBytes = kPage * DIM;                       // one tensor's page
  constexpr int kCopies = kBytes / 1024 / kTileWaves;       // fragments per wave, K and V each
  __shared__ __attribute__((aligned(16))) uint8_t k_img[2][2 * kBytes], v_img[2][2 * kBytes];
  __shared__ int s_dirty[kTileWaves];
  const int64_t total = (int64_t)a.B * a.Hkv * a.splits * a.tiles;
  const int64_t per_xcd = (total + 7) / 8;
  const int64_t item = (int64_t)(blockIdx.x % 8) * per_xcd + blockIdx.x / 8;
  if (item >= total || blockIdx.x / 8 >= per_xcd) return;
  // the last rows first: with the causal mask they see the most
  const int tile = a.tiles - 1 - (int)(item % a.tiles);
  const int split = (int)((item / a.tiles) % a.splits);
  Seq s;
  if (!sequence(a, (int)(item / a.tiles / a.splits), s)) return;
  const int R = s.q * a.G, r0 = tile * kTileRows;
  if (r0 >= R) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, half = lane >> 5;
  const int w0 = r0 + 32 * wave, row = w0 + (lane & 31);
  const bool live = row < R;
  const int tok = live ? row / a.G : 0;
  const int head = s.h * a.G + (live ? row % a.G : 0);

  // pages of this block, and tokens that the wave's first row and the lane's row see
  const int last = (r0 + kTileRows < R ? r0 + kTileRows : R) - 1;
  const int pages = (int)(((int64_t)limit_of(a, s, last / a.G) + kPage - 1) / kPage);
  const int p0 = __builtin_amdgcn_readfirstlane((int)((int64_t)pages * split / a.splits));
  const int p1 = __builtin_amdgcn_readfirstlane((int)((int64_t)pages * (split + 1) / a.splits));
  const int lim_row = live ? limit_of(a, s, tok) : 0;
  // (a wave without rows hides nothing: it would do so on every page)
  const int lim_first = __builtin_amdgcn_readfirstlane(w0 < R ? limit_of(a, s, w0 / a.G) : s.kv);

  // (rows past the last read token 0's; nothing of them is stored)
  QueryRow<DIM> q;
  query_load<DIM>(a.Q + (int64_t)(s.first + tok) * a.ldq + (int64_t)head * DIM, half, q);
  State<DIM> st;
  state_init(st);

  const int64_t head_off = (int64_t)s.h * kBytes + lane * 16;
  const int64_t page_bytes = (int64_t)a.Hkv * kBytes;
  const uint8_t* k_src = a.kc + head_off + wave * kCopies * 1024;
  const uint8_t* v_src = a.vc + head_off + wave * kCopies * 1024;
  u32x4_t kr[kCopies], vr[kCopies];
  auto load_k = [&](int page) {
#pragma unroll
    for (int i = 0; i < kCopies; ++i)
      kr[i] = *reinterpret_cast<const u32x4_t*>(k_src + page * page_bytes + i * 1024);
  };
  auto load_v = [&](int page) {
#pragma unroll
    for (int i = 0; i < kCopies; ++i)
      vr[i] = *reinterpret_cast<const u32x4_t*>(v_src + page * page_bytes + i * 1024);
  };
  // the sequence's last page may hold fewer tokens than slots, and a page outside the cache (page 0
  // is read in its place) holds none
  const int whole = s.kv / kPage;
  // pages that every row of the block sees whole
  const int shared_pages = __builtin_amdgcn_readfirstlane(limit_of(a, s, r0 / a.G) / kPage);
  bool dirty = false;
  auto trim_v = [&](int i, int exps) {
    if (i < shared_pages && (exps & kPresent)) return;
    const int n = !(exps & kPresent) || i > whole ? 0 : i == whole ? s.kv % kPage : kPage;
#pragma unroll
    for (int f = 0; f < kCopies; ++f) vr[f] = drop_slots(vr[f], (wave * kCopies + f) & 1, half, n);
    if (a.causal) {
#pragma unroll
      for (int f = 0; f < kCopies; ++f) vr[f] = clear_nan(vr[f], dirty);
    }
  };
  // step g of the wave's fragment f: 16 tokens of V, or 8 channels of each half of K's block of 64
  auto widen = [&](uint8_t* img, const u32x4_t& r, int f, int g, float scale) {
    *reinterpret_cast<bf16x8_t*>(img + (2 * (wave * kCopies + f) + g) * 1024 + lane * 16) =
        widen8(r[2 * g], r[2 * g + 1], scale);
  };
  auto widen_k = [&](int exps, int slot) {
#pragma unroll
    for (int n = 0; n < 2 * kCopies; ++n)
      widen(k_img[slot], kr[n / 2], n / 2, n % 2, two_to((exps & 255) - 127));
  };
  auto widen_v = [&](int exps, int slot) {
#pragma unroll
    for (int n = 0; n < 2 * kCopies; ++n)
      widen(v_img[slot], vr[n / 2], n / 2, n % 2, two_to(((exps >> 8) & 255) - 127));
  };
  constexpr int kQk = 8 * (DIM / 64), kPv = 4 * (DIM / 32);
  auto k_operand = [&](int slot, int n) {
    return *reinterpret_cast<const bf16x8_t*>(&k_img[slot][n * 1024 + lane * 16]);
  };
  auto product = [&](f32x16_t (&z)[2], int n, bf16x8_t k) {
    const int tb = n / (kQk / 2), m = n % (kQk / 2);
    if (m == 0) z[tb] = f32x16_t{};
    z[tb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k, __builtin_bit_cast(bf16x8_t, q.w[m / 4][m % 4]),
                                                    z[tb], 0, 0, 0);
  };
  auto mask = [&](int i, int exps, f32x16_t (&z)[2]) {
    if (!(exps & kPresent) || i >= lim_first / kPage) {
      const uint32_t t0 = (uint32_t)i * kPage, lim = (uint32_t)lim_row;
      const uint32_t lr = (exps & kPresent) && lim > t0 ? lim - t0 : 0u;
      hide(z, lr > kPage ? kPage : (int)lr, half);
    }
  };

  if (p0 < p1) {
    // lane l: page number and exponents of logical page g0 + l.  The loads need the numbers only,
    // the exponents come and the query is looked over while they are on their way.
    int g0 = p0, meta = page_id(a, s, g0 + lane, p1), meta_e;
    auto lane_of = [&](int i) { return (i < p1 ? i : p1 - 1) - g0; };
    auto page_at = [&](int i) { return __builtin_amdgcn_readlane(meta, lane_of(i)); };
    auto exps_at = [&](int i) { return __builtin_amdgcn_readlane(meta_e, lane_of(i)); };

    f32x16_t za[2], zb[2];
    {
      const int first = page_at(p0);
      load_k(first < 0 ? 0 : first);
      load_v(first < 0 ? 0 : first);
      meta_e = page_exps(a, s, meta);
    }
    query_check(q);
    const int e0 = exps_at(p0);
    trim_v(p0, e0);
    widen_k(e0, 0);
    load_k(page_at(p0 + 1));
    widen_v(e0, 0);
    load_v(page_at(p0 + 1));
    widen_k(exps_at(p0 + 1), 1);
    load_k(page_at(p0 + 2));
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
    for (int n = 0; n < kQk; ++n) product(za, n, k_operand(0, n));
    mask(p0, e0, za);
    raise(st, largest(za, a.c));

    // Page i, whose scores are in z: its exponentials run while the matrix units form the next
    // page's scores, and the next page's V and the keys behind it are widened while they form
    // this page's product.
    // Pages behind the last repeat it; what is computed of them is not used.
    auto step = [&](int i, int slot, f32x16_t (&z)[2], f32x16_t (&zn)[2]) {
      // K of page i + 1 and V of page i are in LDS for every wave, and every wave is done with
      // what takes their places (V of page i + 1 and K of page i + 2 may still be on their way)
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      if (i - g0 >= 61) {
        g0 = i;
        meta = page_id(a, s, g0 + lane, p1);
        meta_e = page_exps(a, s, meta);
      }
      const int e1 = exps_at(i + 1);
      trim_v(i + 1, e1);
      // From here to the masks one block without branches, its order fixed: a wave issues in
      // order, so what is to run under a matrix instruction has to stand right behind it.
      const int v_next = page_at(i + 2), k_next = page_at(i + 3);
      const float k_scale = two_to((exps_at(i + 2) & 255) - 127);
      const float v_scale = two_to(((e1 >> 8) & 255) - 127);
      const uint8_t* vp = v_img[slot] + lane * 16;
      u32x4_t w[4];
      bf16x8_t kb[4], vb[4];
      float sum = 0.0f;
      // V operand n: channels 32 (n % (DIM/32)) on, token step n / (DIM/32)
      auto v_read = [&](int n) {
        const int j = n % (DIM / 32), t = n / (DIM / 32);
        vb[n % 4] = *reinterpret_cast<const bf16x8_t*>(
            vp + ((2 * j + (t >> 1)) * 2 + (t & 1)) * 1024);
      };
      // weights of two tokens: pair n of the lane's sixteen
      auto pair = [&](int n) {
        const int tb = n >> 3, e = 2 * (n & 7);
        const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(z[tb][e], a.c, -st.m));
        const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(z[tb][e + 1], a.c, -st.m));
        sum += x + y;
        uint32_t both = pack_bf16x2(x, y);
        asm volatile("" : "+v"(sum), "+v"(both));  // formed here, not behind the block
        w[n >> 2][n & 3] = both;
      };
#pragma unroll
      for (int n = 0; n < 4; ++n) kb[n] = k_operand(slot ^ 1, n);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int n = 0; n < kQk; ++n) {
        product(zn, n, kb[n % 4]);
        if (n + 4 < kQk) kb[n % 4] = k_operand(slot ^ 1, n + 4);
        if (n == kQk - 1) {
#pragma unroll
          for (int f = 0; f < 4; ++f) v_read(f);
        }
        // (fewer behind the first ones: the last scores are ready when the last weights are)
        constexpr int kEach = 16 / kQk;
#pragma unroll
        for (int f = n * kEach - (n > 0) - (n > 1); f < (n + 1) * kEach - (n < kQk - 1) - (n > 0 && n < kQk - 1); ++f)
          pair(f);
        __builtin_amdgcn_sched_barrier(0);
      }
      asm volatile("" : "+v"(zn[0]), "+v"(zn[1]));  // formed here, not behind the branch
      // The page's maximum is not taken: the sum of its weights tells when they have grown too
      // large for the running maximum (a first page's are small, and 32 of at most 1 after a
      // raise).  Then, seldom, the maximum is raised and the weights are formed again.
      if (__builtin_amdgcn_ballot_w64(!(sum <= kMostSum)) != 0) {
        raise_to(st, largest(z, a.c));
        sum = 0.0f;
#pragma unroll
        for (int n = 0; n < 16; ++n) pair(n);
      }
      st.l += sum;
#pragma unroll
      for (int n = 0; n < kPv; ++n) {
        const int j = n % (DIM / 32), t = n / (DIM / 32);
        st.o[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            vb[n % 4], __builtin_bit_cast(bf16x8_t, w[t]), st.o[j], 0, 0, 0);
        if (n + 4 < kPv) v_read(n + 4);
        // the next page's V, then the keys of the one behind it, a step at a time
        if (n % 2 == 0 && n < kPv / 2) widen(v_img[slot ^ 1], vr[n / 4], n / 4, n / 2 % 2, v_scale);
        if (n % 2 == 0 && n >= kPv / 2)
          widen(k_img[slot], kr[(n - kPv / 2) / 4], (n - kPv / 2) / 4, n / 2 % 2, k_scale);
        if (n == kPv / 2) load_v(v_next);
        if (n == kPv - 1) load_k(k_next);
        __builtin_amdgcn_sched_barrier(0);
      }
      mask(i + 1, e1, zn);
    };
    for (int i = p0; i < p1; i += 2) {
      step(i, 0, za, zb);
      if (i + 1 < p1) step(i + 1, 1, zb, za);
    }
  }
  if (a.causal) {
    s_dirty[wave] = dirty;
    __syncthreads();
    if (s_dirty[0] | s_dirty[1] | s_dirty[2] | s_dirty[3])
      restore_nan(a, s, st, p0 > shared_pages ? p0 : shared_pages, p1, lim_row, half);
  }
  const float l = st.l + other_half(st.l);
  if (live) store_row<DIM>(a, st, l, s.first + tok, head, split, half);
}

// Few rows (single tokens, small groups): blocks of 32, whose four waves take every fourth page each,
// straight into registers, and join their sums through LDS.  Where a key head has more than 32 rows
// (TILES) its blocks are neighbours on one XCD, and the pages stay in its cache for them.
constexpr int kFewRows = 32;
constexpr int64_t kFewMost = 512;  // of a key head, in blocks of so many (measured to there)

template <int DIM, bool TILES>
__global__ __launch_bounds__(256, 2) void k_attn_few(AttnArgs a) {
  constexpr int kBytes = kPage * DIM;
  constexpr int kFrags = kBytes / 1024;
  __shared__ float s_o[4][DIM][33];
  __shared__ float s_m[4][32], s_l[4][32];
  int64_t item = blockIdx.x;
  int r0 = 0;
  if (TILES) {
    const int64_t total = (int64_t)a.B * a.Hkv * a.splits * a.tiles, per_xcd = (total + 7) / 8;
    item = (int64_t)(blockIdx.x % 8) * per_xcd + blockIdx.x / 8;
    if (item >= total || blockIdx.x / 8 >= per_xcd) return;
    r0 = kFewRows * (int)(item % a.tiles);
    item /= a.tiles;
  }
  const int split = (int)(item % a.splits);
  Seq s;
  if (!sequence(a, (int)(item / a.splits), s)) return;
  int R = s.q * a.G - r0;
  if (R <= 0) return;
  R = R < kFewRows ? R : kFewRows;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, half = lane >> 5, n = lane & 31;
  const bool live = n < R;
  const int tok = (r0 + (live ? n : 0)) / a.G;
  const int head = s.h * a.G + (r0 + (live ? n : 0)) % a.G;
  const int pages = (int)(((int64_t)limit_of(a, s, (r0 + R - 1) / a.G) + kPage - 1) / kPage);
  const int p0 = (int)((int64_t)pages * split / a.splits);
  const int p1 = (int)((int64_t)pages * (split + 1) / a.splits);
  const int lim_row = live ? limit_of(a, s, tok) : 0;
  const int lim_first = limit_of(a, s, r0 / a.G);

  QueryRow<DIM> q;
  query_load<DIM>(a.Q + (int64_t)(s.first + tok) * a.ldq + (int64_t)head * DIM, half, q);
  State<DIM> st;
  state_init(st);
  const int64_t head_off = (int64_t)s.h * kBytes + lane * 16, page_bytes = (int64_t)a.Hkv * kBytes;
  query_check(q);
  bool dirty = false;
  for (int g0 = p0 + wave; g0 < p1; g0 += 256) {
    // lane l: logical page g0 + 4 l
    int meta = page_id(a, s, g0 + 4 * lane, p1);
    const int meta_e = page_exps(a, s, meta);
    u32x4_t kr[kFrags], vr[kFrags];
    auto load = [&](u32x4_t (&r)[kFrags], const uint8_t* codes, int page) {
#pragma unroll
      for (int f = 0; f < kFrags; ++f)
        r[f] = TILES ? *reinterpret_cast<const u32x4_t*>(codes + page * page_bytes + head_off + f * 1024)
                     : load_nt(codes + page * page_bytes + head_off + f * 1024);
    };
    const int count = (p1 - g0 + 3) / 4 < 64 ? (p1 - g0 + 3) / 4 : 64;
    load(kr, a.kc, __builtin_amdgcn_readfirstlane(meta));
    load(vr, a.vc, __builtin_amdgcn_readfirstlane(meta));
    for (int d = 0; d < count; ++d) {
      const int exps = __builtin_amdgcn_readlane(meta_e, d);
      const int next = __builtin_amdgcn_readlane(meta, d + 1 < count ? d + 1 : d);
      const int t0 = (g0 + 4 * d) * kPage;
      const float scale = two_to(((exps >> 8) & 255) - 127);
      f32x16_t z[2];
      scores<DIM>(z, q, two_to((exps & 255) - 127), [&](int f) { return kr[f]; });
      load(kr, a.kc, next);
      if (!(exps & kPresent) || t0 > lim_first - kPage) {
        const int lr = (exps & kPresent) ? lim_row - t0 : 0, lk = (exps & kPresent) ? s.kv - t0 : 0;
        hide(z, lr > kPage ? kPage : (lr < 0 ? 0 : lr), half);
#pragma unroll
        for (int f = 0; f < kFrags; ++f)
          vr[f] = drop_slots(vr[f], f & 1, half, lk > kPage ? kPage : lk);
        if (a.causal) {
#pragma unroll
          for (int f = 0; f < kFrags; ++f) vr[f] = clear_nan(vr[f], dirty);
        }
      }
      raise(st, largest(z, a.c));
#pragma unroll
      for (int tb = 0; tb < 2; ++tb)
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const bf16x8_t p = weights(st, z, tb, g, a.c);
#pragma unroll
          for (int j = 0; j < DIM / 32; ++j)
            st.o[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                widen8(vr[2 * j + tb][2 * g], vr[2 * j + tb][2 * g + 1], scale), p, st.o[j], 0, 0, 0);
        }
      load(vr, a.vc, next);
    }
  }
  if (dirty) {
    const int part = lim_first / kPage;
    restore_nan(a, s, st, p0 > part ? p0 : part, p1, lim_row, half);
  }
  // join the four waves
  st.l += other_half(st.l);
  if (half == 0) {
    s_m[wave][n] = st.m;
    s_l[wave][n] = st.l;
  }
  __syncthreads();
  const float m = fmaxf(fmaxf(s_m[0][n], s_m[1][n]), fmaxf(s_m[2][n], s_m[3][n]));
  const float f = __builtin_amdgcn_exp2f(st.m - m);
#pragma unroll
  for (int j = 0; j < DIM / 32; ++j)
#pragma unroll
    for (int i = 0; i < 16; ++i)
      s_o[wave][32 * j + 8 * (i >> 2) + 4 * half + (i & 3)][n] = st.o[j][i] * f;
  __syncthreads();
  for (int o = threadIdx.x; o < R * DIM; o += 256) {
    const int rr = o / DIM, d = o % DIM;
    float sum = 0.0f, l = 0.0f;
    const float mm = fmaxf(fmaxf(s_m[0][rr], s_m[1][rr]), fmaxf(s_m[2][rr], s_m[3][rr]));
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      sum += s_o[w][d][rr];
      l += s_l[w][rr] * __builtin_amdgcn_exp2f(s_m[w][rr] - mm);
    }
    const int64_t token = s.first + (r0 + rr) / a.G;
    const int hd = s.h * a.G + (r0 + rr) % a.G;
    if (a.splits > 1) {
      const int64_t at = ((int64_t)split * a.rows + token) * a.Hq + hd;
      a.part[at * DIM + d] = sum;
      if (d == 0) {
        float* ml = a.part + (int64_t)a.splits * a.rows * a.Hq * DIM + at * 2;
        ml[0] = mm;
        ml[1] = l;
      }
    } else {
      a.O[token * a.ldo + (int64_t)hd * DIM + d] = f32_to_bf16(l != 0.0f ? sum / l * kUp : 0.0f);
      if (a.lse && d == 0)
        a.lse[token * a.Hq + hd] = lse_of(a, mm, l);
    }
  }
}

// The splits of every row joined, a wave a row of sequence blockIdx.y, the blocks in sweeps of
// kJoinMost where a sequence has more rows (a launch has fewer than 2^32 threads in a dimension).  The
// lanes take the splits' maxima side by side, and groups of DIM / 4 lanes, four channels each, take
// every second (DIM 128) or fourth split, several loads under way at once (one split after the other
// with all lanes took 25 us for 128 rows of 48 splits, now 4).
constexpr int64_t kJoinMost = 1 << 20;

template <int DIM>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a) {
  constexpr int kWide = DIM / 4, kGroups = 64 / kWide;
  const int b = blockIdx.y, lane = threadIdx.x & 63;
  const int first = a.cu[b], end = a.cu[b + 1];
  if (first < 0 || end <= first || end > a.rows) return;
  const int n = end - first < a.max_q ? end - first : a.max_q;
  const int64_t each = a.rows * a.Hq, rows = (int64_t)n * a.Hq;
  for (int64_t local = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); local < rows;
       local += (int64_t)gridDim.x * 4) {
    const int64_t at = (int64_t)first * a.Hq + local, token = at / a.Hq;
    const int head = (int)(at % a.Hq);
    const float2* ml = reinterpret_cast<const float2*>(a.part + a.splits * each * DIM) + at;
    float m = kNoMax;
    for (int i = lane; i < a.splits; i += 64) m = fmaxf(m, ml[i * each].x);
#pragma unroll
    for (int k = 1; k < 64; k *= 2) m = fmaxf(m, __shfl_xor(m, k));
    float l = 0.0f;
    for (int i = lane; i < a.splits; i += 64) {
      const float2 v = ml[i * each];
      l += v.y * __builtin_amdgcn_exp2f(v.x - m);
    }
#pragma unroll
    for (int k = 1; k < 64; k *= 2) l += __shfl_xor(l, k);
    const int d = 4 * (lane % kWide);
    f32x4_t o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int i = lane / kWide; i < a.splits; i += kGroups) {
      const float f = __builtin_amdgcn_exp2f(ml[i * each].x - m);
      o += *reinterpret_cast<const f32x4_t*>(a.part + (i * each + at) * DIM + d) * f;
    }
#pragma unroll
    for (int k = kWide; k < 64; k *= 2)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[c] += __shfl_xor(o[c], k);
    if (lane >= kWide) continue;
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
    *reinterpret_cast<uint2*>(a.O + token * a.ldo + (int64_t)head * DIM + d) =
        uint2{pack_bf16x2(o[0] * inv * kUp, o[1] * inv * kUp),
              pack_bf16x2(o[2] * inv * kUp, o[3] * inv * kUp)};
    if (a.lse && lane == 0)
      a.lse[at] = lse_of(a, m, l);
  }
}

struct Plan {
  bool few;
  int64_t tiles, splits;
};

// The kernel and the splits of the page range are the ones of the least time, in pages of a wave
// (1.2 us at 64 channels, 2 at 128).  Both kernels run in rounds of 512 blocks, two a CU.
//   tile: rounds · (pages a block + 4 for its ends), up to 16 splits
//   few:  rounds · (a quarter of the pages + 5), but no less than its reads take: a page for each 32
//         rows from memory, or a little over half of that from the XCD's cache where a key head has
//         several blocks
// and with splits a join: its launch and the blocks' longer ends (4 and 8), and the fp32 rows written
// and read.  The constants are fitted, the same for both head sizes: as rates those of the reads are
// 4.9 and 9 TB/s at 64 channels and a fifth more at 128, those of the rows 5 and 3 TB/s.  For 33 to 512
// rows (75 shapes of 1 to 64 sequences, 4 to 40 heads, 2000 to 30000 tokens at each head size, every
// split of both kernels timed) the choice takes 1.05 of the best one's time at 64 channels and 1.04 at
// 128 on average, 1.16 and 1.14 at the ninth tenth, 1.33 and 1.26 at most.  Up to 32 rows there is no
// choice; above, few has no empty waves but reads each page more often (40 rows x 16 sequences x 8192
// tokens x 8 heads of 64: 34 us against 46; 128 rows x 64 sequences x 2000 tokens x 4 heads of 128: 54
// against 43, taken all the same).  768 blocks of few instead of 512 took 47 us instead of 39 for 32
// rows x 2 sequences x 30000 x 8 heads of 128; one split, two nearly full rounds of a third instead of
// five eighths of one, took tile from 748 to 598 us for 1008 rows x 31688 x 40 heads.
Plan plan(int64_t G, int64_t Hkv, int64_t dim, int64_t rows, int64_t B, int64_t max_q,
          int64_t max_kv) {
  constexpr int64_t kSlots = 512;
  const int64_t R = max_q * G, heads = B * Hkv, pages = (max_kv + kPage - 1) / kPage;
  const int64_t most = pages / 8 > 1 ? pages / 8 : 1;
  Plan best{false, 1, 1};
  double least = -1.0;
  auto offer = [&](bool few, int64_t tiles, int64_t s) {
    if (s < 1 || s > most) return;
    const int64_t items = heads * tiles;
    const double rounds = (double)((items * s + kSlots - 1) / kSlots);
    double cost = rounds * (few ? (double)((pages + 4 * s - 1) / (4 * s)) + 5.0
                                : (double)((pages + s - 1) / s) + 4.0);
    if (few) {
      const double reads = (tiles == 1 ? 2.8 : 1.5) * (double)(items * pages) / (4.0 * kSlots);
      if (cost < reads) cost = reads;
    }
    if (s > 1) cost += (few ? 4.0 : 8.0) + (double)(s * rows * G * Hkv * (dim + 2)) * 8.0 / 6.0e6;
    if (least < 0.0 || cost < least) {
      least = cost;
      best = Plan{few, tiles, s};
    }
  };
  const int64_t small = (R + kFewRows - 1) / kFewRows, large = (R + kTileRows - 1) / kTileRows;
  if (R > kFewRows)
    for (int64_t s = 1; s <= 16; ++s) offer(false, large, s);
  if (R <= kFewMost && heads * small > 0) {
    const int64_t one = kSlots / (heads * small);
    offer(true, small, 1);
    offer(true, small, one < most ? one : most);
    offer(true, small, 2 * one + 1 < most ? 2 * one + 1 : most);
  }
  return best;
}

}  // namespace

int64_t attn_workspace_bytes(int64_t rows, int64_t Hq, int64_t Hkv, int64_t dim, int64_t B,
                             int64_t max_q, int64_t max_kv) {
  const Plan p = plan(Hq / Hkv, Hkv, dim, rows, B, max_q, max_kv);
  return p.splits > 1 ? p.splits * rows * Hq * (dim + 2) * 4 : 0;
}

int64_t attn_blocks(int64_t rows, int64_t Hq, int64_t Hkv, int64_t dim, int64_t B, int64_t max_q,
                    int64_t max_kv) {
  const Plan p = plan(Hq / Hkv, Hkv, dim, rows, B, max_q, max_kv);
  return B * Hkv * p.tiles * p.splits + 8;
}

hipError_t launch_attn(const uint16_t* Q, int64_t ldq, int64_t rows, int64_t Hq, int64_t Hkv,
                       int64_t dim, const int32_t* cu, const int32_t* len, int64_t B,
                       int64_t max_q, int64_t max_kv, const int32_t* table, int64_t max_blocks,
                       int64_t n_pages, const uint8_t* kc, const uint8_t* vc, const uint8_t* ks,
                       const uint8_t* vs, float scale, int causal, uint16_t* O, int64_t ldo,
                       float* lse, void* workspace, hipStream_t s) {
  const Plan p = plan(Hq / Hkv, Hkv, dim, rows, B, max_q, max_kv);
  const float c = (float)((double)scale * 1.4426950408889634);
  const double to_ln = (double)scale / (double)c;
  AttnArgs a{Q, O, lse, (float*)workspace, cu, len, table, kc, vc, ks, vs, ldq, ldo, rows,
             max_blocks, n_pages, (int)B, (int)Hq, (int)Hkv, (int)(Hq / Hkv), (int)p.tiles,
             (int)p.splits, causal, (int)max_q, c, (float)to_ln, (float)(to_ln - (double)(float)to_ln)};
  const int64_t items = B * Hkv * p.tiles * p.splits;
  const unsigned grid = (unsigned)((items + 7) / 8 * 8);
  if (p.few && p.tiles > 1) {
    if (dim == 64)
      k_attn_few<64, true><<<grid, 256, 0, s>>>(a);
    else
      k_attn_few<128, true><<<grid, 256, 0, s>>>(a);
  } else if (p.few) {
    if (dim == 64)
      k_attn_few<64, false><<<(unsigned)items, 256, 0, s>>>(a);
    else
      k_attn_few<128, false><<<(unsigned)items, 256, 0, s>>>(a);
  } else {
    if (dim == 64)
      k_attn_tile<64><<<grid, 64 * kTileWaves, 0, s>>>(a);
    else
      k_attn_tile<128><<<grid, 64 * kTileWaves, 0, s>>>(a);
  }
  if (hipError_t e = hipGetLastError()) return e;
  if (p.splits > 1) {
    // (no sequence has more than all rows, however loose the caller's bound)
    const int64_t blocks = ((max_q < rows ? max_q : rows) * Hq + 3) / 4;
    const dim3 joins((unsigned)(blocks < kJoinMost ? blocks : kJoinMost), (unsigned)B);
    if (dim == 64)
      k_attn_join<64><<<joins, 256, 0, s>>>(a);
    else
      k_attn_join<128><<<joins, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace svdq
