// Softmax attention of bf16 query rows over the paged 8-bit cache (kv_layout.h):
//
//   z[t] = c·(q·k_t) over the tokens t the row sees,  c = scale·log2(e)
//   O = Σ_t 2^(z_t − m) v_t / l,   l = Σ_t 2^(z_t − m),   lse = ln 2·(m + log2 l)
//
// in one pass over the pages with a running maximum m (fp32 statistics and sums).  The rows of
// a key head are its query heads' rows interleaved (row = token·G + member), so grouped heads
// share every page read and single tokens still fill a matrix operand.
//
// Sᵀ = K·Qᵀ runs on the 32x32x64 f8f6f4 MFMA straight from the cached codes.  A bf16 query has
// eight significant bits, an E4M3 code four: q·2^-e = hi + 2^-4·lo splits it into two E4M3 codes
// (e from the row's maximum; what neither holds is below 2^-22 of that maximum), so the product
// costs what a bf16 product would and K needs no conversion.  The page's, the row's and the
// lo part's exponents are the MFMA's own scale operands.
//
// Oᵀ += Vᵀ·Pᵀ runs on the 32x32x16 bf16 MFMA: V's codes are widened exactly (with the page's
// exponent) and P is rounded to bf16 once, a relative 2^-9 per weight against l's unrounded
// sum.  The accumulator of Sᵀ holds, per lane, one row's weights in exactly the token order of
// the stored V, so P needs no exchange between lanes.
//
// The maximum is only raised when a tile exceeds it by more than 2^8: the weights stay below 2^8
// (exact in range for bf16 and fp32) and most tiles skip the rescaling of O.
#include "device.h"
#include "kv_layout.h"
#include "launch.h"

namespace svdq {

namespace {

typedef __attribute__((address_space(1))) void gvoid_t;
typedef __attribute__((address_space(3))) void lvoid_t;

constexpr float kNoMax = -1.0e30f;  // running maximum before the first visible token
constexpr float kRaise = 8.0f;

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
  int B, Hq, Hkv, G, tiles, splits, causal;
  float c;
};

// One sequence and key head of a block.
struct Seq {
  int64_t first;   // packed row of its first token
  int64_t n, kv;   // query tokens, cached tokens
  int b, h;
};

__device__ __forceinline__ bool sequence(const AttnArgs& a, int bh, Seq& s) {
  s.b = bh / a.Hkv;
  s.h = bh % a.Hkv;
  s.first = a.cu[s.b];
  s.n = (int64_t)a.cu[s.b + 1] - s.first;
  if (s.n <= 0 || s.first < 0 || s.first + s.n > a.rows) return false;
  s.kv = a.len[s.b];
  const int64_t room = a.max_blocks * kPage;
  s.kv = s.kv < 0 ? 0 : (s.kv > room ? room : s.kv);
  return true;
}

// Tokens [0, limit) are visible to query token i.
__device__ __forceinline__ int64_t limit_of(const AttnArgs& a, const Seq& s, int64_t i) {
  if (!a.causal) return s.kv;
  const int64_t v = s.kv - s.n + i + 1;
  return v < 0 ? 0 : v;
}

template <int DIM>
struct QueryOp {
  i32x8_t hi[DIM / 64], lo[DIM / 64];
  int s_hi, s_lo;  // E8M0 scale operands
};

// Lane (n, half) of the row's operand: channels 64s + 32·half + 0..31 of step s.
template <int DIM>
__device__ __forceinline__ void query_operand(const uint16_t* q, bool live, int half,
                                              QueryOp<DIM>& op) {
  u32x4_t w[DIM / 64][4];
  float m = 0.0f;
#pragma unroll
  for (int s = 0; s < DIM / 64; ++s)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[s][j] = u32x4_t{0u, 0u, 0u, 0u};
      if (live) w[s][j] = reinterpret_cast<const u32x4_t*>(q + 64 * s + 32 * half)[j];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        m = fmaxf(m, fmaxf(fabsf(bf16_lo(w[s][j][c])), fabsf(bf16_hi(w[s][j][c]))));
    }
  m = fmaxf(m, __shfl_xor(m, 32));
  const int e = page_exponent(m);
  const float up = two_to(-e);
#pragma unroll
  for (int s = 0; s < DIM / 64; ++s)
#pragma unroll
    for (int d = 0; d < 8; ++d) {
      const uint32_t w0 = w[s][d >> 1][2 * (d & 1)], w1 = w[s][d >> 1][2 * (d & 1) + 1];
      const float x[4] = {bf16_lo(w0) * up, bf16_hi(w0) * up, bf16_lo(w1) * up, bf16_hi(w1) * up};
      const int h = (int)e4m3_pack4(x[0], x[1], x[2], x[3]);
      op.hi[s][d] = h;
      op.lo[s][d] = (int)e4m3_pack4((x[0] - __builtin_amdgcn_cvt_f32_fp8(h, 0)) * 16.0f,
                                    (x[1] - __builtin_amdgcn_cvt_f32_fp8(h, 1)) * 16.0f,
                                    (x[2] - __builtin_amdgcn_cvt_f32_fp8(h, 2)) * 16.0f,
                                    (x[3] - __builtin_amdgcn_cvt_f32_fp8(h, 3)) * 16.0f);
    }
  op.s_hi = e + 127;
  op.s_lo = e + 123;
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

__device__ __forceinline__ float other_half(float x) {
  return __shfl_xor(x, 32);
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
// which may hold any byte, NaN codes among them.
__device__ __forceinline__ u32x4_t drop_slots(u32x4_t v, int tb, int half, int n) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    int k = n - (32 * tb + 16 * (d >> 1) + 8 * (d & 1) + 4 * half);
    k = k < 0 ? 0 : (k > 4 ? 4 : k);
    v[d] &= (uint32_t)((1ull << (8 * k)) - 1ull);
  }
  return v;
}

// One page for the wave's 32 rows.  kf(i): the lane's 16 bytes of K fragment i; vf(j, tb, g): its
// V operand of channels 32j on and tokens 32·tb + 16·g on.  EDGE: some row does not see the whole
// page; lim is the number of its tokens that the lane's row sees.  (Two instances rather than
// branches inside: the many small blocks that those leave kept the matrix and vector instructions
// of the common pages from overlapping.)
template <int DIM, bool EDGE, class KF, class VF>
__device__ __forceinline__ void page_step(State<DIM>& st, const QueryOp<DIM>& q, float c, int k_exp,
                                          int lim, int half, KF kf, VF vf) {
  f32x16_t z[2];
#pragma unroll
  for (int tb = 0; tb < 2; ++tb) {
#pragma unroll
    for (int i = 0; i < 16; ++i) z[tb][i] = 0.0f;
#pragma unroll
    for (int s = 0; s < DIM / 64; ++s) {
      const u32x4_t a0 = kf((tb * (DIM / 64) + s) * 2), a1 = kf((tb * (DIM / 64) + s) * 2 + 1);
      const i32x8_t k = {(int)a0[0], (int)a0[1], (int)a0[2], (int)a0[3],
                         (int)a1[0], (int)a1[1], (int)a1[2], (int)a1[3]};
      z[tb] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(k, q.hi[s], z[tb], 0, 0, 0, k_exp, 0,
                                                              q.s_hi);
      z[tb] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(k, q.lo[s], z[tb], 0, 0, 0, k_exp, 0,
                                                              q.s_lo);
    }
  }
  if (EDGE) {
#pragma unroll
    for (int tb = 0; tb < 2; ++tb)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (32 * tb + 8 * (i >> 2) + 4 * half + (i & 3) >= lim) z[tb][i] = -__builtin_inff();
  }
  float top = fmaxf(z[0][0], z[1][0]);
#pragma unroll
  for (int i = 1; i < 16; ++i) top = fmaxf(fmaxf(top, z[0][i]), z[1][i]);
  top = fmaxf(top, other_half(top)) * c;
  if (__builtin_amdgcn_ballot_w64(top > st.m + kRaise) != 0) {
    const float m = fmaxf(st.m, top), f = __builtin_amdgcn_exp2f(st.m - m);
#pragma unroll
    for (int j = 0; j < DIM / 32; ++j)
#pragma unroll
      for (int i = 0; i < 16; ++i) st.o[j][i] *= f;
    st.l *= f;
    st.m = m;
  }
  bf16x8_t p[4];
#pragma unroll
  for (int tb = 0; tb < 2; ++tb)
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      u32x4_t w;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(z[tb][8 * g + 2 * j], c, -st.m));
        const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(z[tb][8 * g + 2 * j + 1], c, -st.m));
        st.l += x + y;
        w[j] = pack_bf16x2(x, y);
      }
      p[2 * tb + g] = __builtin_bit_cast(bf16x8_t, w);
    }
#pragma unroll
  for (int j = 0; j < DIM / 32; ++j)
#pragma unroll
    for (int tb = 0; tb < 2; ++tb)
#pragma unroll
      for (int g = 0; g < 2; ++g)
        st.o[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf(j, tb, g), p[2 * tb + g], st.o[j], 0,
                                                          0, 0);
}

// The lane's page number and exponent bytes of logical page `at` (k | v << 8), page -1 outside
// the table's range or the cache.
__device__ __forceinline__ void page_meta(const AttnArgs& a, const Seq& s, int64_t at, int64_t end,
                                          int& page, int& exps) {
  page = -1;
  exps = 0;
  if (at < end) {
    const int p = a.table[(int64_t)s.b * a.max_blocks + at];
    if (p >= 0 && p < a.n_pages) {
      page = p;
      const int64_t i = (int64_t)p * a.Hkv + s.h;
      exps = (int)a.ks[i] | (int)a.vs[i] << 8;
    }
  }
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
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  uint16_t* o = a.O + token * a.ldo + (int64_t)head * DIM;
#pragma unroll
  for (int j = 0; j < DIM / 32; ++j)
#pragma unroll
    for (int g = 0; g < 4; ++g)
      *reinterpret_cast<uint2*>(o + 32 * j + 8 * g + 4 * half) =
          uint2{pack_bf16x2(st.o[j][4 * g] * inv, st.o[j][4 * g + 1] * inv),
                pack_bf16x2(st.o[j][4 * g + 2] * inv, st.o[j][4 * g + 3] * inv)};
  if (a.lse && half == 0)
    a.lse[token * a.Hq + head] =
        l > 0.0f ? 0.6931471805599453f * (st.m + __builtin_amdgcn_logf(l)) : -__builtin_inff();
}

// Many rows: four waves of 32 rows share each page through LDS.  K's codes are copied there as
// they are, asynchronously, one page ahead.  V's go through registers two pages ahead and are
// widened to bf16 on the way, once for the four waves (each wave widening all of them for itself
// took a third of its vector instructions).  Two images of each, one barrier a page.
constexpr int kTileWaves = 4;
constexpr int kTileRows = 32 * kTileWaves;

template <int DIM>
__global__ __launch_bounds__(64 * kTileWaves, 2) void k_attn_tile(AttnArgs a) {
  constexpr int kBytes = kPage * DIM;                       // one tensor's page
  constexpr int kCopies = kBytes / 1024 / kTileWaves;       // fragments per wave, K and V each
  __shared__ __attribute__((aligned(16))) uint8_t k_img[2][kBytes];
  __shared__ __attribute__((aligned(16))) uint8_t v_img[2][2 * kBytes];
  const int64_t total = (int64_t)a.B * a.Hkv * a.splits * a.tiles;
  const int64_t per_xcd = (total + 7) / 8;
  const int64_t item = (int64_t)(blockIdx.x % 8) * per_xcd + blockIdx.x / 8;
  if (item >= total || blockIdx.x / 8 >= per_xcd) return;
  // the last rows first: with the causal mask they see the most
  const int tile = a.tiles - 1 - (int)(item % a.tiles);
  const int split = (int)((item / a.tiles) % a.splits);
  Seq s;
  if (!sequence(a, (int)(item / a.tiles / a.splits), s)) return;
  const int64_t R = s.n * a.G, r0 = (int64_t)tile * kTileRows;
  if (r0 >= R) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, half = lane >> 5;
  const int64_t w0 = r0 + 32 * wave, row = w0 + (lane & 31);
  const bool live = row < R;
  const int64_t tok = live ? row / a.G : 0;
  const int head = s.h * a.G + (int)(live ? row % a.G : 0);

  // pages this block, and tokens the wave's first and last rows and the lane's row see
  const int64_t last = (r0 + kTileRows < R ? r0 + kTileRows : R) - 1;
  const int64_t pages = (limit_of(a, s, last / a.G) + kPage - 1) / kPage;
  const int64_t p0 = pages * split / a.splits, p1 = pages * (split + 1) / a.splits;
  const int64_t lim_row = live ? limit_of(a, s, tok) : 0;
  const int64_t lim_first = w0 < R ? limit_of(a, s, w0 / a.G) : 0;
  const int64_t w_last = (w0 + 32 < R ? w0 + 32 : R) - 1;
  const int64_t lim_last = w0 < R ? limit_of(a, s, w_last / a.G) : 0;

  QueryOp<DIM> q;
  query_operand<DIM>(a.Q + (s.first + tok) * a.ldq + (int64_t)head * DIM, live, half, q);
  State<DIM> st;
  state_init(st);

  const int64_t head_off = (int64_t)s.h * kBytes + lane * 16;
  const int64_t page_bytes = (int64_t)a.Hkv * kBytes;
  auto copy_k = [&](int page, int slot) {
    const uint8_t* src = a.kc + (int64_t)(page < 0 ? 0 : page) * page_bytes + head_off;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const int f = wave * kCopies + i;
      __builtin_amdgcn_global_load_lds((gvoid_t*)(src + f * 1024),
                                       (lvoid_t*)(&k_img[slot][f * 1024]), 16, 0, 0);
    }
  };
  u32x4_t vr[kCopies];
  auto load_v = [&](int page) {
    const uint8_t* src = a.vc + (int64_t)(page < 0 ? 0 : page) * page_bytes + head_off;
#pragma unroll
    for (int i = 0; i < kCopies; ++i)
      vr[i] = *reinterpret_cast<const u32x4_t*>(src + (wave * kCopies + i) * 1024);
  };
  // fragment f: its two 16-token steps of 1 KB each
  auto widen_v = [&](int64_t at, int exps, int slot) {
    const float scale = two_to((exps >> 8) - 127);
    const int64_t left = s.kv - at * kPage;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const int f = wave * kCopies + i;
      u32x4_t v = vr[i];
      if (left < kPage) v = drop_slots(v, f & 1, half, (int)left);
#pragma unroll
      for (int g = 0; g < 2; ++g)
        *reinterpret_cast<bf16x8_t*>(&v_img[slot][(2 * f + g) * 1024 + lane * 16]) =
            widen8(v[2 * g], v[2 * g + 1], scale);
    }
  };

  // lane i: page and exponents of logical page g0 + i (cur) and g0 + 64 + i (nxt)
  int64_t g0 = p0;
  int cur, cur_e, nxt, nxt_e;
  page_meta(a, s, g0 + lane, p1, cur, cur_e);
  page_meta(a, s, g0 + 64 + lane, p1, nxt, nxt_e);
  auto page_at = [&](int64_t i) {
    const int d = (int)(i - g0);
    return d < 64 ? __builtin_amdgcn_readlane(cur, d) : __builtin_amdgcn_readlane(nxt, d - 64);
  };
  auto exps_at = [&](int64_t i) {
    const int d = (int)(i - g0);
    return d < 64 ? __builtin_amdgcn_readlane(cur_e, d) : __builtin_amdgcn_readlane(nxt_e, d - 64);
  };
  if (p0 < p1) {
    copy_k(page_at(p0), 0);
    load_v(page_at(p0));
    widen_v(p0, exps_at(p0), 0);
    if (p0 + 1 < p1) load_v(page_at(p0 + 1));
  }
  int slot = 0;
  for (int64_t i = p0; i < p1; ++i) {
    if (i - g0 == 64) {
      g0 += 64;
      cur = nxt;
      cur_e = nxt_e;
      page_meta(a, s, g0 + 64 + lane, p1, nxt, nxt_e);
    }
    // page i has landed in LDS for every wave, and every wave is done with page i - 1
    wait_vmcnt<0>();
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (i + 1 < p1) {
      copy_k(page_at(i + 1), slot ^ 1);
      widen_v(i + 1, exps_at(i + 1), slot ^ 1);
      if (i + 2 < p1) load_v(page_at(i + 2));
    }
    const int page = __builtin_amdgcn_readlane(cur, (int)(i - g0));
    const int64_t t0 = i * kPage;
    if (page >= 0 && t0 < lim_last) {
      const int k_exp = __builtin_amdgcn_readlane(cur_e, (int)(i - g0)) & 255;
      const uint8_t *k = k_img[slot] + lane * 16, *v = v_img[slot] + lane * 16;
      auto kf = [&](int f) { return *reinterpret_cast<const u32x4_t*>(k + f * 1024); };
      auto vf = [&](int j, int tb, int g) {
        return *reinterpret_cast<const bf16x8_t*>(v + ((2 * j + tb) * 2 + g) * 1024);
      };
      if (t0 + kPage <= lim_first) {
        page_step<DIM, false>(st, q, a.c, k_exp, kPage, half, kf, vf);
      } else {
        const int64_t lr = lim_row - t0;
        page_step<DIM, true>(st, q, a.c, k_exp, (int)(lr > kPage ? kPage : lr), half, kf, vf);
      }
    }
    slot ^= 1;
  }
  const float l = st.l + other_half(st.l);
  if (live) store_row<DIM>(a, st, l, s.first + tok, head, split, half);
}

// At most 32 rows (single tokens, small groups): the four waves take every fourth page each,
// straight into registers, and join their sums through LDS.
template <int DIM>
__global__ __launch_bounds__(256, 2) void k_attn_few(AttnArgs a) {
  constexpr int kBytes = kPage * DIM;
  constexpr int kFrags = kBytes / 1024;
  __shared__ float s_o[4][DIM][33];
  __shared__ float s_m[4][32], s_l[4][32];
  const int64_t item = blockIdx.x;
  const int split = (int)(item % a.splits);
  Seq s;
  if (!sequence(a, (int)(item / a.splits), s)) return;
  int64_t R = s.n * a.G;
  R = R < 32 ? R : 32;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, half = lane >> 5, n = lane & 31;
  const bool live = n < R;
  const int64_t tok = live ? n / a.G : 0;
  const int head = s.h * a.G + (live ? n % a.G : 0);
  const int64_t pages = (limit_of(a, s, (R - 1) / a.G) + kPage - 1) / kPage;
  const int64_t p0 = pages * split / a.splits, p1 = pages * (split + 1) / a.splits;
  const int64_t lim_row = live ? limit_of(a, s, tok) : 0;
  const int64_t lim_first = limit_of(a, s, 0);

  QueryOp<DIM> q;
  query_operand<DIM>(a.Q + (s.first + tok) * a.ldq + (int64_t)head * DIM, live, half, q);
  State<DIM> st;
  state_init(st);
  const int64_t head_off = (int64_t)s.h * kBytes, page_bytes = (int64_t)a.Hkv * kBytes;
  for (int64_t g0 = p0 + wave; g0 < p1; g0 += 256) {
    int meta, meta_e;
    page_meta(a, s, g0 + 4 * lane, p1, meta, meta_e);
    for (int d = 0; d < 64 && g0 + 4 * d < p1; ++d) {
      const int page = __builtin_amdgcn_readlane(meta, d);
      if (page < 0) continue;
      const int exps = __builtin_amdgcn_readlane(meta_e, d);
      const int64_t at = (int64_t)page * page_bytes + head_off + lane * 16;
      u32x4_t kr[kFrags], vr[kFrags];
#pragma unroll
      for (int f = 0; f < kFrags; ++f) kr[f] = *reinterpret_cast<const u32x4_t*>(a.kc + at + f * 1024);
#pragma unroll
      for (int f = 0; f < kFrags; ++f) vr[f] = *reinterpret_cast<const u32x4_t*>(a.vc + at + f * 1024);
      const int64_t t0 = (g0 + 4 * d) * kPage;
      const float scale = two_to((exps >> 8) - 127);
      auto kf = [&](int f) { return kr[f]; };
      auto vf = [&](int j, int tb, int g) {
        return widen8(vr[2 * j + tb][2 * g], vr[2 * j + tb][2 * g + 1], scale);
      };
      if (t0 + kPage <= lim_first) {
        page_step<DIM, false>(st, q, a.c, exps & 255, kPage, half, kf, vf);
      } else {
        const int64_t lr = lim_row - t0, lk = s.kv - t0;
#pragma unroll
        for (int f = 0; f < kFrags; ++f) vr[f] = drop_slots(vr[f], f & 1, half, (int)(lk > kPage ? kPage : lk));
        page_step<DIM, true>(st, q, a.c, exps & 255, (int)(lr > kPage ? kPage : lr), half, kf, vf);
      }
    }
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
  for (int o = threadIdx.x; o < (int)R * DIM; o += 256) {
    const int rr = o / DIM, d = o % DIM;
    float sum = 0.0f, l = 0.0f;
    const float mm = fmaxf(fmaxf(s_m[0][rr], s_m[1][rr]), fmaxf(s_m[2][rr], s_m[3][rr]));
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      sum += s_o[w][d][rr];
      l += s_l[w][rr] * __builtin_amdgcn_exp2f(s_m[w][rr] - mm);
    }
    const int64_t token = s.first + rr / a.G;
    const int hd = s.h * a.G + rr % a.G;
    if (a.splits > 1) {
      const int64_t at = ((int64_t)split * a.rows + token) * a.Hq + hd;
      a.part[at * DIM + d] = sum;
      if (d == 0) {
        float* ml = a.part + (int64_t)a.splits * a.rows * a.Hq * DIM + at * 2;
        ml[0] = mm;
        ml[1] = l;
      }
    } else {
      a.O[token * a.ldo + (int64_t)hd * DIM + d] = f32_to_bf16(l > 0.0f ? sum / l : 0.0f);
      if (a.lse && d == 0)
        a.lse[token * a.Hq + hd] =
            l > 0.0f ? 0.6931471805599453f * (mm + __builtin_amdgcn_logf(l)) : -__builtin_inff();
    }
  }
}

// The splits of every row joined, one wave per row.  Rows past the last sequence stay as they
// are.
template <int DIM>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a) {
  const int64_t at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  const int64_t token = at / a.Hq;
  if (token >= a.rows || token >= a.cu[a.B]) return;
  const int head = (int)(at % a.Hq);
  const int64_t each = a.rows * a.Hq;
  const float* ml = a.part + a.splits * each * DIM + at * 2;
  float m = kNoMax;
  for (int i = 0; i < a.splits; ++i) m = fmaxf(m, ml[i * each * 2]);
  float l = 0.0f, o[DIM / 64] = {};
  for (int i = 0; i < a.splits; ++i) {
    const float f = __builtin_amdgcn_exp2f(ml[i * each * 2] - m);
    l += ml[i * each * 2 + 1] * f;
#pragma unroll
    for (int j = 0; j < DIM / 64; ++j)
      o[j] += a.part[(i * each + at) * DIM + (DIM / 64) * lane + j] * f;
  }
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  uint16_t* y = a.O + token * a.ldo + (int64_t)head * DIM + (DIM / 64) * lane;
  if (DIM == 128)
    *reinterpret_cast<uint32_t*>(y) = pack_bf16x2(o[0] * inv, o[DIM / 64 - 1] * inv);
  else
    y[0] = f32_to_bf16(o[0] * inv);
  if (a.lse && lane == 0)
    a.lse[at] = l > 0.0f ? 0.6931471805599453f * (m + __builtin_amdgcn_logf(l)) : -__builtin_inff();
}

struct Plan {
  bool few;
  int64_t tiles, splits;
};

// Few rows per key head go to the kernel that splits pages over its waves.  The page range is
// split further until about three blocks per CU run (768 of 256 CUs), but never below eight
// pages a block, where the join costs more than the parallelism brings.
Plan plan(int64_t G, int64_t Hkv, int64_t B, int64_t max_q, int64_t max_kv) {
  Plan p;
  p.few = max_q * G <= 32;
  p.tiles = p.few ? 1 : (max_q * G + kTileRows - 1) / kTileRows;
  const int64_t items = B * Hkv * p.tiles;
  const int64_t pages = (max_kv + kPage - 1) / kPage;
  const int64_t want = (p.few ? 768 : 512) / (items < 1 ? 1 : items);
  const int64_t most = pages / 8;
  p.splits = want < most ? want : most;
  if (p.splits < 1) p.splits = 1;
  return p;
}

}  // namespace

int64_t attn_workspace_bytes(int64_t rows, int64_t Hq, int64_t Hkv, int64_t dim, int64_t B,
                             int64_t max_q, int64_t max_kv) {
  const Plan p = plan(Hq / Hkv, Hkv, B, max_q, max_kv);
  return p.splits > 1 ? p.splits * rows * Hq * (dim + 2) * 4 : 0;
}

int64_t attn_blocks(int64_t Hq, int64_t Hkv, int64_t B, int64_t max_q, int64_t max_kv) {
  const Plan p = plan(Hq / Hkv, Hkv, B, max_q, max_kv);
  return B * Hkv * p.tiles * p.splits + 8;
}

hipError_t launch_attn(const uint16_t* Q, int64_t ldq, int64_t rows, int64_t Hq, int64_t Hkv,
                       int64_t dim, const int32_t* cu, const int32_t* len, int64_t B,
                       int64_t max_q, int64_t max_kv, const int32_t* table, int64_t max_blocks,
                       int64_t n_pages, const uint8_t* kc, const uint8_t* vc, const uint8_t* ks,
                       const uint8_t* vs, float scale, int causal, uint16_t* O, int64_t ldo,
                       float* lse, void* workspace, hipStream_t s) {
  const Plan p = plan(Hq / Hkv, Hkv, B, max_q, max_kv);
  AttnArgs a{Q, O, lse, (float*)workspace, cu, len, table, kc, vc, ks, vs, ldq, ldo, rows,
             max_blocks, n_pages, (int)B, (int)Hq, (int)Hkv, (int)(Hq / Hkv), (int)p.tiles,
             (int)p.splits, causal, (float)((double)scale * 1.4426950408889634)};
  const int64_t items = B * Hkv * p.tiles * p.splits;
  const unsigned grid = (unsigned)(p.few ? items : (items + 7) / 8 * 8);
  if (p.few) {
    if (dim == 64)
      k_attn_few<64><<<grid, 256, 0, s>>>(a);
    else
      k_attn_few<128><<<grid, 256, 0, s>>>(a);
  } else {
    if (dim == 64)
      k_attn_tile<64><<<grid, 64 * kTileWaves, 0, s>>>(a);
    else
      k_attn_tile<128><<<grid, 64 * kTileWaves, 0, s>>>(a);
  }
  if (hipError_t e = hipGetLastError()) return e;
  if (p.splits > 1) {
    const unsigned joins = (unsigned)((rows * Hq + 3) / 4);
    if (dim == 64)
      k_attn_join<64><<<joins, 256, 0, s>>>(a);
    else
      k_attn_join<128><<<joins, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace svdq
