// Softmax attention of bf16 query rows over the paged 4-bit cache (kv4_layout.h), by the formulas and in
// the blocks of the 8-bit cache's attention (attn.hip): one pass over the pages with a running maximum,
// Sᵀ = K·Qᵀ and Oᵀ += Vᵀ·Pᵀ on the 32x32x16 bf16 MFMA, fp32 statistics and sums.  P is rounded to bf16 once, as
// there and for the same reason (fp16 has not the range of V's powers of two): 2.1 to 2.4e-3 of O in the root
// mean square with O's own rounding, which is 1.6 to 1.7e-3 alone.
//
// The codes are widened to bf16 exactly, each block of 32 channels of a token with its own power of two.
// A lane's piece of K is one such block, so its conversions share a scale.  In a lane's piece of V the
// token changes from byte to byte and with it the scale: a byte (two channels of a token) is converted
// with its token's scale, and the two channels go to operands of two MFMAs, so that of the 64 channels
// 2m and 2m + 1 are row m of two accumulators.  That is three vector instructions for two values of V (the
// scale, the conversion, and one of the two that gather the channels), one for two of K.
//
// The scale byte 255 makes its block NaN: a row that sees it in K is NaN, one that sees it in V has NaN
// in the block's channels.  Rows that share a page with it but do not see it must not: on pages that some
// row of the block does not see whole the byte is made 0 with its codes, and the rows that see it get
// the NaN back at the end.
#include "attn_common.h"
#include "device.h"
#include "kv4_layout.h"
#include "launch.h"

namespace svdq {

namespace {

// Eight codes of one block, widened exactly: a lane's part of a step of Sᵀ.
__device__ __forceinline__ bf16x8_t widen8(uint32_t w, float scale) {
  return __builtin_bit_cast(bf16x8_t, u32x4_t{widen2(w, 0, scale), widen2(w, 1, scale),
                                              widen2(w, 2, scale), widen2(w, 3, scale)});
}

// Four tokens at two channels (a dword of V and its scales), the channels apart: words of a token
// pair each, in `even` and `odd`.
__device__ __forceinline__ void widen_pairs(uint32_t w, uint32_t scales, uint32_t (&even)[2],
                                            uint32_t (&odd)[2]) {
  uint32_t c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) c[k] = widen2(w, k, scale4(scales, k));
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    even[k] = __builtin_amdgcn_perm(c[2 * k + 1], c[2 * k], 0x05040100u);
    odd[k] = __builtin_amdgcn_perm(c[2 * k + 1], c[2 * k], 0x07060302u);
  }
}

// A dword of V's codes and its scales (tokens first .. first + 3 of the page) without the slots past
// the page's n tokens, which may hold any byte.
__device__ __forceinline__ void drop_slots(uint32_t& w, uint32_t& scales, int first, int n) {
  int k = n - first;
  k = k < 0 ? 0 : (k > 4 ? 4 : k);
  const uint32_t m = (uint32_t)((1ull << (8 * k)) - 1ull);
  w &= m;
  scales &= m;
}

// The same without its NaN blocks; `dirty` becomes true where a lane of the wave had one.
__device__ __forceinline__ void clear_nan(uint32_t& w, uint32_t& scales, bool& dirty) {
  const uint32_t nan = ((scales & 0x7F7F7F7Fu) + 0x01010101u) & scales & 0x80808080u;
  const uint32_t m = (nan >> 7) * 0xFFu;
  w &= ~m;
  scales &= ~m;
  dirty = dirty || __builtin_amdgcn_ballot_w64(nan != 0) != 0;
}

// The blocks of channels (bit b: 32 b on) in which a token that the lane's row sees, in pages [p0, p1), has
// a NaN block.
template <int DIM>
__device__ __forceinline__ uint32_t nan_blocks(const AttnArgs& a, const Seq& s, int p0, int p1, int lim_row) {
  uint32_t bad = 0;
  for (int p = p0; p < p1; ++p) {
    const int page = a.table[(int64_t)s.b * a.max_blocks + p];
    if (page < 0 || page >= a.n_pages) continue;
    const uint8_t* scales = a.vs + ((int64_t)page * a.Hkv + s.h) * (2 * DIM);
    const int64_t n = lim_row - (int64_t)p * kPage;
    for (int t = 0; t < kPage && t < n; ++t)
#pragma unroll
      for (int b = 0; b < DIM / 32; ++b)
        if (scales[v4_scale_offset(t, 32 * b)] == kNan4) bad |= 1u << b;
  }
  return bad;
}

// NaN in those channels.
template <int DIM>
__device__ __forceinline__ void restore_nan(const AttnArgs& a, const Seq& s, State<DIM>& st, int p0,
                                            int p1, int lim_row) {
  const uint32_t bad = nan_blocks<DIM>(a, s, p0, p1, lim_row);
  // accumulator j has channels 64 (j/2) + 2 m + j%2, register i of it m = 8(i/4) + 4·half + i%4
#pragma unroll
  for (int j = 0; j < DIM / 32; ++j)
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if ((bad >> (2 * (j / 2) + i / 8)) & 1) st.o[j][i] = __builtin_nanf("");
}

// Output of one row: bf16 and lse, or the unnormalised sums of a split.  Two accumulators side by side
// have eight channels in a row.
template <int DIM>
__device__ __forceinline__ void store_row(const AttnArgs& a, const State<DIM>& st, float l,
                                          int64_t token, int head, int split, int half) {
  if (a.splits > 1) {
    const int64_t at = ((int64_t)split * a.rows + token) * a.Hq + head;
    float* o = a.part + at * DIM;
#pragma unroll
    for (int u = 0; u < DIM / 64; ++u)
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int k = 0; k < 4; k += 2)
          *reinterpret_cast<f32x4_t*>(o + 64 * u + 16 * g + 8 * half + 2 * k) =
              f32x4_t{st.o[2 * u][4 * g + k], st.o[2 * u + 1][4 * g + k], st.o[2 * u][4 * g + k + 1],
                      st.o[2 * u + 1][4 * g + k + 1]};
    if (half == 0) {
      float* ml = a.part + (int64_t)a.splits * a.rows * a.Hq * DIM + at * 2;
      ml[0] = st.m;
      ml[1] = l;
    }
    return;
  }
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;
  uint16_t* o = a.O + token * a.ldo + (int64_t)head * DIM;
#pragma unroll
  for (int u = 0; u < DIM / 64; ++u)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      u32x4_t w;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = pack_bf16x2(st.o[2 * u][4 * g + k] * inv, st.o[2 * u + 1][4 * g + k] * inv);
      *reinterpret_cast<u32x4_t*>(o + 64 * u + 16 * g + 8 * half) = w;
    }
  if (a.lse && half == 0) a.lse[token * a.Hq + head] = lse_of(a, st.m, l);
}

// Many rows: the schedule of the 8-bit cache's kernel.  Four waves of 32 rows share each page through
// LDS, where it lies widened: each wave widens a quarter of K and of V on the way, V's codes loaded two
// pages ahead and K's three.  Two images of each, one barrier a page.
// Bound as there, by the power and the vector unit: 16384 rows over 16384 tokens, 40 heads of 128, 4.6 to 4.8 ms,
// 1.16 PFLOP/s; two causal streams of 4001 and 2854 rows, 32 heads on 8 of 64, 161 us.
template <int DIM>
__global__ __launch_bounds__(64 * kTileWaves, 2) void k_attn4_tile(AttnArgs a) {
  constexpr int kBytes = kPage * DIM / 2, kScales = 2 * DIM;  // one tensor's page
  constexpr int kWords = DIM / 32;                            // dwords of codes a lane, K and V each
  __shared__ __attribute__((aligned(16))) uint8_t k_img[2][4 * kBytes], v_img[2][4 * kBytes];
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

  // The wave's quarter: of 128 channels one fragment each, of 64 half of one.  In the order of the
  // operands its dword n of K is operand kWords·wave + n; V's dwords 2k and 2k + 1 are step
  // v_step + k of the accumulators v_acc and v_acc + 1.
  const int frag = DIM == 128 ? wave : wave >> 1, part = DIM == 128 ? 0 : wave & 1;
  const int v_acc = DIM == 128 ? 2 * (wave >> 1) : 0, v_step = DIM == 128 ? 2 * (wave & 1) : wave;
  const int64_t code_off = (int64_t)s.h * kBytes + frag * 1024 + lane * 16 + part * 8;
  const int64_t page_bytes = (int64_t)a.Hkv * kBytes, page_scales = (int64_t)a.Hkv * kScales;
  const uint8_t* k_src = a.kc + code_off;
  const uint8_t* v_src = a.vc + code_off;
  const uint8_t* ks_src = a.ks + (int64_t)s.h * kScales + lane * (DIM / 32) + frag;
  const uint8_t* vs_src = a.vs + (int64_t)s.h * kScales +
                          ((v_acc + ((lane >> 4) & 1)) * 2 + half) * 32 + 8 * v_step;
  uint32_t kr[kWords], vr[kWords], vsr[kWords], ksr;
  auto fetch = [](uint32_t (&r)[kWords], const uint8_t* p) {
    if (DIM == 128) {
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(p);
#pragma unroll
      for (int i = 0; i < kWords; ++i) r[i] = v[i & 3];
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      r[0] = v.x;
      r[1] = v.y;
    }
  };
  auto load_k = [&](int page) {
    page = page < 0 ? 0 : page;
    fetch(kr, k_src + page * page_bytes);
    ksr = ks_src[page * page_scales];
  };
  auto load_v = [&](int page) {
    page = page < 0 ? 0 : page;
    fetch(vr, v_src + page * page_bytes);
    fetch(vsr, vs_src + page * page_scales);
  };
  // the sequence's last page may hold fewer tokens than slots, and a page outside the cache (page 0
  // is read in its place) holds none
  const int whole = s.kv / kPage;
  // pages that every row of the block sees whole
  const int shared_pages = __builtin_amdgcn_readfirstlane(limit_of(a, s, r0 / a.G) / kPage);
  bool dirty = false;
  auto trim_v = [&](int i, int page) {
    if (i < shared_pages && page >= 0) return;
    const int n = page < 0 || i > whole ? 0 : i == whole ? s.kv % kPage : kPage;
#pragma unroll
    for (int d = 0; d < kWords; ++d) {
      drop_slots(vr[d], vsr[d], 16 * (v_step + (d >> 1)) + 8 * (d & 1) + 4 * half, n);
      if (a.causal) clear_nan(vr[d], vsr[d], dirty);
    }
  };
  uint8_t* const k_dst = &k_img[0][0] + kWords * wave * 1024 + lane * 16;
  uint8_t* const v_dst = &v_img[0][0] + (4 * v_acc + v_step) * 1024 + lane * 16;
  auto widen_k = [&](int slot, int n) {
    *reinterpret_cast<bf16x8_t*>(k_dst + slot * (4 * kBytes) + n * 1024) = widen8(kr[n], scale4(ksr, 0));
  };
  // dword n of V: half of a step's operands, which are stored with the second
  uint32_t ev[4], od[4];
  auto widen_v = [&](int slot, int n) {
    uint32_t e[2], o[2];
    widen_pairs(vr[n], vsr[n], e, o);
    ev[2 * (n & 1)] = e[0];
    ev[2 * (n & 1) + 1] = e[1];
    od[2 * (n & 1)] = o[0];
    od[2 * (n & 1) + 1] = o[1];
    if (n & 1) {
      uint8_t* to = v_dst + slot * (4 * kBytes) + (n >> 1) * 1024;
      *reinterpret_cast<u32x4_t*>(to) = u32x4_t{ev[0], ev[1], ev[2], ev[3]};
      *reinterpret_cast<u32x4_t*>(to + 4 * 1024) = u32x4_t{od[0], od[1], od[2], od[3]};
    }
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
  auto mask = [&](int i, int page, f32x16_t (&z)[2]) {
    if (page < 0 || i >= lim_first / kPage) {
      const uint32_t t0 = (uint32_t)i * kPage, lim = (uint32_t)lim_row;
      const uint32_t lr = page >= 0 && lim > t0 ? lim - t0 : 0u;
      hide(z, lr > kPage ? kPage : (int)lr, half);
    }
  };

  if (p0 < p1) {
    // lane l: page number of logical page g0 + l
    int g0 = p0, meta = page_id(a, s, g0 + lane, p1);
    auto page_at = [&](int i) { return __builtin_amdgcn_readlane(meta, (i < p1 ? i : p1 - 1) - g0); };

    f32x16_t za[2], zb[2];
    const int first = page_at(p0);
    load_k(first);
    load_v(first);
    query_check(q);
    trim_v(p0, first);
#pragma unroll
    for (int n = 0; n < kWords; ++n) widen_k(0, n);
    load_k(page_at(p0 + 1));
#pragma unroll
    for (int n = 0; n < kWords; ++n) widen_v(0, n);
    load_v(page_at(p0 + 1));
#pragma unroll
    for (int n = 0; n < kWords; ++n) widen_k(1, n);
    load_k(page_at(p0 + 2));
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
    for (int n = 0; n < kQk; ++n) product(za, n, k_operand(0, n));
    mask(p0, first, za);
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
      }
      const int p_next = page_at(i + 1);
      trim_v(i + 1, p_next);
      // From here to the masks one block without branches, its order fixed: a wave issues in
      // order, so what is to run under a matrix instruction has to stand right behind it.
      const int v_next = page_at(i + 2), k_next = page_at(i + 3);
      const uint8_t* vp = v_img[slot] + lane * 16;
      u32x4_t w[4];
      bf16x8_t kb[4], vb[4];
      float sum = 0.0f;
      // V operand n: accumulator n % (DIM/32), token step n / (DIM/32)
      auto v_read = [&](int n) {
        const int j = n % (DIM / 32), t = n / (DIM / 32);
        vb[n % 4] = *reinterpret_cast<const bf16x8_t*>(vp + (4 * j + t) * 1024);
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
      // large for the running maximum.  Then, seldom, the maximum is raised and the weights are
      // formed again.
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
        // the next page's V, then the keys of the one behind it, a dword at a time
        if (n % 2 == 0 && n < kPv / 2) widen_v(slot ^ 1, n / 2);
        if (n % 2 == 0 && n >= kPv / 2) widen_k(slot, (n - kPv / 2) / 2);
        if (n == kPv / 2) load_v(v_next);
        if (n == kPv - 1) load_k(k_next);
        __builtin_amdgcn_sched_barrier(0);
      }
      mask(i + 1, p_next, zn);
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
      restore_nan(a, s, st, p0 > shared_pages ? p0 : shared_pages, p1, lim_row);
  }
  const float l = st.l + other_half(st.l);
  if (live) store_row<DIM>(a, st, l, s.first + tok, head, split, half);
}

// Element e of a block's [rows, DIM] outputs from its waves' sums: the bf16, or a split's part.
template <int DIM, int PITCH, int WAVES>
__device__ __forceinline__ void store_joined(const AttnArgs& a, const Seq& s, const float (&s_o)[WAVES][DIM][PITCH],
                                             const float (&s_m)[WAVES][PITCH - 1],
                                             const float (&s_l)[WAVES][PITCH - 1], int e, int r0, int split) {
  const int rr = e / DIM, d = e % DIM;
  float sum = 0.0f, l = 0.0f;
  float mm = s_m[0][rr];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) mm = fmaxf(mm, s_m[w][rr]);
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
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
    a.O[token * a.ldo + (int64_t)hd * DIM + d] = f32_to_bf16(l != 0.0f ? sum / l : 0.0f);
    if (a.lse && d == 0) a.lse[token * a.Hq + hd] = lse_of(a, mm, l);
  }
}

// Few rows (single tokens, small groups): blocks of 32, whose four waves take every fourth page each,
// straight into registers, and join their sums through LDS.  Where a key head has more than 32 rows
// (TILES) its blocks are neighbours on one XCD, and the pages stay in its cache for them.  Bound by the bytes
// and the latency of a page: 32 sequences of 8191 tokens, 8 key heads of 128 with 20 rows each, 61 us, 4.7 TB/s.
template <int DIM, bool TILES>
__global__ __launch_bounds__(256, 2) void k_attn4_few(AttnArgs a) {
  constexpr int kBytes = kPage * DIM / 2, kScales = 2 * DIM, kFrags = DIM / 32;
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
  const int64_t page_bytes = (int64_t)a.Hkv * kBytes, page_scales = (int64_t)a.Hkv * kScales;
  const int64_t code_off = (int64_t)s.h * kBytes + lane * 16;
  const uint8_t* ks_src = a.ks + (int64_t)s.h * kScales + lane * (DIM / 32);
  const uint8_t* vs_src = a.vs + (int64_t)s.h * kScales + (((lane >> 4) & 1) * 2 + half) * 32;
  query_check(q);
  bool dirty = false;
  for (int g0 = p0 + wave; g0 < p1; g0 += 256) {
    // lane l: logical page g0 + 4 l
    const int meta = page_id(a, s, g0 + 4 * lane, p1);
    u32x4_t kr[kFrags], vr[kFrags], vsr[kFrags];
    uint32_t ksr;
    auto load16 = [](const uint8_t* p) {
      return TILES ? *reinterpret_cast<const u32x4_t*>(p) : load_nt(p);
    };
    auto load_k = [&](int page) {
      page = page < 0 ? 0 : page;
#pragma unroll
      for (int f = 0; f < kFrags; ++f) kr[f] = load16(a.kc + page * page_bytes + code_off + f * 1024);
      const uint8_t* p = ks_src + page * page_scales;
      ksr = DIM == 128 ? *reinterpret_cast<const uint32_t*>(p) : *reinterpret_cast<const uint16_t*>(p);
    };
    // (fragment f of V and its scales: channels 64 (f/2) on, tokens 32 (f%2) on)
    auto load_v = [&](int page) {
      page = page < 0 ? 0 : page;
#pragma unroll
      for (int f = 0; f < kFrags; ++f) {
        vr[f] = load16(a.vc + page * page_bytes + code_off + f * 1024);
        vsr[f] = *reinterpret_cast<const u32x4_t*>(vs_src + page * page_scales + (f >> 1) * 128 + (f & 1) * 16);
      }
    };
    const int count = (p1 - g0 + 3) / 4 < 64 ? (p1 - g0 + 3) / 4 : 64;
    load_k(__builtin_amdgcn_readfirstlane(meta));
    load_v(__builtin_amdgcn_readfirstlane(meta));
    for (int d = 0; d < count; ++d) {
      const int page = __builtin_amdgcn_readlane(meta, d);
      const int next = __builtin_amdgcn_readlane(meta, d + 1 < count ? d + 1 : d);
      const int t0 = (g0 + 4 * d) * kPage;
      f32x16_t z[2];
#pragma unroll
      for (int tb = 0; tb < 2; ++tb) {
#pragma unroll
        for (int i = 0; i < 16; ++i) z[tb][i] = 0.0f;
#pragma unroll
        for (int c = 0; c < DIM / 64; ++c) {
          const int f = tb * (DIM / 64) + c;
          const float scale = scale4(ksr, f);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            z[tb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                widen8(kr[f][j], scale), __builtin_bit_cast(bf16x8_t, q.w[c][j]), z[tb], 0, 0, 0);
        }
      }
      load_k(next);
      if (page < 0 || t0 > lim_first - kPage) {
        const int lr = page >= 0 ? lim_row - t0 : 0, lk = page >= 0 ? s.kv - t0 : 0;
        hide(z, lr > kPage ? kPage : (lr < 0 ? 0 : lr), half);
#pragma unroll
        for (int f = 0; f < kFrags; ++f)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t w = vr[f][k], sc = vsr[f][k];
            drop_slots(w, sc, 32 * (f & 1) + 16 * (k >> 1) + 8 * (k & 1) + 4 * half, lk > kPage ? kPage : lk);
            if (a.causal) clear_nan(w, sc, dirty);
            vr[f][k] = w;
            vsr[f][k] = sc;
          }
      }
      raise(st, largest(z, a.c));
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const bf16x8_t p = weights(st, z, t >> 1, t & 1, a.c);
#pragma unroll
        for (int u = 0; u < DIM / 64; ++u) {
          const int f = 2 * u + (t >> 1), k = 2 * (t & 1);
          uint32_t e0[2], o0[2], e1[2], o1[2];
          widen_pairs(vr[f][k], vsr[f][k], e0, o0);
          widen_pairs(vr[f][k + 1], vsr[f][k + 1], e1, o1);
          st.o[2 * u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
              __builtin_bit_cast(bf16x8_t, u32x4_t{e0[0], e0[1], e1[0], e1[1]}), p, st.o[2 * u], 0, 0, 0);
          st.o[2 * u + 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
              __builtin_bit_cast(bf16x8_t, u32x4_t{o0[0], o0[1], o1[0], o1[1]}), p, st.o[2 * u + 1], 0, 0, 0);
        }
      }
      load_v(next);
    }
  }
  if (dirty) {
    const int part = lim_first / kPage;
    restore_nan(a, s, st, p0 > part ? p0 : part, p1, lim_row);
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
      s_o[wave][64 * (j >> 1) + 2 * (8 * (i >> 2) + 4 * half + (i & 3)) + (j & 1)][n] = st.o[j][i] * f;
  __syncthreads();
  for (int at = threadIdx.x; at < R * DIM; at += 256) store_joined<DIM, 33, 4>(a, s, s_o, s_m, s_l, at, r0, split);
}

// At most 16 rows of a key head (single tokens whose query heads share it): the same on the 16x16x32 MFMA, in
// half the matrix instructions, exponentials and registers, so that with blocks of four waves three a SIMD have
// their loads on the way and not two (of eight: two, one block a CU).  A block takes `chunk` pages (attn_chunk), its waves every eighth or fourth of them.
//
// The lanes of K's and V's operands differ from the stored ones in one bit of the lane and one of the dword,
// which lane swaps of the codes exchange: lane 16·g + n of K has token n of sixteen at 8 channels, of V
// four tokens 4·g on at channels 2·n, 2·n + 1 of 32.  V's scales come as a word a lane and pass through LDS.
//
// 32 sequences of 8191 tokens, 8 key heads of 128 with 5 rows each: 50 to 53 us in graphs over caches of more
// than 1 GB in turn, 5.7 to 5.4 TB/s, bound by the bytes (with the 32 rows' kernel 54.6).  Ragged ones, 195 MB of
// cache, 45.5 to 46.8 (53.7), 4.2 TB/s: the blocks of the longest sequences last longest, and such a block is
// bound by its instructions, 460 of the vector unit a page, 0.9 us of a SIMD (a lone block of four waves or of
// eight walks 64 pages in 15 us).  On average the SIMDs are busy 0.36 of the time, and the waves wait for loads
// 0.4 of theirs.
constexpr int kLeastRows = 16;

struct Words2 {
  uint32_t a, b;
};
__device__ __forceinline__ Words2 swap16(uint32_t x, uint32_t y) {
  const auto r = __builtin_amdgcn_permlane16_swap(x, y, false, false);
  return Words2{r[0], r[1]};
}
__device__ __forceinline__ Words2 swap32(uint32_t x, uint32_t y) {
  const auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
  return Words2{r[0], r[1]};
}
// Of the four lanes of a row.
__device__ __forceinline__ float row_largest(float m) {
  const Words2 a = swap16(__float_as_uint(m), __float_as_uint(m));
  m = fmaxf(__uint_as_float(a.a), __uint_as_float(a.b));
  const Words2 b = swap32(__float_as_uint(m), __float_as_uint(m));
  return fmaxf(__uint_as_float(b.a), __uint_as_float(b.b));
}

template <int DIM, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 3) void k_attn4_row16(AttnArgs a) {
  constexpr int kBytes = kPage * DIM / 2, kScales = 2 * DIM, kFrags = DIM / 32;
  __shared__ float s_o[WAVES][DIM][kLeastRows + 1];
  __shared__ float s_m[WAVES][kLeastRows], s_l[WAVES][kLeastRows];
  __shared__ __attribute__((aligned(16))) uint32_t s_vs[WAVES][DIM / 2];
  const int split = (int)(blockIdx.x % a.splits), bh = (int)(blockIdx.x / a.splits);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, n = lane & 15;
  // lane l: table entry of the logical page at + WAVES·l (past the table the last), the page if it exists
  auto look_up = [&](int at) {
    const int64_t i = (int64_t)at + WAVES * lane;
    return a.table[(int64_t)(bh / a.Hkv) * a.max_blocks + (i < a.max_blocks ? i : a.max_blocks - 1)];
  };
  auto existing = [&](int page) { return page < a.n_pages ? page : -1; };
  // (asked for beside the lengths, for the case that nothing is split: a block starts with a chain of loads)
  int meta = look_up(wave);
  Seq s;
  if (!sequence(a, bh, s)) return;
  const int R = s.q * a.G;
  const bool live = n < R;
  const int tok = (live ? n : 0) / a.G;
  const int head = s.h * a.G + (live ? n : 0) % a.G;
  const int pages = (int)(((int64_t)limit_of(a, s, (R - 1) / a.G) + kPage - 1) / kPage);
  const int chunk = a.splits > 1 ? __builtin_amdgcn_readfirstlane(attn_chunk(a)) : 0;
  const int p0 = split * chunk;
  if (split > 0 && p0 >= pages) return;   // (the join knows)
  const int p1 = split == a.splits - 1 || pages - p0 < chunk ? pages : p0 + chunk;
  const int lim_row = live ? limit_of(a, s, tok) : 0;
  const int lim_first = limit_of(a, s, 0);

  // step (c, j): channels 64 c + 32 (g/2) + 16 j + 8 (g%2) on
  u32x4_t q[DIM / 64][2];
  const uint16_t* const q_row = a.Q + (int64_t)(s.first + tok) * a.ldq + (int64_t)head * DIM + 32 * (g >> 1) + 8 * (g & 1);
  // Oᵀ: accumulator 4 u + 2 b + k has channels 64 u + 32 b + 2 (4 g + i) + k
  f32x4_t o[DIM / 16];
#pragma unroll
  for (int j = 0; j < DIM / 16; ++j) o[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  float m = kNoMax, l = 0.0f;

  const int64_t page_bytes = (int64_t)a.Hkv * kBytes, page_scales = (int64_t)a.Hkv * kScales;
  const int64_t code_off = (int64_t)s.h * kBytes + lane * 16;
  const uint8_t* ks_src = a.ks + (int64_t)s.h * kScales + lane * (DIM / 32);
  // V's scales: word lane = [block of channels][t/4 %2][t/16][t/8 %2], in LDS the last two in the other order
  const int word = lane % (DIM / 2);
  const uint8_t* vs_src = a.vs + (int64_t)s.h * kScales + 4 * word;
  uint32_t* const vs_put = &s_vs[wave][(word & ~7) + 4 * (word & 1) + ((word >> 1) & 3)];
  const uint32_t* const vs_get = &s_vs[wave][8 * (g & 1) + 4 * (g >> 1)];
  bool dirty = false;
  u32x4_t kr[kFrags], vr[kFrags];
  uint32_t ksr = 0, vsr = 0;
  auto load_k = [&](int page) {
    page = page < 0 ? 0 : page;
#pragma unroll
    for (int f = 0; f < kFrags; ++f) kr[f] = load_nt(a.kc + page * page_bytes + code_off + f * 1024);
    const uint8_t* p = ks_src + page * page_scales;
    ksr = DIM == 128 ? *reinterpret_cast<const uint32_t*>(p) : *reinterpret_cast<const uint16_t*>(p);
  };
  auto load_v = [&](int page) {
    page = page < 0 ? 0 : page;
#pragma unroll
    for (int f = 0; f < kFrags; ++f) vr[f] = load_nt(a.vc + page * page_bytes + code_off + f * 1024);
    vsr = *reinterpret_cast<const uint32_t*>(vs_src + page * page_scales);
  };
  int g0 = p0 + wave;
  // (a wave without pages too: the counts of loads under way stay known)
  meta = existing(a.splits > 1 ? look_up(g0) : meta);
  load_k(__builtin_amdgcn_readfirstlane(meta));
#pragma unroll
  for (int c = 0; c < DIM / 64; ++c)
#pragma unroll
    for (int j = 0; j < 2; ++j) q[c][j] = *reinterpret_cast<const u32x4_t*>(q_row + 64 * c + 16 * j);
  load_v(__builtin_amdgcn_readfirstlane(meta));
  {
    // an infinity or NaN in the row makes all of it NaN (and so every score)
    uint32_t most = 0;
#pragma unroll
    for (int c = 0; c < DIM / 64; ++c)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) most = max_bf16x2(most, q[c][j][k] & 0x7FFF7FFFu);
    most = max_bf16x2(most, most >> 16) & 0xFFFFu;
    const Words2 u = swap16(most, most);
    most = u.a > u.b ? u.a : u.b;
    const Words2 v = swap32(most, most);
    if ((v.a > v.b ? v.a : v.b) >= kInfBits) {
#pragma unroll
      for (int c = 0; c < DIM / 64; ++c)
#pragma unroll
        for (int j = 0; j < 2; ++j) q[c][j] = u32x4_t{0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu};
    }
  }
  for (; g0 < p1; g0 += 64 * WAVES) {
    const int count = (p1 - g0 + WAVES - 1) / WAVES < 64 ? (p1 - g0 + WAVES - 1) / WAVES : 64;
    for (int d = 0; d < count; ++d) {
      const int page = __builtin_amdgcn_readlane(meta, d);
      const int next = __builtin_amdgcn_readlane(meta, d + 1 < count ? d + 1 : d);
      const int t0 = (g0 + WAVES * d) * kPage;
      // z[t]: tokens 16 t + 4 g + i
      f32x4_t z[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) z[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      const Words2 sk = swap16(ksr, ksr);
#pragma unroll
      for (int f = 0; f < kFrags; ++f) {
        const int tb = f / (DIM / 64), c = f % (DIM / 64);
        const float s0 = scale4(sk.a, f), s1 = scale4(sk.b, f);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const Words2 w = swap16(kr[f][2 * j], kr[f][2 * j + 1]);
          const bf16x8_t x = __builtin_bit_cast(bf16x8_t, q[c][j]);
          z[2 * tb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8(w.a, s0), x, z[2 * tb], 0, 0, 0);
          z[2 * tb + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8(w.b, s1), x, z[2 * tb + 1], 0, 0, 0);
        }
      }
      load_k(next);
      *vs_put = vsr;
      __builtin_amdgcn_wave_barrier();   // (LDS keeps a wave's order)
      const bool part = page < 0 || t0 > lim_first - kPage;
      if (part) {
        asm volatile("");   // (a branch, not 32 instructions on every page)
        const int lr = page >= 0 ? lim_row - t0 : 0;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (16 * t + 4 * g + i >= lr) z[t][i] = -__builtin_inff();
      }
      float top = fmaxf(z[0][0], z[0][1]);
#pragma unroll
      for (int i = 2; i < 16; i += 2) top = fmaxf(fmaxf(top, z[i >> 2][i & 3]), z[i >> 2][(i & 3) + 1]);
      top = row_largest(top) * a.c;
      if (__builtin_amdgcn_ballot_w64(top > m + kRaise) != 0) {
        const float up = fmaxf(m, top), f = __builtin_amdgcn_exp2f(m - up);
#pragma unroll
        for (int j = 0; j < DIM / 16; ++j) o[j] *= f;
        l *= f;
        m = up;
      }
      u32x4_t p[2];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(z[j >> 1][2 * (j & 1)], a.c, -m));
        const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(z[j >> 1][2 * (j & 1) + 1], a.c, -m));
        l += x + y;
        p[j >> 2][j & 3] = pack_bf16x2(x, y);
      }
      __builtin_amdgcn_sched_barrier(0);
      const int lk = page < 0 ? 0 : s.kv - t0 > kPage ? kPage : s.kv - t0;
#pragma unroll
      for (int u = 0; u < DIM / 64; ++u) {
        // w[b][t]: tokens 16 t + 4 g on at channels 64 u + 32 b + 2 n, + 1
        uint32_t w[2][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const u32x4_t& v = vr[2 * u + (t >> 1)];
          const Words2 x = swap32(v[2 * (t & 1)], v[2 * (t & 1) + 1]), y = swap16(x.a, x.b);
          w[0][t] = y.a;
          w[1][t] = y.b;
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          u32x4_t sv = *reinterpret_cast<const u32x4_t*>(vs_get + 16 * (2 * u + b));
          if (part) {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              uint32_t sc = sv[t];
              drop_slots(w[b][t], sc, 16 * t + 4 * g, lk);
              if (a.causal) clear_nan(w[b][t], sc, dirty);
              sv[t] = sc;
            }
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t e0[2], o0[2], e1[2], o1[2];
            widen_pairs(w[b][2 * k], sv[2 * k], e0, o0);
            widen_pairs(w[b][2 * k + 1], sv[2 * k + 1], e1, o1);
            const bf16x8_t weight = __builtin_bit_cast(bf16x8_t, p[k]);
            const int at = 2 * (2 * u + b);
            o[at] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bf16x8_t, u32x4_t{e0[0], e0[1], e1[0], e1[1]}), weight, o[at], 0, 0, 0);
            o[at + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bf16x8_t, u32x4_t{o0[0], o0[1], o1[0], o1[1]}), weight, o[at + 1], 0, 0, 0);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      load_v(next);
    }
    if (g0 + 64 * WAVES < p1) {
      meta = existing(look_up(g0 + 64 * WAVES));
      load_k(__builtin_amdgcn_readfirstlane(meta));
      load_v(__builtin_amdgcn_readfirstlane(meta));
    }
  }
  if (dirty) {
    const int whole = lim_first / kPage;
    const uint32_t bad = nan_blocks<DIM>(a, s, p0 > whole ? p0 : whole, p1, lim_row);
#pragma unroll
    for (int j = 0; j < DIM / 16; ++j)
      if ((bad >> (j / 2)) & 1) o[j] = o[j] * __builtin_nanf("");
  }
  // join the waves
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (g == 0) {
    s_m[wave][n] = m;
    s_l[wave][n] = l;
  }
  __syncthreads();
  float most = s_m[0][n];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) most = fmaxf(most, s_m[w][n]);
  const float f = __builtin_amdgcn_exp2f(m - most);
#pragma unroll
  for (int j = 0; j < DIM / 16; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) s_o[wave][32 * (j >> 1) + 2 * (4 * g + i) + (j & 1)][n] = o[j][i] * f;
  __syncthreads();
  for (int at = threadIdx.x; at < R * DIM; at += 64 * WAVES)
    store_joined<DIM, kLeastRows + 1, WAVES>(a, s, s_o, s_m, s_l, at, 0, split);
}

}  // namespace

// Up to 16 rows of a key head: blocks of eight waves for at most one a CU, the pages of the longest sequence
// split where that leaves some idle (a second block a CU takes longer: 32 ragged sequences of up to 8191
// tokens, 8 key heads of 128, 58 us for 47), blocks of four, three a CU, beyond (64 sequences of 4096 tokens,
// 16 heads of 64, 57 us for 71; the other way round 32 ragged ones 56 for 47).  At least eight pages a
// block, one for each wave, and none split below 24: the join is a launch (one head over 16 pages 10.7 us in two
// splits and 9.5 in one, over 32 11.5 in four and 13.4).  More rows: as for the 8-bit cache, by constants that are
// fitted to its kernels and not to these: 1008 causal rows of 40 heads of 128 over 31688 tokens take 631 us (8
// bits: 613), two sequences of 256 rows of 24 heads over 16384 149 (135), four of 128 rows of 40 / 8 heads over
// 8192 102 (101), 16 of 40 rows of 8 heads of 64 over 8192 39 (46), 17 rows of 40 heads of 128 over 30000 44 (61).
static AttnPlan attn4_plan(int64_t G, int64_t Hkv, int64_t dim, int64_t rows, int64_t B, int64_t max_q,
                           int64_t max_kv) {
  constexpr int64_t kCus = 256, kLeast = 8, kLeastSplit = 24;
  if (max_q * G > kLeastRows) return attn_plan(G, Hkv, dim, rows, B, max_q, max_kv);
  const int64_t pages = (max_kv + kPage - 1) / kPage;
  int64_t splits = kCus / (B * Hkv);
  if (splits > pages / kLeast) splits = pages / kLeast;
  if (pages < kLeastSplit) splits = 1;
  return AttnPlan{true, 1, splits > 1 ? splits : 1, (int)kLeast};
}

int64_t attn4_workspace_bytes(int64_t rows, int64_t Hq, int64_t Hkv, int64_t dim, int64_t B,
                              int64_t max_q, int64_t max_kv) {
  const AttnPlan p = attn4_plan(Hq / Hkv, Hkv, dim, rows, B, max_q, max_kv);
  return p.splits > 1 ? p.splits * rows * Hq * (dim + 2) * 4 : 0;
}

int64_t attn4_blocks(int64_t rows, int64_t Hq, int64_t Hkv, int64_t dim, int64_t B, int64_t max_q,
                     int64_t max_kv) {
  const AttnPlan p = attn4_plan(Hq / Hkv, Hkv, dim, rows, B, max_q, max_kv);
  return B * Hkv * p.tiles * p.splits + 8;
}

hipError_t launch_attn4(const uint16_t* Q, int64_t ldq, int64_t rows, int64_t Hq, int64_t Hkv,
                        int64_t dim, const int32_t* cu, const int32_t* len, int64_t B,
                        int64_t max_q, int64_t max_kv, const int32_t* table, int64_t max_blocks,
                        int64_t n_pages, const uint8_t* kc, const uint8_t* vc, const uint8_t* ks,
                        const uint8_t* vs, float scale, int causal, uint16_t* O, int64_t ldo,
                        float* lse, void* workspace, hipStream_t s) {
  const AttnPlan p = attn4_plan(Hq / Hkv, Hkv, dim, rows, B, max_q, max_kv);
  const AttnArgs a = attn_args(Q, ldq, rows, Hq, Hkv, cu, len, B, max_q, table, max_blocks, n_pages,
                               kc, vc, ks, vs, scale, causal, O, ldo, lse, workspace, p, 1.0f);
  const int64_t items = B * Hkv * p.tiles * p.splits;
  const unsigned grid = (unsigned)((items + 7) / 8 * 8);
  if (p.chunk > 0) {
    if (items > 256) {
      if (dim == 64)
        k_attn4_row16<64, 4><<<(unsigned)items, 256, 0, s>>>(a);
      else
        k_attn4_row16<128, 4><<<(unsigned)items, 256, 0, s>>>(a);
    } else {
      if (dim == 64)
        k_attn4_row16<64, 8><<<(unsigned)items, 512, 0, s>>>(a);
      else
        k_attn4_row16<128, 8><<<(unsigned)items, 512, 0, s>>>(a);
    }
  } else if (p.few && p.tiles > 1) {
    if (dim == 64)
      k_attn4_few<64, true><<<grid, 256, 0, s>>>(a);
    else
      k_attn4_few<128, true><<<grid, 256, 0, s>>>(a);
  } else if (p.few) {
    if (dim == 64)
      k_attn4_few<64, false><<<(unsigned)items, 256, 0, s>>>(a);
    else
      k_attn4_few<128, false><<<(unsigned)items, 256, 0, s>>>(a);
  } else {
    if (dim == 64)
      k_attn4_tile<64><<<grid, 64 * kTileWaves, 0, s>>>(a);
    else
      k_attn4_tile<128><<<grid, 64 * kTileWaves, 0, s>>>(a);
  }
  if (hipError_t e = hipGetLastError()) return e;
  return p.splits > 1 ? launch_attn_join(a, dim, s) : hipSuccess;
}

}  // namespace svdq
