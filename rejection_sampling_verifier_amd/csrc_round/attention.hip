// Attention of a round's new tokens over the paged 8-bit cache, the bf16 tail
// and each other (spec_verify_attention), for gfx950.
//
// Mathematics: S = scale Q K^T, online softmax (running maximum m and sum l
// per query, base 2), O = sum exp2(S - m) V.  The rows of one product are
// the M = T * H / Hkv queries that share a kv head, in tiles of 16 NQ.
//
// Work is cut along the keys as well: a row's keys come in tiles (64 cached
// tokens, or 32 tail or new tokens), and a split is a run of c tiles.  c is
// chosen on the device, from all rows' lengths, so that the splits fill the
// chip whatever the lengths; the grid is its upper bound, and work-groups
// past the last split leave.  A work-group takes one (split, kv head, row
// tile); its four waves take the split's tiles in turn, each with a softmax
// state of its own, without a barrier, and join at the end.  Splits of the
// same row are joined by a second kernel.
//
// The products are transposed, S^T = K Q^T and O^T = V^T P^T, and tile rows
// are dealt to the matrix instruction so that nothing is shuffled: lane
// group g = lane / 16 holds, for query lane % 16, the scores of keys 16 g ..
// 16 g + 15 of the tile, which is just the operand that O^T needs, and the
// keys of one lane lie in one block (16 <= page), so a block's scales are a
// factor per lane.  Codes go from memory to registers 16 bytes at a time
// and are widened to bf16 there (exact for e4m3 and int8).

#include <algorithm>
#include <cmath>
#include <climits>
#include <type_traits>

#include "cache.h"

using namespace sv;
using namespace svr;

namespace {

constexpr int TARGET = 1024;   // splits x heads x row tiles that fill the chip
constexpr int CMIN = 4;        // tiles of a split at least: one per wave
constexpr float GROW = 8.f;    // a maximum may lag this much (a factor of 256) before the sums are rescaled
constexpr float UP = 6.f;      // probabilities are held 2^6 up: with GROW, f16 takes them from 2^14 down to 2^-24
constexpr float VMIN = 0x1p-90f;  // smallest value scale told apart (see spec_verify.h)

struct AttnArgs {
  const uint16_t* q;
  const uint16_t* kn;
  const uint16_t* vn;
  int64_t q_row, q_tok, kv_row, kv_tok;
  sv_cache c;
  const int32_t* positions;
  const int32_t* blocks;
  const int32_t* parents;
  const int32_t* qlens;
  int T, H, G, M, mtiles, HM;  // HM: kv heads x row tiles
  float scale2;                // scale * log2(e)
  uint16_t* out;
  float* weights;
  float* part_o;   // [slots][MT][D] sums of unfinished rows, against their maximum
  float2* part_ml; // [slots][MT] {m, l}
  int2* info;      // [B][HM] the row's first split and their count
  float* lse;      // [B][Hkv][mtiles * MT] log2 of the softmax denominator
  float* mass;     // [B][Hkv][sub-blocks][mtiles * MT] log2 of a sub-block's sum
  int sub;         // keys of a sub-block: min(page, 64)
  int nsub;        // sub-blocks of a row's table: max_blocks * page / sub
};

__device__ __forceinline__ int query_len(const AttnArgs& a, int b) {
  return a.qlens ? min(max(a.qlens[b], 0), a.T) : a.T;
}
__device__ __forceinline__ int cached_tiles(const AttnArgs& a, int blocks) { return (blocks * a.c.page + 63) / 64; }
__device__ __forceinline__ int row_tiles(const AttnArgs& a, int b) {
  const int nq = query_len(a, b);
  if (nq == 0) return 0;
  const RowState s = row_state(a.c, a.positions, a.blocks, b);
  return cached_tiles(a, s.blocks) + (s.tail + nq + 31) / 32;
}

struct Split {
  int b, index, count, first;  // row, number within the row, the row's splits and the first one's number
  int tiles;                   // c
};

// The splits of all rows, and this work-group's unit of (split, head, row
// tile): dealt so that the row tiles of one head, which read the same keys,
// run on one XCD next to each other (hardware deals work-groups to the 8
// XCDs in turn).  hm: its head and row tile.  False past the last unit.  Every
// work-group does this for itself: the lengths are on the device.
__device__ __forceinline__ bool find_split(const AttnArgs& a, int& hm, Split& out) {
  __shared__ int sums[NWAVE];
  __shared__ Split found;
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  const int per = (a.c.B + WG - 1) / WG;
  const int r0 = min(t * per, a.c.B), r1 = min(r0 + per, a.c.B);
  int mine = 0;
  for (int r = r0; r < r1; ++r) mine += row_tiles(a, r);
  int all = mine;
#pragma unroll
  for (int o = 32; o; o >>= 1) all += __shfl_xor(all, o, 64);
  if (lane == 0) sums[w] = all;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int k = 0; k < NWAVE; ++k) total += sums[k];
  __syncthreads();
  const int c = max(CMIN, (int)(((int64_t)total * a.HM + TARGET - 1) / TARGET));
  int n = mine;
  if (per > 1) {
    n = 0;
    for (int r = r0; r < r1; ++r) n += (row_tiles(a, r) + c - 1) / c;
  } else {
    n = (mine + c - 1) / c;
  }
  int inc = n;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(inc, o, 64);
    if (lane >= o) inc += u;
  }
  if (lane == 63) sums[w] = inc;
  __syncthreads();
  int at = inc - n, splits = 0;
#pragma unroll
  for (int k = 0; k < NWAVE; ++k) {
    if (k < w) at += sums[k];
    splits += sums[k];
  }
  const int live = splits * a.HM, each = (live + 7) / 8;
  const int unit = (int)(blockIdx.x & 7) * each + (int)(blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= each || unit >= live) return false;
  const int split = unit / a.HM;
  hm = unit % a.HM;
  if (split >= at && split < at + n) {
    for (int r = r0; r < r1; ++r) {
      const int k = (per > 1 ? row_tiles(a, r) + c - 1 : mine + c - 1) / c;
      if (split < at + k) {
        found = Split{r, split - at, k, at, c};
        break;
      }
      at += k;
    }
  }
  __syncthreads();
  out = found;
  return true;
}

// ---- lanes 16 and 32 apart --------------------------------------------------
__device__ __forceinline__ void swap16(float x, float& u, float& v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  u = __uint_as_float(r[0]);
  v = __uint_as_float(r[1]);
}
__device__ __forceinline__ void swap32(float x, float& u, float& v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  u = __uint_as_float(r[0]);
  v = __uint_as_float(r[1]);
}
__device__ __forceinline__ float sum16(float x) { float u, v; swap16(x, u, v); return u + v; }
__device__ __forceinline__ float sum32(float x) { float u, v; swap32(x, u, v); return u + v; }
__device__ __forceinline__ float groups_sum(float x) { return sum32(sum16(x)); }
__device__ __forceinline__ float groups_max(float x) {
  float u, v;
  swap16(x, u, v);
  x = fmaxf(u, v);
  swap32(x, u, v);
  return fmaxf(u, v);
}

// ---- codes to 16 bits -----------------------------------------------------------
// Eight codes (two words) as a matrix operand: bf16 beside the queries, f16
// beside the probabilities.  Both kinds are exact in either.
template <int KIND>
__device__ __forceinline__ bf16x8 widen(uint32_t w0, uint32_t w1) {
  union { bf16x2 p[4]; uint32_t u[4]; bf16x8 v; } r;
  if (KIND == SV_E4M3) {
    r.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.f, false);
    r.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.f, true);
    r.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.f, false);
    r.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.f, true);
  } else {
    // An int8 is exact in bf16: the upper half of its float32.
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t w = k < 2 ? w0 : w1;
      const int s = (k & 1) * 16;
      const float x = (float)(int8_t)(w >> s), y = (float)(int8_t)(w >> (s + 8));
      r.u[k] = __builtin_amdgcn_perm(__float_as_uint(y), __float_as_uint(x), 0x07060302u);
    }
  }
  return r.v;
}
template <int KIND>
__device__ __forceinline__ f16x8 widen_f16(uint32_t w0, uint32_t w1) {
  union { f16x2 p[4]; f16x8 v; } r;
  if (KIND == SV_E4M3) {
    r.p[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.f, false);
    r.p[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.f, true);
    r.p[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.f, false);
    r.p[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.f, true);
  } else {
    // 0x6400 + u is the f16 1024 + u: with u = code + 128, minus 1152.
    const f16x2 off = {(_Float16)1152.f, (_Float16)1152.f};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t w = (k < 2 ? w0 : w1) ^ 0x80808080u;
      const uint32_t m = __builtin_amdgcn_perm(0x64646464u, w, (k & 1) ? 0x04030402u : 0x04010400u);
      r.p[k] = __builtin_bit_cast(f16x2, m) - off;
    }
  }
  return r.v;
}
__device__ __forceinline__ bf16x8 as_bf16(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

template <int D, int NQ>
struct State {
  f32x4 o[D / 16][NQ];  // O^T: lane (g, query) holds channels 16 dt + 4 g + r
  float m[NQ], l[NQ];   // l: of the lane's own keys
};

// A tile's softmax; the lane holds N scores of one query, raw, and their keys
// share the factor c and the value scale 2^lv.  The running maximum m is that
// of s c + lv, so the p = 2^(s c + lv - m + UP) that come out are the
// probabilities times the value scale, and need no product with it; l takes
// p / 2^lv.  any: the lane's keys exist.
template <int D, int NQ, int N>
__device__ __forceinline__ void softmax_tile(State<D, NQ>& st, int n, const float (&s)[N], float c, float lv,
                                             float inv, bool any, float (&p)[N], float& psum) {
  float mx = s[0];
#pragma unroll
  for (int i = 1; i < N; ++i) mx = fmaxf(mx, s[i]);
  mx = groups_max(any ? fmaf(mx, c, lv) : NEG_INF);
  if (__any(mx > st.m[n] + GROW || (st.m[n] == NEG_INF && mx > NEG_INF))) {
    const float m = fmaxf(st.m[n], mx);
    const float f = m == NEG_INF ? 1.f : exp2_fast(st.m[n] - m);
    st.m[n] = m;
    st.l[n] *= f;
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt) st.o[dt][n] *= f;
  }
  const float off = any ? lv + UP - (st.m[n] == NEG_INF ? 0.f : st.m[n]) : NEG_INF;
  const float k = any ? c : 0.f;
  psum = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    p[i] = exp2_fast(fmaf(s[i], k, off));
    psum += p[i];
  }
  psum *= inv;
  st.l[n] += psum;
}

constexpr int VPAD = 8;  // bf16 between the rows of the transposing buffer

template <int D, int NQ>
struct Lds {
  static constexpr int MT = 16 * NQ;
  union {
    uint16_t v[NWAVE][32 * (D + VPAD)];  // a wave's 32 tail or new values
    float slab[2][NWAVE][MT * 20];       // joining: 16 channels of every query, twice
  };
  float m[NWAVE][MT], l[NWAVE][MT];
  uint64_t path[64];
};

// The codes of one 64-key tile in a wave's registers.
template <int D>
struct Codes {
  u32x4 k[4][D / 64];
  u32x4 v[D / 16];
  float ks, vs;  // the scales of the lane's keys
  bool ok;       // the lane's keys exist
};

// SMALL: page < 64, so the lane groups of a tile may lie in different pages.
template <int D, bool SMALL>
struct Loader {
  const AttnArgs& a;
  const int32_t* table;
  int h, keys, g, lane;

  __device__ __forceinline__ int page_of(int group) const {
    if (group * 16 >= keys) return -1;
    return table[group * 16 / a.c.page];
  }
  // Pages of the lane's K rows and of its V keys (and scales).
  __device__ __forceinline__ int2 pages(int tile) const {
    if (SMALL) return make_int2(page_of(tile * 4 + ((lane & 15) >> 2)), page_of(tile * 4 + g));
    const int p = page_of(tile * 4);
    return make_int2(p, p);
  }
  __device__ __forceinline__ int clamp(int p) const { return (uint32_t)p < (uint32_t)a.c.num_pages ? p : 0; }
  __device__ __forceinline__ void load_k(Codes<D>& r, int tile, int2 pg) const {
    const int page = a.c.page, group = (lane & 15) >> 2;
    const int in = (SMALL ? (group * 16) % page : (tile * 64) % page + group * 16) + (lane & 3);
    const uint8_t* p = a.c.k_pages + (((int64_t)clamp(pg.x) * a.c.Hkv + h) * page + in) * D + g * 16;
#pragma unroll
    for (int ut = 0; ut < 4; ++ut)
#pragma unroll
      for (int d = 0; d < D / 64; ++d) r.k[ut][d] = *reinterpret_cast<const u32x4*>(p + ut * 4 * D + d * 64);
    const int64_t at = (int64_t)clamp(pg.y) * a.c.Hkv + h;
    r.ks = a.c.k_scale[at];
    r.ok = (uint32_t)pg.y < (uint32_t)a.c.num_pages;
  }
  __device__ __forceinline__ void load_v(Codes<D>& r, int tile, int2 pg) const {
    const int page = a.c.page;
    const int in = SMALL ? (g * 16) % page : (tile * 64) % page + g * 16;
    const int64_t at = (int64_t)clamp(pg.y) * a.c.Hkv + h;
    const uint8_t* p = a.c.v_pages + (at * D + (lane & 15)) * page + in;
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt) r.v[dt] = *reinterpret_cast<const u32x4*>(p + dt * 16 * page);
    r.vs = a.c.v_scale[at];
  }
};

template <int KIND, int D, int NQ, bool SMALL>
__global__ __launch_bounds__(WG) __attribute__((amdgpu_waves_per_eu(2))) void cache_attention_kernel(AttnArgs a) {
  constexpr int MT = 16 * NQ;
  __shared__ Lds<D, NQ> sh;
  const int t = threadIdx.x, lane = t & 63, g = lane >> 4, col = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);

  int hm = 0;
  Split sp;
  if (!find_split(a, hm, sp)) return;
  const int h = hm / a.mtiles, mt = hm % a.mtiles;
  const int b = sp.b;
  const int nq = query_len(a, b);
  if (mt * MT >= nq * a.G) return;  // a row tile of queries past the row's own
  const RowState row = row_state(a.c, a.positions, a.blocks, b);
  const int n8 = cached_tiles(a, row.blocks);
  const int nall = n8 + (row.tail + nq + 31) / 32;
  const int t0 = sp.index * sp.tiles, t1 = min(t0 + sp.tiles, nall);

  if (a.parents && t < 64) {
    // Path masks: lane v starts with itself and its parent; each step doubles
    // the length of the paths known.
    int up = -1;
    if (t > 0 && t < a.T) {
      const int p = a.parents[(int64_t)b * a.T + t];
      up = p >= 0 && p < t ? p : -1;
    }
    uint64_t m = 1ull << t;
#pragma unroll
    for (int s = 0; s < 6; ++s) {
      const int src = up < 0 ? t : up;
      const uint32_t lo = __shfl((uint32_t)m, src, 64), hi = __shfl((uint32_t)(m >> 32), src, 64);
      const int next = __shfl(up, src, 64);
      if (up >= 0) {
        m |= ((uint64_t)hi << 32) | lo;
        up = next;
      }
    }
    sh.path[t] = m;
  }
  __syncthreads();

  // Q: lane (g, query) of k-step ks = 2 d + half holds channels 64 d + 16 g +
  // 8 half + 0..7, the order in which a lane's K bytes come.
  bf16x8 q[NQ][D / 32];
  int tok[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int r = mt * MT + n * 16 + col;
    const bool live = r < nq * a.G;
    tok[n] = live ? r / a.G : 0;
    const uint16_t* p = a.q + b * a.q_row + tok[n] * a.q_tok + (int64_t)(h * a.G + (live ? r % a.G : 0)) * D + g * 16;
#pragma unroll
    for (int ks = 0; ks < D / 32; ++ks)
      q[n][ks] = as_bf16(*reinterpret_cast<const u32x4*>(p + (ks >> 1) * 64 + (ks & 1) * 8));
  }

  State<D, NQ> st;
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    st.m[n] = NEG_INF;
    st.l[n] = 0.f;
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt) st.o[dt][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  // ---- cached tiles ---------------------------------------------------------
  int i = t0 + w;
  const int end8 = min(t1, n8);
  if (i < end8) {
    const Loader<D, SMALL> ld{a, a.c.block_table + (int64_t)b * a.c.max_blocks, h, row.blocks * a.c.page, g, lane};
    Codes<D> r;
    int2 pg = ld.pages(i);
    ld.load_k(r, i, pg);
    ld.load_v(r, i, pg);
    int2 next = ld.pages(min(i + NWAVE, end8 - 1));
    for (; i < end8; i += NWAVE) {
      const int in = min(i + NWAVE, end8 - 1);  // the last tile is loaded again, not used
      f32x4 s[4][NQ];
#pragma unroll
      for (int ut = 0; ut < 4; ++ut)
#pragma unroll
        for (int n = 0; n < NQ; ++n) s[ut][n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ut = 0; ut < 4; ++ut)
#pragma unroll
        for (int ks = 0; ks < D / 32; ++ks) {
          const u32x4 v = r.k[ut][ks >> 1];
          const bf16x8 k8 = (ks & 1) ? widen<KIND>(v[2], v[3]) : widen<KIND>(v[0], v[1]);
#pragma unroll
          for (int n = 0; n < NQ; ++n) s[ut][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k8, q[n][ks], s[ut][n], 0, 0, 0);
        }
      const float c = r.ks * a.scale2, vs = r.vs < VMIN ? VMIN : r.vs;
      const float lv = __builtin_amdgcn_logf(vs), inv = __builtin_amdgcn_rcpf(vs);
      const bool ok = r.ok;
      if (!__all(ok)) {
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt)
          if (!ok) r.v[dt] = u32x4{0, 0, 0, 0};  // a code may be NaN
#pragma unroll
        for (int ut = 0; ut < 4; ++ut)
#pragma unroll
          for (int n = 0; n < NQ; ++n)
            if (!ok) s[ut][n] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
      ld.load_k(r, in, next);
      f16x8 p8[2][NQ];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float x[16], p[16], psum;
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = s[j >> 2][n][j & 3];
        softmax_tile<D, NQ, 16>(st, n, x, c, lv, ok ? inv : 0.f, ok, p, psum);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          union { f16x2 h[4]; f16x8 v; } y;
#pragma unroll
          for (int j = 0; j < 4; ++j) y.h[j] = __builtin_convertvector(f32x2{p[8 * u + 2 * j], p[8 * u + 2 * j + 1]}, f16x2);
          p8[u][n] = y.v;
        }
        if (a.mass) {
          float z = psum;
          if (a.sub > 16) z = sum16(z);
          if (a.sub > 32) z = sum32(z);
          const int at = (i * 64 + g * 16) / a.sub;
          if ((g * 16) % a.sub == 0 && i * 64 + g * 16 < row.blocks * a.c.page)
            a.mass[(((int64_t)b * a.c.Hkv + h) * a.nsub + at) * (a.mtiles * MT) + mt * MT + n * 16 + col] =
                st.m[n] - UP + __builtin_amdgcn_logf(z);  // -inf where the page does not exist
        }
      }
#pragma unroll
      for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const f16x8 v8 = widen_f16<KIND>(r.v[dt][2 * u], r.v[dt][2 * u + 1]);
#pragma unroll
          for (int n = 0; n < NQ; ++n)
            st.o[dt][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v8, p8[u][n], st.o[dt][n], 0, 0, 0);
        }
      ld.load_v(r, in, next);
      next = ld.pages(min(i + 2 * NWAVE, end8 - 1));
    }
  }

  // ---- tail and new tokens: 32 keys a tile, key 8 g + j of a tile at lane
  // group g; values are transposed through LDS ----------------------------------
  for (; i < t1; i += NWAVE) {
    const int j0 = (i - n8) * 32, have = row.tail + nq;
    auto address = [&](int j, bool val) -> const uint16_t* {
      j = min(j, have - 1);
      if (j < row.tail)
        return (val ? a.c.v_tail : a.c.k_tail) +
               (((int64_t)b * a.c.tail + (row.start + j) % a.c.tail) * a.c.Hkv + h) * D;
      return (val ? a.vn : a.kn) + b * a.kv_row + (j - row.tail) * a.kv_tok + (int64_t)h * D;
    };
    u32x4 kk[2][D / 32];
#pragma unroll
    for (int ut = 0; ut < 2; ++ut) {
      const uint16_t* p = address(j0 + (col >> 2) * 8 + ut * 4 + (col & 3), false) + g * 16;
#pragma unroll
      for (int ks = 0; ks < D / 32; ++ks) kk[ut][ks] = *reinterpret_cast<const u32x4*>(p + (ks >> 1) * 64 + (ks & 1) * 8);
    }
    uint16_t* vt = sh.v[w];
    constexpr int PER = D / 8;  // 16-byte pieces of a value
#pragma unroll
    for (int e = 0; e < 32 * PER / 64; ++e) {
      const int piece = e * 64 + lane, j = piece / PER, d = piece % PER * 8;
      u32x4 v = *reinterpret_cast<const u32x4*>(address(j0 + j, true) + d);
      if (j0 + j >= have) v = u32x4{0, 0, 0, 0};
      *reinterpret_cast<u32x4*>(vt + j * (D + VPAD) + d) = v;
    }
    f32x4 s[2][NQ];
#pragma unroll
    for (int ut = 0; ut < 2; ++ut)
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        s[ut][n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < D / 32; ++ks)
          s[ut][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(kk[ut][ks]), q[n][ks], s[ut][n], 0, 0, 0);
      }
    // Values may be anything that bf16 holds, so probabilities enter in bf16
    // too, each as the sum of two (16 bits together).
    bf16x8 hi[NQ], lo[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      float x[8], p[8], psum;
      // Seen: the tail (node < 0) and, of the new tokens, a chain's up to the
      // query's own or those of its path.  Plain bit operations: the compiler
      // made wrong code of the same condition written with branches.
      const int last = a.parents ? -1 : tok[n];
      const uint64_t path = a.parents ? sh.path[tok[n]] : 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int key = j0 + g * 8 + j, node = key - row.tail;
        const bool see = (key < have) & ((node <= last) | (bool)((path >> (node & 63)) & 1));
        x[j] = see ? s[j >> 2][n][j & 3] : NEG_INF;
      }
      softmax_tile<D, NQ, 8>(st, n, x, a.scale2, 0.f, 1.f, true, p, psum);
      union { bf16x2 h[4]; bf16x8 v; } y, z;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x2 e = {p[2 * j], p[2 * j + 1]};
        y.h[j] = __builtin_convertvector(e, bf16x2);
        z.h[j] = __builtin_convertvector(e - __builtin_convertvector(y.h[j], f32x2), bf16x2);
      }
      hi[n] = y.v;
      lo[n] = z.v;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt) {
      union { uint16_t e[8]; bf16x8 v; } v8;
#pragma unroll
      for (int j = 0; j < 8; ++j) v8.e[j] = vt[(g * 8 + j) * (D + VPAD) + dt * 16 + col];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        st.o[dt][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v8.v, lo[n], st.o[dt][n], 0, 0, 0);
        st.o[dt][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v8.v, hi[n], st.o[dt][n], 0, 0, 0);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }

  // ---- the four waves join ------------------------------------------------------
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const float l = groups_sum(st.l[n]);
    if (g == 0) {
      sh.m[w][n * 16 + col] = st.m[n];
      sh.l[w][n * 16 + col] = l;
    }
  }
  __syncthreads();
  auto joined = [&](int r, float& m, float& l) {
    m = sh.m[0][r];
#pragma unroll
    for (int k = 1; k < NWAVE; ++k) m = fmaxf(m, sh.m[k][r]);
    l = 0.f;
#pragma unroll
    for (int k = 0; k < NWAVE; ++k) l += sh.m[k][r] == NEG_INF ? 0.f : sh.l[k][r] * exp2_fast(sh.m[k][r] - m);
  };
  float f[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    float m, l;
    joined(n * 16 + col, m, l);
    f[n] = st.m[n] == NEG_INF ? 0.f : exp2_fast(st.m[n] - m);
    if (sp.count == 1) f[n] /= l;
  }
  const int64_t slot = (int64_t)sp.first + sp.index;
  const int64_t part = (slot * a.HM + hm) * MT;
  if (t == 0 && sp.index == 0) a.info[b * a.HM + hm] = make_int2(sp.first, sp.count);
  if (t < MT) {
    float m, l;
    joined(t, m, l);
    if (sp.count > 1) a.part_ml[part + t] = make_float2(m, l);
    else if (a.mass) a.lse[((int64_t)b * a.c.Hkv + h) * (a.mtiles * MT) + mt * MT + t] = m - UP + __builtin_amdgcn_logf(l);
  }
#pragma unroll
  for (int dt = 0; dt < D / 16; ++dt) {
    float* slab = sh.slab[dt & 1][w];
#pragma unroll
    for (int n = 0; n < NQ; ++n) *reinterpret_cast<f32x4*>(slab + (n * 16 + col) * 20 + g * 4) = st.o[dt][n] * f[n];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int r = n * 16 + (t >> 4), d = t & 15;
      float x = 0.f;
#pragma unroll
      for (int k = 0; k < NWAVE; ++k) x += sh.slab[dt & 1][k][r * 20 + d];
      if (sp.count > 1) {
        a.part_o[(part + r) * D + dt * 16 + d] = x;
      } else {
        const int qr = mt * MT + r;
        if (qr < nq * a.G)
          a.out[(((int64_t)b * a.T + qr / a.G) * a.H + h * a.G + qr % a.G) * D + dt * 16 + d] =
              __builtin_bit_cast(uint16_t, (__bf16)x);
      }
    }
  }
}

// Joins the splits of one row, kv head and 16 queries.
template <int D, int NQ>
__global__ __launch_bounds__(WG) void attention_combine_kernel(AttnArgs a) {
  constexpr int MT = 16 * NQ;
  extern __shared__ float fac[];  // [count][16]
  __shared__ float2 part[16][16];
  const int t = threadIdx.x;
  const int n = blockIdx.x % NQ, unit = blockIdx.x / NQ;
  const int hm = unit % a.HM, b = unit / a.HM, h = hm / a.mtiles, mt = hm % a.mtiles;
  const int r0 = mt * MT + n * 16, nq = query_len(a, b);
  if (r0 >= nq * a.G) return;
  const int2 sp = a.info[unit];
  const int first = sp.x, count = sp.y;
  if (count < 2) return;
  const float2* ml = a.part_ml + ((int64_t)first * a.HM + hm) * MT + n * 16;
  const float* po = a.part_o + (((int64_t)first * a.HM + hm) * MT + n * 16) * D;
  const int64_t step = (int64_t)a.HM * MT;
  const int r = t & 15, k = t >> 4;
  float m = NEG_INF, l = 0.f;
  for (int s = k; s < count; s += 16) {
    const float2 x = ml[s * step + r];
    if (x.x == NEG_INF) continue;
    const float big = fmaxf(m, x.x);
    l = l * (m == NEG_INF ? 0.f : exp2_fast(m - big)) + x.y * exp2_fast(x.x - big);
    m = big;
  }
  part[k][r] = make_float2(m, l);
  __syncthreads();
  m = NEG_INF;
#pragma unroll
  for (int j = 0; j < 16; ++j) m = fmaxf(m, part[j][r].x);
  l = 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) l += part[j][r].x == NEG_INF ? 0.f : part[j][r].y * exp2_fast(part[j][r].x - m);
  for (int s = k; s < count; s += 16) {
    const float x = ml[s * step + r].x;
    fac[s * 16 + r] = x == NEG_INF ? 0.f : exp2_fast(x - m) / l;
  }
  if (a.mass && k == 0) a.lse[((int64_t)b * a.c.Hkv + h) * (a.mtiles * MT) + r0 + r] = m - UP + __builtin_amdgcn_logf(l);
  __syncthreads();
  constexpr int V4 = 16 * D / 4 / WG;  // float4 per thread
#pragma unroll
  for (int v = 0; v < V4; ++v) {
    const int e = (v * WG + t) * 4, row = e / D, d = e % D, qr = r0 + row;
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int s = 0; s < count; ++s) x += *reinterpret_cast<const f32x4*>(po + s * step * D + e) * fac[s * 16 + row];
    if (qr < nq * a.G) {
      union { bf16x2 p[2]; uint2 u; } y;
      y.p[0] = __builtin_convertvector(f32x2{x[0], x[1]}, bf16x2);
      y.p[1] = __builtin_convertvector(f32x2{x[2], x[3]}, bf16x2);
      *reinterpret_cast<uint2*>(a.out + (((int64_t)b * a.T + qr / a.G) * a.H + h * a.G + qr % a.G) * D + d) = y.u;
    }
  }
}

// weights[b][t][j] = sum over heads and sub-blocks of exp2(mass - lse); the G
// heads of a kv head lie side by side (V of them a load).
template <int V>
__global__ __launch_bounds__(WG) void attention_weights_kernel(AttnArgs a, int mpad) {
  typedef float vec __attribute__((ext_vector_type(V)));
  const int64_t e = (int64_t)blockIdx.x * WG + threadIdx.x;
  const int t = (int)(e % a.T);
  const int j = (int)(e / a.T % a.c.max_blocks), b = (int)(e / a.T / a.c.max_blocks);
  if (b >= a.c.B || t >= query_len(a, b)) return;
  float x = 0.f;
  if (j < row_state(a.c, a.positions, a.blocks, b).blocks) {
    const int per = a.c.page / a.sub;
    const float* lse = a.lse + (int64_t)b * a.c.Hkv * mpad + t * a.G;
    const float* mass = a.mass + ((int64_t)b * a.c.Hkv * a.nsub + (int64_t)j * per) * mpad + t * a.G;
    for (int s = 0; s < per; ++s)
#pragma unroll 4
      for (int h = 0; h < a.c.Hkv; ++h)
#pragma unroll 2
        for (int k = 0; k < a.G; k += V) {
          const vec p = *reinterpret_cast<const vec*>(mass + ((int64_t)h * a.nsub + s) * mpad + k);
          const vec q = *reinterpret_cast<const vec*>(lse + (int64_t)h * mpad + k);
#pragma unroll
          for (int i = 0; i < V; ++i) x += exp2_fast(p[i] - q[i]);
        }
  }
  a.weights[((int64_t)b * a.T + t) * a.c.max_blocks + j] = x;
}

struct Plan {
  int nq, mtiles, grid, nsub, sub;
  size_t o, ml, info, lse, mass, total;
};

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

int make_plan(const sv_cache& c, int T, int H, bool weights, Plan& pl) {
  const int M = T * (H / c.Hkv);
  pl.nq = M <= 16 ? 1 : 2;
  const int mt = 16 * pl.nq;
  pl.mtiles = (M + mt - 1) / mt;
  const int64_t hm = (int64_t)c.Hkv * pl.mtiles;
  const int64_t most = ((int64_t)c.max_blocks * c.page + 63) / 64 + (c.page - 1 + T + 31) / 32;
  if (most * c.B > INT_MAX || hm > INT_MAX / 64) return SV_ERR_UNSUPPORTED;
  const int64_t units = std::min((int64_t)TARGET + c.B * hm, c.B * ((most + CMIN - 1) / CMIN) * hm);
  if (units > INT_MAX / 2 || c.B * hm * pl.nq > INT_MAX) return SV_ERR_UNSUPPORTED;
  pl.grid = (int)((units + 7) / 8 * 8);
  pl.sub = std::min(c.page, 64);
  const int64_t nsub = (int64_t)c.max_blocks * (c.page / pl.sub);
  pl.nsub = (int)nsub;
  size_t off = 0;
  pl.o = off;
  off = align256(off + sizeof(float) * (size_t)pl.grid * mt * c.D);
  pl.ml = off;
  off = align256(off + sizeof(float2) * (size_t)pl.grid * mt);
  pl.info = off;
  off = align256(off + sizeof(int2) * (size_t)c.B * hm);
  if (weights) {
    const size_t rows = (size_t)c.B * c.Hkv, mpad = (size_t)pl.mtiles * mt;
    pl.lse = off;
    off = align256(off + sizeof(float) * rows * mpad);
    pl.mass = off;
    off = align256(off + sizeof(float) * rows * mpad * (size_t)nsub);
    if (((int64_t)c.B * T * c.max_blocks + WG - 1) / WG > INT_MAX) return SV_ERR_UNSUPPORTED;
  }
  pl.total = off;
  return SV_OK;
}

template <int KIND, int D, int NQ>
int launch(const AttnArgs& a, const Plan& pl, hipStream_t st) {
  void (*const k)(AttnArgs) =
      a.c.page < 64 ? cache_attention_kernel<KIND, D, NQ, true> : cache_attention_kernel<KIND, D, NQ, false>;
  hipLaunchKernelGGL(k, dim3(pl.grid), dim3(WG), 0, st, a);
  if (hipGetLastError() != hipSuccess) return SV_ERR_HIP;
  hipLaunchKernelGGL((attention_combine_kernel<D, NQ>), dim3(a.c.B * a.HM * NQ), dim3(WG),
                     (TARGET / a.HM + 2) * 16 * sizeof(float), st, a);
  if (hipGetLastError() != hipSuccess) return SV_ERR_HIP;
  if (a.weights) {
    const int64_t n = (int64_t)a.c.B * a.T * a.c.max_blocks;
    void (*const wk)(AttnArgs, int) = a.G % 4 == 0   ? attention_weights_kernel<4>
                                      : a.G % 2 == 0 ? attention_weights_kernel<2>
                                                     : attention_weights_kernel<1>;
    hipLaunchKernelGGL(wk, dim3((uint32_t)((n + WG - 1) / WG)), dim3(WG), 0, st, a,
                       a.mtiles * 16 * NQ);
    if (hipGetLastError() != hipSuccess) return SV_ERR_HIP;
  }
  return SV_OK;
}
template <int KIND, int D>
int launch_rows(const AttnArgs& a, const Plan& pl, hipStream_t st) {
  return pl.nq == 1 ? launch<KIND, D, 1>(a, pl, st) : launch<KIND, D, 2>(a, pl, st);
}
template <int KIND>
int launch_dim(const AttnArgs& a, const Plan& pl, hipStream_t st) {
  return a.c.D == 64 ? launch_rows<KIND, 64>(a, pl, st) : launch_rows<KIND, 128>(a, pl, st);
}

}  // namespace

extern "C" int spec_verify_attention(const void* q, int64_t q_row, int64_t q_tok, const void* k_new, const void* v_new,
                                     int64_t kv_row, int64_t kv_tok, const sv_cache* cache, const int32_t* positions,
                                     const int32_t* blocks, const int32_t* parents, const int32_t* query_lens, int T,
                                     int H, float scale, void* out, float* weights, void* workspace,
                                     size_t* workspace_bytes, hipStream_t stream) {
  if (!workspace_bytes) return SV_ERR_ARG;
  const int bad = check_cache(cache);
  if (bad != SV_OK) return bad;
  const sv_cache& c = *cache;
  if (T < 1 || H < 1 || H % c.Hkv) return SV_ERR_ARG;
  if (T > (parents ? SV_MAX_NODES : SV_MAX_K + 1) || H > (1 << 16)) return SV_ERR_UNSUPPORTED;
  Plan pl;
  const int rc = make_plan(c, T, H, weights != nullptr, pl);
  if (rc != SV_OK) return rc;
  if (!workspace) {
    *workspace_bytes = pl.total;
    return SV_OK;
  }
  if (*workspace_bytes < pl.total) return SV_ERR_WORKSPACE;
  if (!q || !k_new || !v_new || !positions || !blocks || !out) return SV_ERR_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return SV_ERR_ARG;
  const void* aligned[] = {q, k_new, v_new, out};
  for (const void* p : aligned)
    if (reinterpret_cast<uintptr_t>(p) % 16) return SV_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(workspace) % 256 || reinterpret_cast<uintptr_t>(weights) % 4) return SV_ERR_ARG;
  constexpr int64_t FAR = int64_t(1) << 40;
  const int64_t strides[] = {q_row, q_tok, kv_row, kv_tok};
  for (int64_t s : strides)
    if (s < 0 || s > FAR || s % 8) return SV_ERR_ARG;
  AttnArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.kn = static_cast<const uint16_t*>(k_new);
  a.vn = static_cast<const uint16_t*>(v_new);
  a.q_row = q_row;
  a.q_tok = q_tok;
  a.kv_row = kv_row;
  a.kv_tok = kv_tok;
  a.c = c;
  a.positions = positions;
  a.blocks = blocks;
  a.parents = parents;
  a.qlens = query_lens;
  a.T = T;
  a.H = H;
  a.G = H / c.Hkv;
  a.M = T * a.G;
  a.mtiles = pl.mtiles;
  a.HM = c.Hkv * pl.mtiles;
  a.scale2 = scale * LOG2E;
  a.out = static_cast<uint16_t*>(out);
  a.weights = weights;
  char* ws = static_cast<char*>(workspace);
  a.part_o = reinterpret_cast<float*>(ws + pl.o);
  a.part_ml = reinterpret_cast<float2*>(ws + pl.ml);
  a.info = reinterpret_cast<int2*>(ws + pl.info);
  a.lse = weights ? reinterpret_cast<float*>(ws + pl.lse) : nullptr;
  a.mass = weights ? reinterpret_cast<float*>(ws + pl.mass) : nullptr;
  a.sub = pl.sub;
  a.nsub = pl.nsub;
  (void)hipGetLastError();
  return c.kind == SV_E4M3 ? launch_dim<SV_E4M3>(a, pl, stream) : launch_dim<SV_INT8>(a, pl, stream);
}
