// Attention over a prefix that several rows share, computed for all of them at
// once (the prefix of spec_verify_attention_prefix), and its join with what
// each row has of its own, for gfx950.
//
// Mathematics: S = scale Q K^T, online softmax, O = sum exp2(S - m) V, as in
// attention.hip, but one product holds the queries of all rows that begin with
// the prefix: n rows with T tokens and H / Hkv heads each are M = n T H / Hkv
// rows of it per kv head, and each key is read and widened once for MT of
// them, not once per row.  Parts join as means with the weights that they
// have.
//
// A work-group takes MT = 128 queries, 32 to a wave, and one of S parts of the
// prefix's keys, in tiles of 64.  The tile's codes come to registers while the
// tile before is worked on, are widened once for the work-group, K's to bf16
// and V's to f16 (both exact), and kept in LDS twice, so that one barrier a
// tile will do.  The products are transposed, S^T = K Q^T and O^T = V^T P^T,
// with the keys dealt so that lane group g = lane / 32 of a product has the
// scores of keys 16 g .. 16 g + 15 of 32, which is the operand that O^T needs:
// probabilities stay in their lanes.  They take their block's value scale and
// a power of two that follows the tile's largest of both, as in attention.hip,
// so that f16 holds 11 bits of them whatever the scales are.  Where some lie too
// far below the largest for f16, what it loses goes into a product of its own.

#include <algorithm>
#include <climits>

#include "matrix.h"
#include "prefix.h"

using namespace sv;
using namespace svr;

namespace {

constexpr int KEYS = 64;         // of a tile
constexpr int MT = 32 * NWAVE;   // queries of one
constexpr int RESIDENT = 2;      // work-groups of a CU, by registers and LDS
// A tile's largest probability times value scale makes 2^(MID - HALF) to 2^(MID
// + HALF + 1) in f16, which holds at least 8 bits of what is 2^LEAST and more.
constexpr float MID = 8.f, HALF = 6.f, STEP = 3.f;
constexpr int LEAST = -17;
constexpr int FRESH = -200;      // a power of two that no tile has: of sums that hold nothing yet

// A group's prefix and its rows, brought into range.
struct Group {
  int first, rows, blocks, tiles, per, parts;  // per: tiles of a part
};
__device__ __forceinline__ Group group_of(const PrefixArgs& a, int g) {
  Group r;
  r.first = min(max(a.p.starts[g], 0), a.c.B);
  r.rows = max(min(max(a.p.starts[g + 1], 0), a.c.B) - r.first, 0);
  r.blocks = min(max(a.p.blocks[g], 0), a.p.max_blocks);
  r.tiles = (int)(((int64_t)r.blocks * a.c.page + KEYS - 1) / KEYS);
  r.per = (r.tiles + a.splits - 1) / a.splits;
  r.parts = r.per ? (r.tiles + r.per - 1) / r.per : 0;
  return r;
}

typedef short i16x2 __attribute__((ext_vector_type(2)));

// Codes in f16 as bf16, which holds them exactly too, times 2^-112: the exponent of f16 in the place of bf16's, two
// instructions to two codes (none has more than 8 bits or is below 2^-9, so what the shift drops is zero).
constexpr float CODE = 0x1p112f;
__device__ __forceinline__ bf16x8 f16_as_bf16(f16x8 v) {
  u32x4 r = __builtin_bit_cast(u32x4, v);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t two = r[k];  // of r[k] itself __builtin_bit_cast takes r's first word (clang of ROCm 7.2.0)
    r[k] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(i16x2, two) >> 3) & 0x8FFF8FFFu;
  }
  return as_bf16(r);
}

// A tile's place in LDS: pieces of 8 values (16 bytes), piece p of a row at p ^
// twist, so that the rows that LDS serves together differ in their banks.
template <int D>
struct Tile {
  u32x4 k[KEYS * (D / 8)];   // [key][channel]
  u32x4 v[D * (KEYS / 8)];   // [channel][key]
  __device__ __forceinline__ static int at_k(int key, int p) { return key * (D / 8) + (p ^ (key & (D / 8 - 1))); }
  __device__ __forceinline__ static int at_v(int d, int p) { return d * (KEYS / 8) + (p ^ (d & (KEYS / 8 - 1))); }
};

// SMALL: page < 64, so the keys of a tile may lie in different pages.  Otherwise
// page, addresses and scales are the whole tile's.
template <int KIND, int D, bool SMALL>
__global__ __launch_bounds__(WG) __attribute__((amdgpu_waves_per_eu(RESIDENT, RESIDENT))) void prefix_attention_kernel(PrefixArgs a) {
  constexpr int NP = KEYS * D / 16 / WG;  // 16-byte pieces of K's codes, and of V's, per thread
  __shared__ Tile<D> sh[2];
  const int t = threadIdx.x, lane = t & 63, g = lane >> 5, col = lane & 31, w = t >> 6;

  // Which unit: part and head of a prefix first, tiles of queries, which read
  // the same keys, next to each other on one XCD.
  const int each = gridDim.x / 8, unit = (int)(blockIdx.x & 7) * each + (int)(blockIdx.x >> 3);
  int qt = unit % a.qtiles;
  const int h = unit / a.qtiles % a.c.Hkv, part = unit / a.qtiles / a.c.Hkv;
  if (part >= a.splits) return;
  // The prefix that the tile of queries belongs to: 64 of them looked up at a time.
  const int each_row = a.T * a.G;
  int which = 0;
  Group grp = {};
  for (;; which += 64) {
    if (which >= a.p.count) return;
    if (which + lane < a.p.count) grp = group_of(a, which + lane);
    else grp.rows = 0;
    const int n = (grp.rows * each_row + MT - 1) / MT;  // below 2^23
    int inc = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(inc, o, 64);
      if (lane >= o) inc += u;
    }
    const uint64_t past = __ballot(qt < inc);
    if (past) {
      const int at = __builtin_ctzll(past);
      qt -= __builtin_amdgcn_readlane(inc - n, at);
      which += at;
      break;
    }
    qt -= __builtin_amdgcn_readlane(inc, 63);
  }
#pragma unroll
  for (int k = 0; k < (int)(sizeof(Group) / 4); ++k)  // past the loop, so that they are scalars
    reinterpret_cast<int*>(&grp)[k] = __builtin_amdgcn_readlane(reinterpret_cast<int*>(&grp)[k], which & 63);
  const int tile0 = part * grp.per, tile1 = min(tile0 + grp.per, grp.tiles);
  if (tile0 >= tile1) return;

  // The lane's query.
  struct Query {
    int b, tok, head;
    bool live;
  };
  auto query_of = [&](int t, int G) {
    const int r = qt * MT + (t >> 6) * 32 + (t & 31), in = r / (a.T * G), rest = r % (a.T * G), tok = rest / G;
    const int b = grp.first + min(in, grp.rows - 1);
    return Query{b, tok, h * G + rest % G, in < grp.rows && tok < (a.qlens ? min(max(a.qlens[b], 0), a.T) : a.T)};
  };
  const auto [b, tok, head, live] = query_of(t, a.G);
  const bool queries = __any(live);  // a wave without only brings keys
  bf16x8 q[D / 16];
  {
    const uint16_t* from = a.q + b * a.q_row + tok * a.q_tok + (int64_t)head * D + g * 8;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      u32x4 x = {0, 0, 0, 0};
      if (live) x = *reinterpret_cast<const u32x4*>(from + s * 16);
      q[s] = __builtin_bit_cast(bf16x8, x);
    }
  }

  const int32_t* table = a.p.table + (int64_t)which * a.p.max_blocks;
  const int keys = grp.blocks * a.c.page;  // at most 2^24
  auto page_at = [&](int key) { return key < keys ? table[key >> a.pshift] : -1; };
  auto there = [&](int pg) { return (uint32_t)pg < (uint32_t)a.c.num_pages; };
  // The tile on its way: codes, and what goes with the lane's keys.
  constexpr int HALVES = SMALL ? 2 : 1;
  u32x4 kc[NP], vc[NP];
  float ks[HALVES], vs[HALVES];  // of the lane's keys in each half,
  bool ok[HALVES];               // where they exist
  int pv;                        // the page of the tile after it, or of its 16 keys from 16 vp on
  const int vp = t & 3;          // the keys of the thread's value pieces: 16 vp ..
  auto find = [&](int tile) {
    pv = page_at(tile * KEYS + (SMALL ? vp * 16 : 0));
  };
  auto bring = [&](int tile) {
    const int mask = a.c.page - 1;
    if constexpr (SMALL) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int s = i * WG + t, key = tile * KEYS + s / (D / 16), p = s % (D / 16);
        const int pk = __builtin_amdgcn_readlane(pv, (i * WG + __builtin_amdgcn_readfirstlane(w) * 64) / D);  // a wave's keys are of one
        kc[i] = u32x4{0, 0, 0, 0};
        if (there(pk))
          kc[i] = *reinterpret_cast<const u32x4*>(a.c.k_pages + (((int64_t)pk * a.c.Hkv + h) * a.c.page + (key & mask)) * D + p * 16);
      }
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int d = (i * WG + t) / 4;
        vc[i] = u32x4{0, 0, 0, 0};
        if (there(pv))
          vc[i] = *reinterpret_cast<const u32x4*>(a.c.v_pages + (((int64_t)pv * a.c.Hkv + h) * D + d) * a.c.page + ((tile * KEYS + vp * 16) & mask));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int p0 = __builtin_amdgcn_readlane(pv, 2 * i), p1 = __builtin_amdgcn_readlane(pv, 2 * i + 1), pl = g ? p1 : p0;
        ok[i] = there(pl);
        ks[i] = ok[i] ? a.c.k_scale[(int64_t)pl * a.c.Hkv + h] : 0.f;
        vs[i] = ok[i] ? a.c.v_scale[(int64_t)pl * a.c.Hkv + h] : 1.f;
      }
    } else {
      const int pg = __builtin_amdgcn_readfirstlane(pv);
      ok[0] = there(pg);
      if (ok[0]) {
        const int64_t at = (int64_t)pg * a.c.Hkv + h;
        const int in = (tile * KEYS) & mask;
        const uint8_t* const k0 = a.c.k_pages + (at * a.c.page + in) * D;  // 64 keys side by side
        const uint8_t* const v0 = a.c.v_pages + at * D * a.c.page + in;
        const int row = (t >> 2) * a.c.page + vp * 16;
#pragma unroll
        for (int i = 0; i < NP; ++i) kc[i] = *reinterpret_cast<const u32x4*>(k0 + (i * WG + t) * 16);
#pragma unroll
        for (int i = 0; i < NP; ++i) vc[i] = *reinterpret_cast<const u32x4*>(v0 + row + i * (WG / 4) * a.c.page);
        ks[0] = a.c.k_scale[at];
        vs[0] = a.c.v_scale[at];
      } else {
#pragma unroll
        for (int i = 0; i < NP; ++i) kc[i] = vc[i] = u32x4{0, 0, 0, 0};
        ks[0] = 0.f;
        vs[0] = 1.f;
      }
    }
  };
  auto store = [&](Tile<D>& to) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int s = i * WG + t, key = s / (D / 16), p = s % (D / 16) * 2;
      to.k[Tile<D>::at_k(key, p)] = __builtin_bit_cast(u32x4, widen<KIND>(kc[i][0], kc[i][1]));
      to.k[Tile<D>::at_k(key, p + 1)] = __builtin_bit_cast(u32x4, widen<KIND>(kc[i][2], kc[i][3]));
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int d = (i * WG + t) / 4;
      to.v[Tile<D>::at_v(d, vp * 2)] = __builtin_bit_cast(u32x4, widen_f16<KIND>(vc[i][0], vc[i][1]));
      to.v[Tile<D>::at_v(d, vp * 2 + 1)] = __builtin_bit_cast(u32x4, widen_f16<KIND>(vc[i][2], vc[i][3]));
    }
  };

  f32x16 o[D / 32];
#pragma unroll
  for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[dt][i] = 0.f;
  float m = NEG_INF, l = 0.f;  // l: of the lane's own keys
  int x = FRESH;               // the sums o are times 2^x

  find(tile0);
  bring(tile0);
  find(min(tile0 + 1, tile1 - 1));
  for (int tile = tile0; tile < tile1; ++tile) {
    Tile<D>& now = sh[(tile - tile0) & 1];
    store(now);
    float c[HALVES], v[HALVES];
    bool here[HALVES];
#pragma unroll
    for (int i = 0; i < HALVES; ++i) {
      here[i] = ok[i];
      c[i] = ok[i] ? ks[i] * a.scale2 : 0.f;
      v[i] = vs[i];
    }
    __syncthreads();
    if (tile + 1 < tile1) {
      bring(tile + 1);
      find(min(tile + 2, tile1 - 1));
    }
    if (!queries) continue;
    // Pages whose value scales are too unlike for f16 are worked on one after the other, as parts of 16 keys: those of
    // one half and lane group each.
    int passes = 1;
    if constexpr (SMALL) {
      const float e0 = value_scale(v[0], here[0]).e, e1 = value_scale(v[1], here[1]).e;
      float x0, x1;
      swap32(fmaxf(here[0] ? e0 : -150.f, here[1] ? e1 : -150.f), x0, x1);
      const float least = fmaxf(x0, x1) - ALIKE;
      if (__any((here[0] & (e0 < least)) | (here[1] & (e1 < least)))) passes = 4;
    }
    for (int pass = 0; pass < passes; ++pass) {
      bool on[HALVES];
      ValueScale sc[HALVES];
      if constexpr (SMALL) asm volatile("" : "+v"(v[0]), "+v"(v[1]) :: "memory");  // nothing is kept in registers from pass to pass
#pragma unroll
      for (int i = 0; i < HALVES; ++i) {
        on[i] = here[i] & (passes == 1 || pass == 2 * i + g);
        sc[i] = value_scale(v[i], on[i]);
      }
      f32x16 s[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int j = 0; j < 16; ++j) s[i][j] = 0.f;
        const int key = i * 32 + 16 * (col >> 2 & 1) + 4 * (col >> 3) + (col & 3);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          s[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, now.k[Tile<D>::at_k(key, ks * 2 + g)]), q[ks],
                                                         s[i], 0, 0, 0);
      }
      float mx = NEG_INF, top = HALVES == 1 ? (float)sc[0].e : -150.f;  // the tile's largest score and value scale
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float most = s[i][0];
#pragma unroll
        for (int j = 1; j < 16; ++j) most = fmaxf(most, s[i][j]);
        mx = fmaxf(mx, on[i % HALVES] ? most * c[i % HALVES] : NEG_INF);
        if (HALVES > 1) top = fmaxf(top, on[i % HALVES] ? (float)sc[i % HALVES].e : -150.f);
      }
      {
        float u, v;
        swap32(mx, u, v);
        mx = fmaxf(u, v);
        if (HALVES > 1) {
          swap32(top, u, v);
          top = fmaxf(u, v);
        }
      }
      // Maximum and power of two follow the tile (see softmax_cached in attention.hip).
      auto off_range = [&]() { return fabsf(fmaxf(mx - m, LOW) + (top - MID + (float)x)) > HALF; };
      if (__any((mx > m + GROW) | off_range())) {
        const float to = fmaxf(m, mx), f = to == NEG_INF ? 1.f : exp2_fast(m - to);
        const bool fresh = __all(m == NEG_INF);  // the sums are zero
        m = to;
        l *= f;
        const float e = fmaxf(mx - m, LOW) + top;
        const float goal = x == FRESH ? MID + HALF - GROW : e + (float)x > MID ? MID + HALF - STEP : MID - HALF + STEP;
        int dx = mx > NEG_INF && off_range() ? (int)rintf(goal - e) - x : 0;
        if (!fresh) {
#pragma unroll
          for (int dt = 0; dt < D / 32; ++dt) o[dt] *= f;
          if (__any(dx != 0)) {
            float big = 0.f;
#pragma unroll
            for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
              for (int j = 0; j < 16; ++j) big = fmaxf(big, fabsf(o[dt][j]));
            float u, v;
            swap32(big, u, v);
            big = fmaxf(u, v);
            if (big > 0.f) dx = min(dx, TOP - __builtin_amdgcn_frexp_expf(big));
            int left = dx;
            do {  // once, but between the ends of float32's range
              const int step = min(max(left, -120), 120);
              left -= step;
              const float k = ldexpf(1.f, step);
#pragma unroll
              for (int dt = 0; dt < D / 32; ++dt) o[dt] *= k;
            } while (__any(left != 0));
          }
        }
        x += dx;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // Beside sums that may not be raised further: what is added for 2^LOST is 2^-130 of the largest of them.
        const int up = max(sc[i % HALVES].e + x, LOST);
        const float off = (float)up + sc[i % HALVES].log - fmaxf(m, -FAR);  // -inf where there is no block
        float y[16], sum = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          y[j] = exp2_fast(fmaf(s[i][j], c[i % HALVES], off));
          sum += y[j];
        }
        l += ldexpf(sum * sc[i % HALVES].inv, -up);
        float low = y[0];
#pragma unroll
        for (int j = 1; j < 16; ++j) low = fminf(low, y[j]);
        f16x8 p[2];
        const bool lost = __any(on[i % HALVES] & (low < ldexpf(1.f, LEAST)));
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          union { f16x2 h[4]; f16x8 v; } z;
#pragma unroll
          for (int j = 0; j < 4; ++j) z.h[j] = __builtin_convertvector(f32x2{y[8 * u + 2 * j], y[8 * u + 2 * j + 1]}, f16x2);
          p[u] = z.v;
          // What f16 lost, in bf16, which has float32's range.  Tiles whose scores span e^13 to e^21 and more come here,
          // by where they lie in f16's: 64 x 6 tokens over 8192 keys take 79 us with scores of a standard deviation of
          // 1, 35 more with 4.
          if (lost) {
            union { bf16x2 h[4]; bf16x8 v; } r;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              r.h[j] = __builtin_convertvector(f32x2{fmaf((float)z.v[2 * j], -CODE, y[8 * u + 2 * j] * CODE),
                                                     fmaf((float)z.v[2 * j + 1], -CODE, y[8 * u + 2 * j + 1] * CODE)}, bf16x2);
            asm volatile("" ::: "memory");  // the values are read where they are used: there are no registers for more
#pragma unroll
            for (int dt = 0; dt < D / 32; ++dt)
              o[dt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                  f16_as_bf16(__builtin_bit_cast(f16x8, now.v[Tile<D>::at_v(dt * 32 + col, i * 4 + g * 2 + u)])), r.v, o[dt], 0, 0, 0);
            asm volatile("" ::: "memory");
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int dt = 0; dt < D / 32; ++dt)
            o[dt] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                __builtin_bit_cast(f16x8, now.v[Tile<D>::at_v(dt * 32 + col, i * 4 + g * 2 + u)]), p[u], o[dt], 0, 0, 0);
      }
    }
  }
  l = sum32(l);
  int again = t, group = a.G;
  asm volatile("" : "+v"(again), "+s"(group));
  const Query of = query_of(again, group);  // anew: there are no registers to keep it in
  if (!of.live) return;
  float whole = l == 0.f ? 0.f : 1.f / l;
  if (__any((x < -80) | (x > 80))) {  // by two factors, each in float32's range
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt) o[dt] *= ldexpf(1.f, -x / 2);
    whole = ldexpf(whole, -x - -x / 2);
  } else {
    whole = ldexpf(whole, -x);
  }
  const int64_t at = (((int64_t)part * a.c.B + of.b) * a.T + of.tok) * a.H + of.head;
  if (g == 0) *reinterpret_cast<float2*>(a.part_ml + at * 2) = make_float2(m, l);
#pragma unroll
  for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4 x = {o[dt][4 * i], o[dt][4 * i + 1], o[dt][4 * i + 2], o[dt][4 * i + 3]};
      *reinterpret_cast<f32x4*>(a.part_o + at * D + dt * 32 + i * 8 + g * 4) = x * whole;
    }
}

// out = the mean of what a row has of its own and of its prefix's parts, each
// with its weight; on the way too x is a mean, so that no sum of it passes
// float32's range.  D / 4 threads take every PG-th part of a token's head, four
// parts' loads at once, and the PG groups join in their order.  PG = 8 beside
// many parts (8 rows of one token, 64 parts: 5.7 us, 18 with PG = 1), 1 beside
// up to 8 (64 x 6 tokens, 5 parts: 9.6 us, 25 with PG = 8).
template <int D, int PG>
__global__ __launch_bounds__(WG) void prefix_join_kernel(PrefixArgs a) {
  constexpr int L = D / 4, ROWS = WG / (L * PG), AHEAD = 4;
  __shared__ f32x4 sx[PG > 1 ? WG : 1];
  __shared__ float2 sml[PG > 1 ? WG / L : 1];
  const int lane = threadIdx.x % L, pg = threadIdx.x / L % PG, d = lane * 4;
  const int64_t all = (int64_t)a.c.B * a.T * a.H, e = (int64_t)blockIdx.x * ROWS + threadIdx.x / (L * PG);
  const int head = (int)(e % a.H), tok = (int)(e / a.H % a.T), b = (int)min(e / a.H / a.T, (int64_t)a.c.B - 1);
  const bool live = e < all && !(a.qlens && tok >= a.qlens[b]);
  // The last group that starts at or before the row.
  int lo = 0, hi = a.p.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.p.starts[mid] <= b) lo = mid;
    else hi = mid;
  }
  const Group g = group_of(a, lo);
  const int parts = live && b >= g.first && b < g.first + g.rows ? g.parts : 0;
  const int64_t at = ((int64_t)b * a.c.Hkv + head / a.G) * a.mpad + tok * a.G + head % a.G;
  // Own part in group 0.  A part of nothing (its every score -inf) counts for nothing.
  float top = NEG_INF, sum = 0.f;
  f32x4 x = {0.f, 0.f, 0.f, 0.f};
  if (pg == 0 && live) {
    top = a.lse[at];
    x = *reinterpret_cast<const f32x4*>(a.own + e * D + d);
    sum = top == NEG_INF ? 0.f : 1.f;
  }
  const bool none = pg == 0 && top == NEG_INF;  // x is NaN there, and stays so if no part has anything
  const f32x4 kept = x;
  if (none) x = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int s0 = pg; s0 < parts; s0 += PG * AHEAD) {
    float2 ml[AHEAD];
    f32x4 y[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int64_t s = min(s0 + k * PG, parts - 1) * all + e;
      ml[k] = *reinterpret_cast<const float2*>(a.part_ml + s * 2);
      y[k] = *reinterpret_cast<const f32x4*>(a.part_o + s * D + d);
    }
    float to = top;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) to = fmaxf(to, ml[k].x);  // a part read twice is no other maximum
    const float f = top == NEG_INF ? 0.f : sum * exp2_fast(top - to);
    float w[AHEAD];
    sum = f;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const bool nothing = s0 + k * PG >= parts || (ml[k].x == NEG_INF && ml[k].y == ml[k].y);
      w[k] = nothing ? 0.f : ml[k].y * exp2_fast(ml[k].x - to);
      sum += w[k];
    }
    const float whole = sum == 0.f ? 0.f : 1.f / sum;
    x *= f * whole;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (w[k] != 0.f) x += y[k] * (w[k] * whole);
    top = to;
  }
  if constexpr (PG > 1) {
    sx[threadIdx.x] = x;
    if (lane == 0) sml[threadIdx.x / L] = make_float2(top, sum);
    __syncthreads();
    if (pg) return;
    const int first = threadIdx.x / L;
#pragma unroll
    for (int k = 1; k < PG; ++k) top = fmaxf(top, sml[first + k].x);
    float w[PG];
    sum = 0.f;
#pragma unroll
    for (int k = 0; k < PG; ++k) {
      const float2 ml = sml[first + k];
      w[k] = ml.x == NEG_INF && ml.y == 0.f ? 0.f : ml.y * exp2_fast(ml.x - top);
      sum += w[k];
    }
    const float whole = sum == 0.f ? 0.f : 1.f / sum;
    x = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < PG; ++k)
      if (w[k] != 0.f) x += sx[threadIdx.x + k * L] * (w[k] * whole);
  }
  if (!live) return;
  if (none && !(sum > 0.f)) x = kept;
  union { bf16x2 p[2]; uint2 u; } y;
  y.p[0] = __builtin_convertvector(f32x2{x[0], x[1]}, bf16x2);
  y.p[1] = __builtin_convertvector(f32x2{x[2], x[3]}, bf16x2);
  *reinterpret_cast<uint2*>(a.out + e * D + d) = y.u;
  if (d == 0 && parts) a.lse[at] = top + __builtin_amdgcn_logf(sum);
}

constexpr int join_threads(int splits) { return splits <= 8 ? 1 : 8; }  // PG
int64_t join_groups(const sv_cache& c, int T, int H, int splits) {
  const int rows = WG / (c.D / 4 * join_threads(splits));
  return ((int64_t)c.B * T * H + rows - 1) / rows;
}
template <int D, int PG>
int join(const PrefixArgs& a, hipStream_t st) {
  const int64_t groups = join_groups(a.c, a.T, a.H, a.splits);
  hipLaunchKernelGGL((prefix_join_kernel<D, PG>), dim3((uint32_t)groups), dim3(WG), 0, st, a);
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
}

template <int KIND>
auto kernel_of(const sv_cache& c) -> void (*)(PrefixArgs) {
  if (c.D == 64) return c.page < 64 ? prefix_attention_kernel<KIND, 64, true> : prefix_attention_kernel<KIND, 64, false>;
  return c.page < 64 ? prefix_attention_kernel<KIND, 128, true> : prefix_attention_kernel<KIND, 128, false>;
}

}  // namespace

namespace svr {

int check_prefix(const sv_prefix* p) {
  if (!p || !p->table || !p->blocks || !p->starts || p->count < 1 || p->max_blocks < 1) return SV_ERR_ARG;
  if (p->count > 65536 || p->max_blocks > SV_MAX_BLOCKS) return SV_ERR_UNSUPPORTED;
  const void* words[] = {p->table, p->blocks, p->starts};
  for (const void* w : words)
    if (reinterpret_cast<uintptr_t>(w) % 4) return SV_ERR_ARG;
  return SV_OK;
}

int prefix_plan(const sv_cache& c, const sv_prefix& p, int T, int H, PrefixPlan& pl) {
  const int64_t m = (int64_t)c.B * T * (H / c.Hkv);  // queries of a kv head, of all groups
  const int64_t full = (m + MT - 1) / MT;
  const int64_t qtiles = m / MT + std::min(p.count, c.B);  // each group's last tile may be a part of one
  // As many parts of the keys as fill the chip once, but none under two tiles.
  const int64_t tiles = ((int64_t)p.max_blocks * c.page + KEYS - 1) / KEYS;
  pl.splits = (int)std::max<int64_t>(1, std::min(256 * RESIDENT / (full * c.Hkv), (tiles + 1) / 2));
  const int64_t grid = qtiles * c.Hkv * pl.splits;
  if (grid > (1 << 23) || join_groups(c, T, H, pl.splits) > MAX_ITEMS / WG) return SV_ERR_UNSUPPORTED;
  pl.qtiles = (int)qtiles;
  const size_t rows = (size_t)c.B * T * H, al = 255;
  pl.o = 0;
  pl.ml = (rows * pl.splits * c.D * sizeof(float) + al) / 256 * 256;
  pl.own = pl.ml + (rows * pl.splits * 2 * sizeof(float) + al) / 256 * 256;
  pl.total = pl.own + (rows * c.D * sizeof(float) + al) / 256 * 256;
  return SV_OK;
}

int prefix_launch(const PrefixArgs& a, hipStream_t st) {
  void (*const k)(PrefixArgs) = a.c.kind == SV_E4M3 ? kernel_of<SV_E4M3>(a.c) : kernel_of<SV_INT8>(a.c);
  const int64_t grid = ((int64_t)a.qtiles * a.c.Hkv * a.splits + 7) / 8 * 8;
  hipLaunchKernelGGL(k, dim3((uint32_t)grid), dim3(WG), 0, st, a);
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
}

int prefix_join(const PrefixArgs& a, hipStream_t st) {
  const bool few = join_threads(a.splits) == 1;
  return a.c.D == 64 ? (few ? join<64, 1>(a, st) : join<64, 8>(a, st)) : (few ? join<128, 1>(a, st) : join<128, 8>(a, st));
}

}  // namespace svr
