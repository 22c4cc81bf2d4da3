// Attention of a step's new tokens over the paged 8-bit cache, the bf16 tail
// and each other (spec_verify_attention), for gfx950.
//
// Mathematics: S = scale Q K^T, online softmax (running maximum m and sum l
// per query, base 2), O = sum exp2(S - m) V.  The rows of one product are
// the M = T * H / Hkv queries that share a kv head, in tiles of 16 NQ.
//
// Work is cut along the keys as well: a row's keys come in tiles (32 tail or
// new tokens, then 64 cached ones each); for each row tile of queries the
// tiles of all rows that have such queries stand in a line, and each
// work-group takes a run of c of them for one kv head, whatever rows they
// belong to.  c is found on the device, from the rows' lengths, so that the
// work-groups fill the chip once and get equal work.  The four waves take a
// segment's tiles in turn, each with a softmax state and a part of LDS of its
// own, without a barrier, and join at the segment's end.
// The parts of a row that several work-groups hold are joined by the last of
// them to arrive, in the order of the parts, so that the result does not
// depend on who that is.  Parts go through write-through stores and counters
// that are zero between calls (see sv_device.h).
//
// The products are transposed, S^T = K Q^T and O^T = V^T P^T, and tile rows
// are dealt to the matrix instruction so that nothing is shuffled: lane
// group g = lane / 16 holds, for query lane % 16, the scores of keys 16 g ..
// 16 g + 15 of the tile, which is just the operand that O^T needs, and the
// keys of one lane lie in one block (16 <= page), so a block's scales are a
// factor per lane.  Codes go from memory to LDS 16 bytes a lane and are
// widened in the operands' registers, K's to bf16 and V's to f16 (both exact
// for e4m3 and int8); the next tile's are on their way meanwhile.

#include <algorithm>
#include <cmath>
#include <climits>
#include <type_traits>

#include "cache.h"

using namespace sv;
using namespace svr;

namespace {

constexpr int CUS = 256;
constexpr int MAX_GROUP = 256;   // query heads per kv head
constexpr int MAX_MTILES = (MAX_GROUP * (SV_MAX_K + 1) + 15) / 16;
constexpr int CMIN = 4;        // tiles of a run at least: one per wave

// Work-groups of the attention kernel per CU: waves per SIMD by its registers.
// Two, each with a whole tile on its way, beat three of half the registers
// (16 rows of up to 16k tokens, one query each, D = 128: 76 against 83 us).
constexpr int RESIDENT = 2;
constexpr float GROW = 4.f;    // a maximum may lag this much (a factor of 16) before the sums are rescaled
// Where f16 takes probabilities times value scales: a tile's largest of both
// makes 2^(MID - HALF) to 2^(MID + HALF + 1), at most 2^15 and, as f16's
// smallest step is 2^-24, a probability is off by at most 2^-21 of the
// largest, where scales differ by a factor of 2^(ALIKE + 1) by 2^-16.
constexpr float MID = 5.f, HALF = 9.f, STEP = 3.f;
// Tail and new tokens: 2^x that the sums take, so that 2^GROW times 320 of
// them times the largest bf16 stay below 2^127.
constexpr int NEAR_X = -18;
constexpr float ALIKE = 4.f;   // value scales of one tile that differ by 2^5 and more need more range than f16 has
constexpr float LOW = -110.f;  // scores further below the maximum count as this far, so that 2^x stays in float32's range
constexpr float VMIN = 0x1p-126f;  // smallest value scale told apart (see spec_verify.h)
constexpr float FAR = 0x1p127f;  // in place of an infinite -m, where every score is -inf
constexpr int TOP = 100;       // sums are not raised above 2^TOP
constexpr int LOST = -40;

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
  int T, H, G, mtiles;
  int even;                    // runs of all row tiles' lines, per head, if no line ended with a part of one; with
                               // c = ceil(tiles / even) tiles to a run, the sum over lines of ceil(line / c) is at
                               // most even + mtiles - 1, for which the grid is made
  float scale2;                // scale * log2(e)
  uint16_t* out;
  float* weights;
  unsigned* arrived; // [B][Hkv][mtiles] parts that are there; zero between calls
  float* part_o;     // [parts][Hkv][mtiles][MT][D] sums of a part of a row, against its maximum
  float* part_ml;    // [parts][Hkv][mtiles][MT][2] {m, l}
  float* lse;      // [B][Hkv][mtiles * MT] log2 of the softmax denominator
  float* mass;     // [B][Hkv][sub-blocks][mtiles * MT] log2 of a sub-block's sum
  int pshift;      // log2 page
  int sshift;      // log2 of a sub-block's keys: min(page, 64)
  int nsub;        // sub-blocks of a row's table: max_blocks * page / sub
};

__device__ __forceinline__ int query_len(const AttnArgs& a, int b) {
  return a.qlens ? min(max(a.qlens[b], 0), a.T) : a.T;
}
// A row as the lines of tiles have it.
struct Row {
  int n;      // its tiles: near, then cached
  int near;   // those of the tail and the new tokens
  int reps;   // row tiles that hold queries
  int nq, blocks, tail, start;
};
template <int MT>
__device__ __forceinline__ Row row_of(const AttnArgs& a, int b) {
  Row r;
  const RowState s = row_state(a.c, a.positions, a.blocks, b);
  r.nq = query_len(a, b);
  r.blocks = s.blocks;
  r.tail = s.tail;
  r.start = s.start;
  r.near = (s.tail + r.nq + 31) / 32;
  r.n = r.near + (s.blocks * a.c.page + 63) / 64;
  r.reps = (r.nq * a.G + MT - 1) / MT;
  return r;
}

// A work-group's run: tiles [at, end) of row tile mt's line for head h, the
// first of them in row b, whose tiles begin at `begin`; c tiles per run.
struct Run {
  int b, begin, at, end, c, h, mt;
};

// Inclusive prefix over the work-group's threads, and the total.
__device__ __forceinline__ int scan(int v, int* sums, int& total) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(v, o, 64);
    if (lane >= o) v += u;
  }
  if (lane == 63) sums[w] = v;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int k = 0; k < NWAVE; ++k) {
    if (k < w) v += sums[k];
    total += sums[k];
  }
  __syncthreads();
  return v;
}

// This work-group's run.  With U(mt) runs in row tile mt's line (fewer the
// larger mt, as rows with fewer queries have fewer row tiles), units are
// numbered by run, then head, then row tile, and dealt so that neighbours,
// which read the same keys, are on one XCD (hardware deals work-groups to the
// 8 XCDs in turn).  False past the last unit.  Every work-group does this for
// itself: the lengths are on the device.
template <int MT>
__device__ __forceinline__ bool find_run(const AttnArgs& a, Row* rows, Run& out) {
  if (a.c.B <= 64 && a.mtiles == 1) {
    // A row per lane, by every wave for itself: no barriers.
    const int lane = threadIdx.x & 63;
    Row x = {};
    if (lane < a.c.B) x = row_of<MT>(a, lane);
    if (threadIdx.x < 64) rows[lane] = x;
    const int n = x.reps > 0 ? x.n : 0;
    int inc = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(inc, o, 64);
      if (lane >= o) inc += u;
    }
    const int total = __builtin_amdgcn_readlane(inc, 63);
    const int c = max(CMIN, (total + a.even - 1) / a.even);
    const int units = (total + c - 1) / c * a.c.Hkv, each = (units + 7) / 8;
    const int unit = (int)(blockIdx.x & 7) * each + (int)(blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= each || unit >= units) return false;
    const int at = unit / a.c.Hkv * c;
    const int b = __builtin_ctzll(__ballot(at < inc));
    out = Run{b, __builtin_amdgcn_readlane(inc - n, b), at, min(at + c, total), c, unit % a.c.Hkv, 0};
    return true;
  }
  __shared__ int sums[NWAVE];
  __shared__ int lines[MAX_MTILES + 1];  // tiles of row tile mt's line
  __shared__ int place[2];
  __shared__ Run found;
  const int t = threadIdx.x;
  const int per = (a.c.B + WG - 1) / WG;
  const int r0 = min(t * per, a.c.B), r1 = min(r0 + per, a.c.B);
  int total, begin = 0, mine = 0, c, run, mt = 0;
  int n1 = 0, reps1 = 0;  // of the thread's row, where it has one
  if (a.mtiles == 1) {
    for (int r = r0; r < r1; ++r) {
      const Row x = row_of<MT>(a, r);
      mine += x.reps > 0 ? x.n : 0;
    }
    begin = scan(mine, sums, total) - mine;
    c = max(CMIN, (total + a.even - 1) / a.even);
  } else {
    for (int k = t; k <= a.mtiles; k += WG) lines[k] = 0;
    __syncthreads();
    for (int r = r0; r < r1; ++r) {
      const Row x = row_of<MT>(a, r);
      if (x.reps > 0) atomicAdd(&lines[x.reps - 1], x.n);
      n1 = x.n;
      reps1 = x.reps;
      mine += x.n * x.reps;
    }
    scan(mine, sums, total);
    c = max(CMIN, (total + a.even - 1) / a.even);
    if (t == 0)
      for (int k = a.mtiles - 2; k >= 0; --k) lines[k] += lines[k + 1];
    __syncthreads();
    total = lines[0];
  }
  // Units of the runs before `run`, per head: the sum over mt of min(U(mt), run).
  auto before = [&](int r) {
    if (a.mtiles == 1) return min((total + c - 1) / c, r);
    int n = 0;
    for (int k = 0; k < a.mtiles; ++k) n += min((lines[k] + c - 1) / c, r);
    return n;
  };
  const int u0 = (total + c - 1) / c;
  const int units = before(u0) * a.c.Hkv, each = (units + 7) / 8;
  const int unit = (int)(blockIdx.x & 7) * each + (int)(blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= each || unit >= units) return false;
  int h;
  if (a.mtiles == 1) {
    run = unit / a.c.Hkv;
    h = unit % a.c.Hkv;
  } else {
    for (int r = t; r < u0; r += WG) {
      const int lo = before(r) * a.c.Hkv, hi = before(r + 1) * a.c.Hkv;
      if (unit >= lo && unit < hi) {
        place[0] = r;
        place[1] = unit - lo;
      }
    }
    __syncthreads();
    run = place[0];
    const int live = before(run + 1) - before(run);  // row tiles that have this run
    h = place[1] / live;
    mt = place[1] % live;
    total = lines[mt];
    mine = 0;
    if (per == 1) mine = reps1 > mt ? n1 : 0;
    else
      for (int r = r0; r < r1; ++r) {
        const Row x = row_of<MT>(a, r);
        mine += x.reps > mt ? x.n : 0;
      }
    int all;
    begin = scan(mine, sums, all) - mine;
  }
  const int at = run * c;
  if (at >= begin && at < begin + mine) {
    int r = r0;
    if (per > 1)
      for (; r < r1; ++r) {
        const Row x = row_of<MT>(a, r);
        const int n = x.reps > mt ? x.n : 0;
        if (at < begin + n) break;
        begin += n;
      }
    found = Run{r, begin, at, min(at + c, total), c, h, mt};
  }
  __syncthreads();
  out = found;
  return true;
}

// Two neighbouring words published, and read, at once.
__device__ __forceinline__ void pub_store2(float* p, float x, float y) {
  const uint64_t v = (uint64_t)__float_as_uint(y) << 32 | __float_as_uint(x);
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 pub_load2(const float* p) {
  const uint64_t v = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
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
  f32x4 o[D / 16][NQ];  // O^T times 2^x: lane (g, query) holds channels 16 dt + 4 g + r
  float m[NQ], l[NQ];   // l: of the lane's own keys
  int xs[(NQ + 1) / 2];  // x, two 16-bit numbers to a word: beside 64 queries every register counts

  __device__ __forceinline__ int x(int n) const { return n & 1 ? xs[n / 2] >> 16 : (int)(int16_t)xs[n / 2]; }
  __device__ __forceinline__ void set_x(int n, int v) {
    xs[n / 2] = n & 1 ? (xs[n / 2] & 0xFFFF) | v << 16 : (xs[n / 2] & ~0xFFFF) | (v & 0xFFFF);
  }
};

// The running maximum follows mx, a tile's largest score.
template <int D, int NQ>
__device__ __forceinline__ float follow(State<D, NQ>& st, int n, float mx) {
  const float m = fmaxf(st.m[n], mx);
  const float f = m == NEG_INF ? 1.f : exp2_fast(st.m[n] - m);
  st.m[n] = m;
  st.l[n] *= f;
  return f;
}
template <int D, int NQ>
__device__ __forceinline__ bool lags(const State<D, NQ>& st, int n, float mx) {
  return mx > st.m[n] + GROW;
}

// The softmax of a tile of tail and new tokens; the lane holds 8 scores of one
// query, raw.  p: probabilities times 2^NEAR_X.
template <int D, int NQ>
__device__ __forceinline__ void softmax_near(State<D, NQ>& st, int n, const float (&s)[8], float c, float (&p)[8]) {
  float mx = s[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) mx = fmaxf(mx, s[i]);
  mx = groups_max(mx * c);
  if (__any(lags(st, n, mx))) {
    const float f = follow(st, n, mx);
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt) st.o[dt][n] *= f;
  }
  const float off = NEAR_X - fmaxf(st.m[n], -FAR);
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    p[i] = exp2_fast(fmaf(s[i], c, off));
    sum += p[i];
  }
  st.l[n] = fmaf(sum, (float)(1 << -NEAR_X), st.l[n]);
}

// A block's value scale as 2^e f, 1 <= f < 2.
struct ValueScale {
  int e;
  float log, inv;  // log2 f, 1 / f; -inf and 0 where there is no block
};
__device__ __forceinline__ ValueScale value_scale(float v, bool any) {
  v = !any ? 1.f : v < VMIN ? VMIN : v;
  const float f = 2.f * __builtin_amdgcn_frexp_mantf(v);
  return {__builtin_amdgcn_frexp_expf(v) - 1, any ? __builtin_amdgcn_logf(f) : NEG_INF, any ? __builtin_amdgcn_rcpf(f) : 0.f};
}

// The softmax of a cached tile; the lane holds 16 scores of one query, raw,
// whose keys share the factor c and the value scale v; top: the largest v.e
// of the tile's.  any: the lane's keys exist.  p: probabilities times the
// value scale times 2^x, or, where scales are unlike, times f alone; psum: the
// sum of the probabilities.
//
// f16 has five bits of exponent, so x follows the tile's largest score and
// scale (their product lies at 2^e before x), up and down, the float32 sums
// with it, whatever the scales of the tiles before were.  x and the running
// maximum move apart: a probability in the denominator does not depend on any
// value scale.  18 binades of e are one x, so it moves seldom: 32 trees of 61
// nodes take 166 us with scores of a standard deviation of 1, 172 with 4 and
// 182 with 16; 64 chains over 8192 keys 122, 124 and 125.  One maximum of score
// and scale together takes 156 and 119 us at any, and loses every cached value
// of a wave that is small beside its tail's or another block's.
template <int D, int NQ>
__device__ __forceinline__ void softmax_cached(State<D, NQ>& st, int n, const float (&s)[16], float c, const ValueScale& v,
                                               float top, bool any, bool unlike, float (&p)[16], float& psum) {
  float mx = s[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) mx = fmaxf(mx, s[i]);
  mx = groups_max(any ? mx * c : NEG_INF);
  auto off_range = [&]() { return fabsf(fmaxf(mx - st.m[n], LOW) + (top - MID + (float)st.x(n))) > HALF; };
  // Plain bit operations: branches would part the tile's instructions.
  if (__any(lags(st, n, mx) | off_range())) {
    const bool fresh = __all(st.m[n] == NEG_INF);  // the sums are zero
    const float f = follow(st, n, mx);
    const float e = fmaxf(mx - st.m[n], LOW) + top;
    // No further than needed, so that high and low tiles in turn find one x;
    // the first tile with room for a maximum that lags.
    const float y = e + (float)st.x(n);
    const float to = y > MID ? MID + HALF - STEP : st.x(n) == NEAR_X ? MID + HALF - GROW : MID - HALF + STEP;
    int dx = mx > NEG_INF && off_range() ? (int)rintf(to - e) - st.x(n) : 0;
    if (!fresh) {
#pragma unroll
      for (int dt = 0; dt < D / 16; ++dt) st.o[dt][n] *= f;
      if (__any(dx != 0)) {
        float big = 0.f;
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
          for (int r = 0; r < 4; ++r) big = fmaxf(big, fabsf(st.o[dt][n][r]));
        if (__any(big == __builtin_inff())) {  // an infinite tail or new value: the others go by themselves
          big = 0.f;
#pragma unroll
          for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float y = fabsf(st.o[dt][n][r]);
              big = fmaxf(big, y == __builtin_inff() ? 0.f : y);
            }
        }
        big = groups_max(big);
        if (big > 0.f) dx = min(dx, TOP - __builtin_amdgcn_frexp_expf(big));
        int left = dx;
        do {  // once, but between the ends of float32's range
          const int step = min(max(left, -120), 120);
          left -= step;
          const float k = ldexpf(1.f, step);
#pragma unroll
          for (int dt = 0; dt < D / 16; ++dt) st.o[dt][n] *= k;
        } while (__any(left != 0));
      }
    }
    st.set_x(n, st.x(n) + dx);
  }
  // Beside sums that may not be raised further, f16 takes a tile for zeros (of
  // 2^LOST 2^GROW it knows no step); its probabilities still count.
  const int up = unlike ? 0 : max(v.e + st.x(n), LOST);
  const float off = (float)up + v.log - fmaxf(st.m[n], -FAR);
  psum = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    p[i] = exp2_fast(fmaf(s[i], c, off));
    psum += p[i];
  }
  psum = ldexpf(psum * v.inv, -up);
  st.l[n] += psum;
}

typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int VPAD = 8;  // bf16 between the rows of the transposing buffer

constexpr int ROWS = 64;  // rows that are looked up at once

template <int D, int NQ>
struct Lds {
  static constexpr int MT = 16 * NQ;
  union {
    struct {
      u32x4 k[4 * D];  // a wave's codes of a cached tile,
      union {
        u32x4 v[4 * D];
        uint16_t near[32 * (D + VPAD)];  // or its 32 tail or new values
      };
    } wave[NWAVE];
    float o[NWAVE][MT * (D + 4)];        // joining: the waves' sums
  };
  float m[NWAVE][MT], l[NWAVE][MT];
  uint64_t path[64];
  Row rows[ROWS];
  int last;
};

// The codes of one 64-key tile in a wave's registers.
template <int D>
struct Codes {
  u32x4 k[4][D / 64];
  u32x4 v[D / 16];
  float ks, vs;  // the scales of the lane's keys
  bool ok;       // the lane's keys exist
};

// Brings a wave's tiles: from memory into its own part of LDS, in pieces of
// 16 bytes with four neighbouring lanes 64 bytes side by side, and from there
// into the operands' registers, where 16 lanes hold 16 keys.  Loads straight
// into those registers take the vector cache four times the cycles, and can
// begin only when the registers are free (trees of 64 nodes: 174 us against
// 160; chains that read 623 MB: 139 against 120).
// K has D / 16 pieces to a key, V four to a channel.  Piece p lies at place
// p ^ twist, so that the eight lanes that LDS serves together differ in
// their banks.
// SMALL: page < 64, so the lane groups of a tile may lie in different pages.
template <int D, bool SMALL>
struct Loader {
  static constexpr int KP = D / 16;  // pieces of a key, and copies of 64 pieces, of K and of V
  const AttnArgs& a;
  const int32_t* table;
  int h, keys, g, lane;

  __device__ __forceinline__ int page_of(int group) const {
    if (group * 16 >= keys) return -1;
    return table[group * 16 >> a.pshift];
  }
  // The pages of a tile: lane l has that of 16-key group l / 16.
  __device__ __forceinline__ int pages(int tile) const { return page_of(tile * 4 + (SMALL ? g : 0)); }
  __device__ __forceinline__ int clamp(int p) const { return (uint32_t)p < (uint32_t)a.c.num_pages ? p : 0; }
  __device__ __forceinline__ static int twist_k(int key) {
    return KP == 8 ? (key & 3) | (key >> 4 & 1) << 2 : (key >> 1 & 1) | (key >> 4 & 1) << 1;
  }
  __device__ __forceinline__ static int twist_v(int d) { return d >> 1 & 3; }
  template <int CPOL>
  __device__ __forceinline__ static void bring(const uint8_t* from, u32x4* to) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                     (__attribute__((address_space(3))) void*)to, 16, 0, CPOL);
  }
  template <int CPOL>
  __device__ __forceinline__ void copy_k(u32x4* to, int tile, int pg) const {
    const int page = a.c.page, base = (tile * 64) & (page - 1);
#pragma unroll
    for (int k = 0; k < KP; ++k) {
      const int s = k * 64 + lane, key = s / KP, p = (s % KP) ^ twist_k(key);
      const int own = __builtin_amdgcn_readlane(pg, SMALL ? k * 4 / KP * 16 : 0);
      const int in = SMALL ? key & (page - 1) : key;
      bring<CPOL>(a.c.k_pages + (((int64_t)clamp(own) * a.c.Hkv + h) * page + (SMALL ? 0 : base)) * D + (in * D + p * 16),
                  to + k * 64);
    }
  }
  template <int CPOL>
  __device__ __forceinline__ void copy_v(u32x4* to, int tile, int pg) const {
    const int page = a.c.page, base = (tile * 64) & (page - 1);
    const int p = (lane & 3) ^ twist_v(lane / 4);
    const int own = SMALL ? __shfl(pg, p * 16, 64) : __builtin_amdgcn_readfirstlane(pg);
    const uint8_t* at = a.c.v_pages + ((int64_t)clamp(own) * a.c.Hkv + h) * D * page + (SMALL ? 0 : base);
    const int in = lane / 4 * page + (SMALL ? (p * 16) & (page - 1) : p * 16);
#pragma unroll
    for (int k = 0; k < KP; ++k) bring<CPOL>(at + in + k * 16 * page, to + 64 * KP + k * 64);
  }
  __device__ __forceinline__ void scales(Codes<D>& r, int pg) const {
    const int64_t at = (int64_t)clamp(pg) * a.c.Hkv + h;
    r.ks = a.c.k_scale[at];
    r.vs = a.c.v_scale[at];
    r.ok = (uint32_t)pg < (uint32_t)a.c.num_pages;
  }
  // Past the caches (NT) where whole lines are used once: one row tile and,
  // for V, no page in which 64 keys of a channel are half a line.  Chains
  // that read 623 MB in pages of 64: 120 us with both past the caches, 125 with
  // V alone, 136 with neither; 32 rows of 8192 tokens in pages of 128: 118 us
  // with K alone, 138 with both.
  static constexpr int NT = 2;
  __device__ __forceinline__ void copy_k(u32x4* to, int tile, int pg) const {
    if (a.mtiles == 1) copy_k<NT>(to, tile, pg);
    else copy_k<0>(to, tile, pg);
  }
  __device__ __forceinline__ void copy_v(u32x4* to, int tile, int pg) const {
    if (a.mtiles == 1 && a.c.page <= 64) copy_v<NT>(to, tile, pg);
    else copy_v<0>(to, tile, pg);
  }
  __device__ __forceinline__ void take(Codes<D>& r, const u32x4* from) const {
    const int col = lane & 15;
#pragma unroll
    for (int ut = 0; ut < 4; ++ut)
#pragma unroll
      for (int d = 0; d < D / 64; ++d) {
        const int key = (col >> 2) * 16 + ut * 4 + (col & 3);
        r.k[ut][d] = from[key * KP + ((d * 4 + g) ^ twist_k(key))];
      }
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt) {
      const int d = dt * 16 + col;
      r.v[dt] = from[64 * KP + d * 4 + (g ^ twist_v(d))];
    }
  }
};

// The kernel's arguments read anew (they are its first and only parameter).
// What only a late step needs is then not held in registers through the main
// loop, where they are short.
__device__ __forceinline__ const AttnArgs& args_again() {
  typedef const AttnArgs __attribute__((address_space(4))) * KernArgs;
  KernArgs p = (KernArgs)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const AttnArgs*)p;
}

template <int D>
__device__ __forceinline__ void store_out(const AttnArgs& a, int b, int h, int qr, int d, f32x4 x) {
  union { bf16x2 p[2]; uint2 u; } y;
  y.p[0] = __builtin_convertvector(f32x2{x[0], x[1]}, bf16x2);
  y.p[1] = __builtin_convertvector(f32x2{x[2], x[3]}, bf16x2);
  *reinterpret_cast<uint2*>(a.out + (((int64_t)b * a.T + qr / a.G) * a.H + h * a.G + qr % a.G) * D + d) = y.u;
}

template <int KIND, int D, int NQ, bool SMALL>
__global__ __launch_bounds__(WG) __attribute__((amdgpu_waves_per_eu(RESIDENT, RESIDENT))) void cache_attention_kernel(AttnArgs a) {
  constexpr int MT = 16 * NQ;
  __shared__ Lds<D, NQ> sh;
  Run run;
  if (!find_run<MT>(a, sh.rows, run)) return;
  const int h = run.h, mt = run.mt;
  // Rows base .. base + ROWS - 1 are looked up; find_run did so for few rows.
  int b = run.b, begin = run.begin, at = run.at, base = a.c.B <= ROWS && a.mtiles == 1 ? 0 : b - ROWS;
  __syncthreads();

  while (at < run.end) {
  // Made anew for each segment: what the compiler derives from them would
  // otherwise be kept in registers across the loop, beyond what there are.
  int t = threadIdx.x;
  asm volatile("" : "+v"(t));
  const int lane = t & 63, g = lane >> 4, col = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);

  if (b - base >= ROWS) {
    base = b;
    __syncthreads();  // idle rows are passed without one
    if (t < ROWS && b + t < a.c.B) sh.rows[t] = row_of<MT>(args_again(), b + t);
    __syncthreads();
  }
  Row row = sh.rows[b - base];
#pragma unroll
  for (int k = 0; k < (int)(sizeof(Row) / 4); ++k)
    reinterpret_cast<int*>(&row)[k] = __builtin_amdgcn_readfirstlane(reinterpret_cast<int*>(&row)[k]);
  if (row.reps <= mt) row.n = 0;
  if (at >= begin + row.n) {  // the row has no such queries, or ended
    begin += row.n;
    ++b;
    continue;
  }
  const int t0 = at - begin, t1 = min(row.n, run.end - begin);
  // The row's parts: one for each run that holds some of it.  The numbers of
  // run and row together tell the parts apart.
  const int nparts = (begin + row.n - 1) / run.c - begin / run.c + 1;
  const int part0 = begin / run.c + b, part = at / run.c + b;
  at = begin + t1;
  const int nq = row.nq;

  // The wave's first cached tile is on its way while the rest is set up.
  const Loader<D, SMALL> ld{a, a.c.block_table + (int64_t)b * a.c.max_blocks, h, row.blocks * a.c.page, g, lane};
  int i = t0 + w;
  int i8 = i < row.near ? i + (row.near - i + NWAVE - 1) / NWAVE * NWAVE : i;
  Codes<D> r, ahead;
  u32x4* const codes = sh.wave[w].k;
  int next, first;
  const bool has_near = i < min(t1, row.near);
  if (i8 < t1) {
    first = ld.pages(i8 - row.near);
    ld.copy_k(codes, i8 - row.near, first);
    if (!has_near) ld.copy_v(codes, i8 - row.near, first);
    ld.scales(ahead, first);
    next = ld.pages(min(i8 + NWAVE, t1 - 1) - row.near);
  }

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
  if (a.parents) __syncthreads();

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
    st.set_x(n, NEAR_X);
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt) st.o[dt][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  // ---- tail and new tokens: 32 keys a tile, key 8 g + j of a tile at lane
  // group g; values are transposed through LDS ----------------------------------
  for (; i < min(t1, row.near); i += NWAVE) {
    const int j0 = i * 32, have = row.tail + nq;
    auto address = [&](int j, bool val) -> const uint16_t* {
      j = min(j, have - 1);
      if (j < row.tail)
        return (val ? a.c.v_tail : a.c.k_tail) +
               (((int64_t)b * a.c.tail + row.start + j) * a.c.Hkv + h) * D;  // a block does not wrap
      return (val ? a.vn : a.kn) + b * a.kv_row + (j - row.tail) * a.kv_tok + (int64_t)h * D;
    };
    u32x4 kk[2][D / 32];
#pragma unroll
    for (int ut = 0; ut < 2; ++ut) {
      const uint16_t* p = address(j0 + (col >> 2) * 8 + ut * 4 + (col & 3), false) + g * 16;
#pragma unroll
      for (int ks = 0; ks < D / 32; ++ks) kk[ut][ks] = *reinterpret_cast<const u32x4*>(p + (ks >> 1) * 64 + (ks & 1) * 8);
    }
    uint16_t* vt = sh.wave[w].near;
    constexpr int PER = D / 8;  // 16-byte pieces of a value
    uint32_t wild = 0;          // keys whose values are not all finite
#pragma unroll
    for (int e = 0; e < 32 * PER / 64; ++e) {
      const int piece = e * 64 + lane, j = piece / PER, d = piece % PER * 8;
      u32x4 v = *reinterpret_cast<const u32x4*>(address(j0 + j, true) + d);
      if (j0 + j >= have) v = u32x4{0, 0, 0, 0};
      *reinterpret_cast<u32x4*>(vt + j * (D + VPAD) + d) = v;
      // Its infinities and NaN (an exponent of ones carries into the sign's place).
      uint32_t odd = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) odd |= (v[k] & 0x7F807F80u) + 0x00800080u;
      const uint64_t lanes = __ballot((odd & 0x80008000u) != 0);
      if (lanes)
#pragma unroll
        for (int k = 0; k < 64 / PER; ++k)
          if (lanes >> (k * PER) & ((1ull << PER) - 1)) wild |= 1u << (e * 64 / PER + k);
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
      float x[8], p[8];
      // Seen: the tail (node < 0) and, of the new tokens, a chain's up to the
      // query's own or those of its path.  Plain bit operations: written as
      // key < have && (node < 0 || (parents ? path bit : node <= tok)), the
      // compiler (clang 22 of ROCm 7.2.0) puts the path's bit into the score's
      // register, sets the result to -inf for every new token and leaves the
      // block that should give the seen ones their score empty.
      const int last = a.parents ? -1 : tok[n];
      const uint64_t path = a.parents ? sh.path[tok[n]] : 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int key = j0 + g * 8 + j, node = key - row.tail;
        const bool see = (key < have) & ((node <= last) | (bool)((path >> (node & 63)) & 1));
        x[j] = see ? s[j >> 2][n][j & 3] : NEG_INF;
      }
      softmax_near(st, n, x, a.scale2, p);
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
    // A product would take such an element to the queries that do not see it
    // too (0 * inf): it leaves the tile, and is added to those that do.
    while (wild) {
      const int k = __builtin_ctz(wild), node = j0 + k - row.tail;
      wild &= wild - 1;
      bool see[NQ];
#pragma unroll
      for (int n = 0; n < NQ; ++n)
        see[n] = a.parents ? (node < 0) | (bool)((sh.path[tok[n]] >> (node & 63)) & 1) : node <= tok[n];
#pragma unroll
      for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint16_t* e = vt + k * (D + VPAD) + dt * 16 + g * 4 + j;
          const uint32_t v = *e;
          if ((v & 0x7F80u) == 0x7F80u) {
#pragma unroll
            for (int n = 0; n < NQ; ++n)
              if (see[n]) st.o[dt][n][j] += __uint_as_float(v << 16);
            *e = 0;  // by the 16 lanes that have read it
          }
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt) {
      // Read transposed: of four keys' 16 channels, 4 in each of four lanes, a
      // lane gets its channel of the four keys.
      union { s16x4 e[2]; bf16x8 v; } v8;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        v8.e[j] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(
            vt + (g * 8 + j * 4 + (col >> 2)) * (D + VPAD) + dt * 16 + (col & 3) * 4));
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        st.o[dt][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v8.v, lo[n], st.o[dt][n], 0, 0, 0);
        st.o[dt][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v8.v, hi[n], st.o[dt][n], 0, 0, 0);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }

  // ---- cached tiles ---------------------------------------------------------
  if (has_near && i8 < t1) {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the values have left their place
    ld.copy_v(codes, i8 - row.near, first);
  }
  // A tile's sums are written when the next one's loads are on their way, so
  // that no wait for loads waits for these too.
  float sums[NQ];
  int told = -1;
  auto tell = [&]() {
    const int key = told * 64 + g * 16;
    if (told >= 0 && (key & ((1 << a.sshift) - 1)) == 0 && key < row.blocks * a.c.page)
#pragma unroll
      for (int n = 0; n < NQ; ++n)
        a.mass[(((int64_t)b * a.c.Hkv + h) * a.nsub + (key >> a.sshift)) * (a.mtiles * MT) + mt * MT + n * 16 + col] = sums[n];
  };
  for (; i8 < t1; i8 += NWAVE) {
    const int tile = i8 - row.near;
    wait_vmem();  // the tile is in LDS
    ld.take(r, codes);
    r.ks = ahead.ks;
    r.vs = ahead.vs;
    r.ok = ahead.ok;
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // and in registers: the next may come
    if (a.mass) tell();
    if (i8 + NWAVE < t1) {
      ld.copy_k(codes, i8 + NWAVE - row.near, next);
      ld.copy_v(codes, i8 + NWAVE - row.near, next);
      ld.scales(ahead, next);
      next = ld.pages(min(i8 + 2 * NWAVE, t1 - 1) - row.near);
    }
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
    const bool ok = r.ok;
    const float c = ok ? r.ks * a.scale2 : 0.f;
    const ValueScale vs = value_scale(r.vs, ok);
    bool unlike = false;
    float top = (float)vs.e;
    if (SMALL) {
      top = groups_max(ok ? top : -150.f);
      unlike = __any(ok & ((float)vs.e < top - ALIKE));
    }
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
    f16x8 p8[2][NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      float x[16], p[16], psum;
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = s[j >> 2][n][j & 3];
      softmax_cached(st, n, x, c, vs, top, ok, unlike, p, psum);
      if (unlike) {
        // Blocks of small values beside some of large ones (or of zeros, whose
        // scale is 1): bf16 pairs, which have float32's range.
        const int up = vs.e + st.x(n);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          union { bf16x2 h[4]; bf16x8 v; } y, z;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const f32x2 e = {ldexpf(p[8 * u + 2 * j], up), ldexpf(p[8 * u + 2 * j + 1], up)};
            y.h[j] = __builtin_convertvector(e, bf16x2);
            z.h[j] = __builtin_convertvector(e - __builtin_convertvector(y.h[j], f32x2), bf16x2);
          }
#pragma unroll
          for (int dt = 0; dt < D / 16; ++dt) {
            uint32_t w0 = r.v[dt][2 * u], w1 = r.v[dt][2 * u + 1];
            asm volatile("" : "+v"(w0), "+v"(w1));  // widened here, and not kept for the next n
            const bf16x8 v8 = widen<KIND>(w0, w1);
            st.o[dt][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v8, z.v, st.o[dt][n], 0, 0, 0);
            st.o[dt][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v8, y.v, st.o[dt][n], 0, 0, 0);
          }
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) p[j] = 0.f;
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        union { f16x2 h[4]; f16x8 v; } y;
#pragma unroll
        for (int j = 0; j < 4; ++j) y.h[j] = __builtin_convertvector(f32x2{p[8 * u + 2 * j], p[8 * u + 2 * j + 1]}, f16x2);
        p8[u][n] = y.v;
      }
      if (a.mass) {
        float z = psum;
        if (a.sshift > 4) z = sum16(z);
        if (a.sshift > 5) z = sum32(z);
        sums[n] = st.m[n] + __builtin_amdgcn_logf(z);  // -inf where the page does not exist
      }
    }
    told = tile;
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const f16x8 v8 = widen_f16<KIND>(r.v[dt][2 * u], r.v[dt][2 * u + 1]);
#pragma unroll
        for (int n = 0; n < NQ; ++n)
          st.o[dt][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v8, p8[u][n], st.o[dt][n], 0, 0, 0);
      }
  }

  if (a.mass) tell();
  // ---- the four waves join ------------------------------------------------------
  // Each wave, and each part, puts out a mean of values with the weight that
  // the mean has, so that nothing passes float32's range on the way.
  float whole[NQ];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const float l = groups_sum(st.l[n]);
    whole[n] = l == 0.f ? 0.f : 1.f / l;
    const int x = st.x(n);
    if (__any((x < -80) | (x > 80))) {  // by two factors, each in float32's range
#pragma unroll
      for (int dt = 0; dt < D / 16; ++dt) st.o[dt][n] *= ldexpf(1.f, -x / 2);
      whole[n] = ldexpf(whole[n], -x - -x / 2);
    } else {
      whole[n] = ldexpf(whole[n], -x);
    }
    if (g == 0) {
      sh.m[w][n * 16 + col] = st.m[n];
      sh.l[w][n * 16 + col] = l;
    }
  }
  __syncthreads();  // every wave is past its use of the transposing buffer
#pragma unroll
  for (int n = 0; n < NQ; ++n)
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt)
      *reinterpret_cast<f32x4*>(&sh.o[w][(n * 16 + col) * (D + 4) + dt * 16 + g * 4]) = st.o[dt][n] * whole[n];
  __syncthreads();
  const AttnArgs& z = args_again();
  const int64_t step = (int64_t)z.c.Hkv * z.mtiles * MT, at0 = ((int64_t)h * z.mtiles + mt) * MT;
  const int64_t slot = part * step + at0;
  const int64_t tile = ((int64_t)b * z.c.Hkv + h) * z.mtiles + mt;
  constexpr int V4 = MT * D / 4 / WG;  // float4 per thread
#pragma unroll
  for (int v = 0; v < V4; ++v) {
    const int e = v * WG + t, rr = e / (D / 4), d = e % (D / 4) * 4;
    float m = sh.m[0][rr], l = 0.f;
#pragma unroll
    for (int k = 1; k < NWAVE; ++k) m = fmaxf(m, sh.m[k][rr]);
    float f[NWAVE];
#pragma unroll
    for (int k = 0; k < NWAVE; ++k) {
      f[k] = sh.m[k][rr] == NEG_INF ? 0.f : sh.l[k][rr] * exp2_fast(sh.m[k][rr] - m);
      l += f[k];
    }
    // 0 times infinity, NaN, where every score is -inf; not before the last join.
    const float whole = nparts > 1 && l == 0.f ? 0.f : 1.f / l;
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < NWAVE; ++k) x += *reinterpret_cast<const f32x4*>(&sh.o[k][rr * (D + 4) + d]) * (f[k] * whole);
    if (nparts > 1) {
      pub_store2(z.part_o + (slot + rr) * D + d, x[0], x[1]);
      pub_store2(z.part_o + (slot + rr) * D + d + 2, x[2], x[3]);
      if (d == 0) pub_store2(z.part_ml + (slot + rr) * 2, m, l);
    } else {
      const int qr = mt * MT + rr;
      if (qr < nq * z.G) store_out<D>(z, b, h, qr, d, x);
      if (z.mass && d == 0) z.lse[tile * MT + rr] = m + __builtin_amdgcn_logf(l);
    }
  }
  if (nparts > 1) {
    wait_vmem();
    __syncthreads();
    if (t == 0) {
      const unsigned n = __hip_atomic_fetch_add(z.arrived + tile, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      sh.last = n == (unsigned)nparts - 1;
      if (sh.last) __hip_atomic_store(z.arrived + tile, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (sh.last) {
      // J parts' loads go out at once.
      constexpr int J = 8 / V4;
      const float* ml = z.part_ml + (part0 * step + at0) * 2;
      const float* po = z.part_o + (part0 * step + at0) * D + t * 4;
      f32x4 x[V4];
      float big[V4], sum[V4];
#pragma unroll
      for (int v = 0; v < V4; ++v) {
        big[v] = NEG_INF;
        sum[v] = 0.f;
        x[v] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
      for (int s0 = 0; s0 < nparts; s0 += J) {
        float2 y[J][V4][2], e[J][V4];
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const int64_t s = min(s0 + j, nparts - 1) * step;
#pragma unroll
          for (int v = 0; v < V4; ++v) {
            y[j][v][0] = pub_load2(po + s * D + v * WG * 4);
            y[j][v][1] = pub_load2(po + s * D + v * WG * 4 + 2);
            e[j][v] = pub_load2(ml + (s + (v * WG + t) / (D / 4)) * 2);
          }
        }
#pragma unroll
        for (int v = 0; v < V4; ++v) {
          float top = big[v];
#pragma unroll
          for (int j = 0; j < J; ++j) top = fmaxf(top, e[j][v].x);  // a part read twice is no other maximum
          const float keep = big[v] == NEG_INF ? 0.f : sum[v] * exp2_fast(big[v] - top);
          float f[J];
          sum[v] = keep;
#pragma unroll
          for (int j = 0; j < J; ++j) {
            f[j] = s0 + j >= nparts || e[j][v].x == NEG_INF ? 0.f : e[j][v].y * exp2_fast(e[j][v].x - top);
            sum[v] += f[j];
          }
          const float whole = sum[v] == 0.f ? 0.f : 1.f / sum[v];
          x[v] *= keep * whole;
#pragma unroll
          for (int j = 0; j < J; ++j) x[v] += f32x4{y[j][v][0].x, y[j][v][0].y, y[j][v][1].x, y[j][v][1].y} * (f[j] * whole);
          big[v] = top;
        }
      }
#pragma unroll
      for (int v = 0; v < V4; ++v) {
        const int e = v * WG + t, rr = e / (D / 4), d = e % (D / 4) * 4, qr = mt * MT + rr;
        if (qr < nq * z.G) store_out<D>(z, b, h, qr, d, x[v] + 0.f * (1.f / sum[v]));
        if (z.mass && d == 0) z.lse[tile * MT + rr] = big[v] + __builtin_amdgcn_logf(sum[v]);
      }
    }
  }
  __syncthreads();  // the shared arrays are free for the next segment
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
    const int per = a.c.page >> a.sshift;
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
  int nq, mtiles, grid, runs, even, nsub;
  size_t o, ml, lse, mass, total;
};

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

int make_plan(const sv_cache& c, int T, int H, bool weights, Plan& pl) {
  const int M = T * (H / c.Hkv);
  // 64 rows beside D = 128 would leave one wave per SIMD (61-node trees over
  // up to 4k tokens: 261 against 181 us); beside D = 64 they halve the reads
  // and conversions (64 rows over 131k int8 tokens: 114 against 131 us).
  pl.nq = M <= 16 ? 1 : M <= 32 || c.D == 128 ? 2 : 4;
  const int mt = 16 * pl.nq;
  pl.mtiles = (M + mt - 1) / mt;
  const int64_t tiles = (int64_t)c.B * pl.mtiles, heads = tiles * c.Hkv;
  const int64_t most = ((int64_t)c.max_blocks * c.page + 63) / 64 + (c.page - 1 + T + 31) / 32;
  // The device counts a line's tiles, and that many once more, in 32 bits.
  if (most * tiles > INT_MAX / 2 || heads > INT_MAX) return SV_ERR_UNSUPPORTED;
  // Runs that the chip holds at once (see the kernel's registers).  Each row
  // tile's line may end with a part of a run, so the length of a run is
  // chosen for that many fewer (half of them where row tiles are many).
  const int64_t room = std::max<int64_t>(1, CUS * RESIDENT / c.Hkv);
  pl.even = (int)std::max<int64_t>(room - (pl.mtiles - 1), (room + 1) / 2);
  pl.runs = (int)std::min<int64_t>(pl.even, (most * tiles + CMIN - 1) / CMIN) + pl.mtiles - 1;
  pl.grid = (pl.runs * c.Hkv + 7) / 8 * 8;
  const int64_t parts = ((int64_t)pl.runs + c.B) * c.Hkv * pl.mtiles;
  const int64_t nsub = (int64_t)c.max_blocks * (c.page / std::min(c.page, 64));
  pl.nsub = (int)nsub;
  // The counters come first: they are what must be zero.
  size_t off = align256(sizeof(unsigned) * (size_t)heads);
  pl.o = off;
  off = align256(off + sizeof(float) * (size_t)parts * mt * c.D);
  pl.ml = off;
  off = align256(off + sizeof(float2) * (size_t)parts * mt);
  if (weights) {
    const size_t rows = (size_t)c.B * c.Hkv, mpad = (size_t)pl.mtiles * mt;
    pl.lse = off;
    off = align256(off + sizeof(float) * rows * mpad);
    pl.mass = off;
    off = align256(off + sizeof(float) * rows * mpad * (size_t)nsub);
    if (((int64_t)c.B * T * c.max_blocks + WG - 1) / WG > MAX_ITEMS / WG) return SV_ERR_UNSUPPORTED;
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
  if constexpr (D == 64)
    if (pl.nq == 4) return launch<KIND, D, 4>(a, pl, st);
  return pl.nq == 1 ? launch<KIND, D, 1>(a, pl, st) : launch<KIND, D, 2>(a, pl, st);
}
template <int KIND>
int launch_dim(const AttnArgs& a, const Plan& pl, hipStream_t st) {
  return a.c.D == 64 ? launch_rows<KIND, 64>(a, pl, st) : launch_rows<KIND, 128>(a, pl, st);
}

}  // namespace

// Whether any of `rows` stretches of `span` bytes, `stride` bytes apart, shares
// a byte with the n at `out`.
static bool crosses(const void* base, int64_t stride, int rows, int64_t span, const void* out, int64_t n) {
  const int64_t d = reinterpret_cast<intptr_t>(out) - reinterpret_cast<intptr_t>(base);  // row k: k stride < d + n, d < k stride + span
  if (stride == 0 || rows == 1) return 0 < d + n && d < span;
  const int64_t first = d < span ? 0 : (d - span) / stride + 1;  // the first row that ends behind `out`'s start
  return first < rows && first * stride < d + n;
}

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
  if (T > (parents ? SV_MAX_NODES : SV_MAX_K + 1) || H / c.Hkv > MAX_GROUP) return SV_ERR_UNSUPPORTED;
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
  // The output is written while other work-groups still read.
  const int64_t bytes = (int64_t)c.B * T * H * c.D * 2, mass = (int64_t)c.B * T * c.max_blocks * 4;
  for (const void* p : {q, k_new, v_new}) {
    const bool kv = p != q;
    const int64_t row = (kv ? kv_row : q_row) * 2;
    const int64_t span = ((T - 1) * (kv ? kv_tok : q_tok) + (int64_t)(kv ? c.Hkv : H) * c.D) * 2;
    if (crosses(p, row, c.B, span, out, bytes) || (weights && crosses(p, row, c.B, span, weights, mass)))
      return SV_ERR_ARG;
  }
  const size_t nb = (size_t)c.B * 4, pages = (size_t)c.num_pages * c.Hkv, tail = (size_t)c.B * c.tail * c.Hkv * c.D * 2;
  const Output written[] = {{{out, (size_t)bytes}, nullptr}, {{weights, (size_t)mass}, nullptr}, {{workspace, pl.total}, nullptr}};
  const Array read[] = {{positions, nb}, {blocks, nb}, {query_lens, nb}, {parents, nb * T}, {c.block_table, nb * c.max_blocks},
                        {c.k_pages, pages * c.page * c.D}, {c.v_pages, pages * c.page * c.D}, {c.k_scale, pages * 4},
                        {c.v_scale, pages * 4}, {c.k_tail, tail}, {c.v_tail, tail}};
  if (outputs_overlap(written, read)) return SV_ERR_ARG;
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
  a.mtiles = pl.mtiles;
  a.even = pl.even;
  a.scale2 = scale * LOG2E;
  a.out = static_cast<uint16_t*>(out);
  a.weights = weights;
  char* ws = static_cast<char*>(workspace);
  a.arrived = reinterpret_cast<unsigned*>(ws);
  a.part_o = reinterpret_cast<float*>(ws + pl.o);
  a.part_ml = reinterpret_cast<float*>(ws + pl.ml);
  a.lse = weights ? reinterpret_cast<float*>(ws + pl.lse) : nullptr;
  a.mass = weights ? reinterpret_cast<float*>(ws + pl.mass) : nullptr;
  for (a.pshift = 4; 1 << a.pshift < c.page; ++a.pshift) {}
  a.sshift = std::min(a.pshift, 6);
  a.nsub = pl.nsub;
  (void)hipGetLastError();
  return c.kind == SV_E4M3 ? launch_dim<SV_E4M3>(a, pl, stream) : launch_dim<SV_INT8>(a, pl, stream);
}
