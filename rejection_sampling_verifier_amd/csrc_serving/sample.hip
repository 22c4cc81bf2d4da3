// Tokens drawn from logits under temperature, top-k, top-p and min-p
// (spec_verify_sample), and logits cut by the same rules
// (spec_verify_truncate), for gfx950.
//
// Mathematics: with w(x) = exp((l(x) - max) / T), all three cuts leave a
// prefix of the tokens in the order (logit descending, id ascending), so a
// row's kept set is one bound: a logit and, among the tokens that have just
// that logit, an id.  The bound is found by counting (top-k) or adding up
// (top-p) over bins of the logits' order, not by sorting.  Weights are formed
// in float64 and added as whole numbers of 2^-43: such sums do not depend on
// their order, so atomics may form them, and a token is the one that 64 bits
// give unless a border lies within about 2^-36 of the draw.
//
// HBM reads bound it.  sample_stats_kernel reads each logit once: per chunk of
// a row the maximum and, where a rule or a draw needs it, the sum.  Where
// rules cut the row it also puts out the chunk's candidates, those that a bound
// from the chunk alone does not exclude: a chunk's top k are found among the k
// largest of its lanes' maxima, its nucleus above (1 - p) / V of its sum, min-p
// below its maximum.  sample_row_kernel, a work-group per row, finds the
// row's bound among the candidates and draws.  A chunk with more candidates
// than its list holds is read again there.

#include <climits>
#include <cmath>

#include "cache.h"

using namespace sv;
using namespace svr;

namespace {

constexpr int MAX_VOCAB = 1 << 20;   // so that sums of weights of up to 2^43 stay below 2^63
constexpr int MAX_DRAWS = SV_MAX_NODES;
constexpr int MAX_CHUNKS = 512;
constexpr int RW = 1024;             // threads of the kernel over rows
constexpr int BINS = 2 * RW;
constexpr int HELD = 6144;           // candidates of a row that LDS holds
constexpr double ONE = 0x1p43;       // a weight of 1 as a whole number

struct Chunk {
  double sum;       // of its weights against its own maximum
  float top, low;   // its maximum; at least as many of its logits as top-k asks for are this large
  int first;        // the id of its maximum
  int listed;       // candidates in its list, or -1: more than it holds
};

struct SampleArgs {
  const void* logits;
  int64_t row, pos;   // strides in elements
  const float* uniforms;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int32_t* tokens;
  float* logprobs;
  void* out;          // of spec_verify_truncate
  int64_t out_row, out_pos;
  Chunk* chunks;      // [rows][C]
  double* subs;       // [rows][C][4 NV] sums of a wave's vectors, rows without a cut; of spec_verify_sample
  uint64_t* lists;    // [rows][C][cap] order << 32 | id
  uint2* bounds;      // [rows] of spec_verify_truncate
  int B, P, V, n, C, cap;
};

// A row's rules.
struct Rules {
  float T, p, m;
  int k;   // 0: none
  bool greedy, by_p, by_m;
  __device__ __forceinline__ bool cut() const { return k || by_p || by_m; }
  // The sum over the whole row is asked for: the mass of top-p, and of a draw without a cut.
  __device__ __forceinline__ bool whole() const { return !cut() || (by_p && !k); }
  // What min-p leaves out is not asked for: unless it counts in the mass of the top k.
  __device__ __forceinline__ bool m_first() const { return by_m && !(k && by_p); }
};
__device__ __forceinline__ Rules rules_of(const SampleArgs& a, int b) {
  Rules r;
  r.T = a.temperature[b];
  r.greedy = !(r.T > 0.f);
  r.k = a.top_k ? a.top_k[b] : 0;
  if (r.k < 0 || r.k >= a.V) r.k = 0;
  r.p = a.top_p ? a.top_p[b] : 1.f;
  r.by_p = r.p < 1.f;
  r.p = fmaxf(r.p, 0.f);
  r.m = a.min_p ? a.min_p[b] : 0.f;
  r.by_m = r.m > 0.f;
  r.m = fminf(r.m, 1.f);
  return r;
}

// 2^y for y <= 0, to about 2^-50: y's whole part goes into the exponent, the
// rest, at most 1/2, into the series of exp(r ln 2), whose 13th power is below
// 2^-50.  fp64 multiply-adds run at the rate of fp32 ones here.
__device__ __forceinline__ double exp2_64(double y) {
  const double n = rint(y), r = (y - n) * 0.69314718055994530942;
  double s = 1.0 / 479001600.0;
  s = fma(s, r, 1.0 / 39916800.0);
  s = fma(s, r, 1.0 / 3628800.0);
  s = fma(s, r, 1.0 / 362880.0);
  s = fma(s, r, 1.0 / 40320.0);
  s = fma(s, r, 1.0 / 5040.0);
  s = fma(s, r, 1.0 / 720.0);
  s = fma(s, r, 1.0 / 120.0);
  s = fma(s, r, 1.0 / 24.0);
  s = fma(s, r, 1.0 / 6.0);
  s = fma(s, r, 0.5);
  s = fma(s, r, 1.0);
  s = fma(s, r, 1.0);
  return ldexp(s, (int)fmax(n, -1100.0));
}
// The weight of a logit against a maximum, c = log2(e) / T.  1 at the maximum,
// whatever it is, 0 for -inf.
__device__ __forceinline__ double weight(float l, float top, double c) {
  if (l == top) return 1.0;
  return l == NEG_INF ? 0.0 : exp2_64(fmax(((double)l - (double)top) * c, -2000.0));
}
// ln of a token's part of the sum `total` of the weights.
__device__ __forceinline__ float log_part(float l, float top, float T, double total) {
  return (float)((l == top ? 0.0 : ((double)l - (double)top) / (double)T) - log(total));
}
__device__ __forceinline__ double rate(float T) { return 1.4426950408889634074 / (double)T; }
__device__ __forceinline__ uint64_t whole_of(double w) {
  return (uint64_t)(__double_as_longlong(w + 512.0) - __double_as_longlong(512.0));  // steps of 2^-43
}

// A logit that is T ln x below `top`, or a little less: what lies under it has
// a weight under x for sure.
__device__ __forceinline__ float under(float top, float T, double x) {
  const double l = (double)top + (double)T * log(x);
  const float f = (float)(l - (fabs(l) + fabs((double)top) + 1.0) * 1e-6);
  return f == f ? f : NEG_INF;
}

// The order of logits as whole numbers: for bf16 the upper half of its float32's.
template <typename ET>
__device__ __forceinline__ uint32_t order_of(float l) {
  const uint32_t k = order_key(l);
  return sizeof(ET) == 2 ? k >> 16 : k;
}
template <typename ET>
__device__ __forceinline__ float logit_of(uint32_t o) {
  if (sizeof(ET) == 2) o = o & 0x8000u ? o << 16 : o << 16 | 0xFFFFu;
  return key_value(o);
}

// The vectors of a row: vector q holds ids q VEC - lead .. + VEC - 1, so that
// each is 16-byte aligned, whatever the row's alignment.  Elements outside the
// row, and NaN, read as -inf.
template <typename ET>
struct RowOf {
  static constexpr int VEC = Tr<ET>::VEC;
  const ET* p;
  int lead, V;
  __device__ __forceinline__ RowOf(const void* base, int64_t at, int V) : p(static_cast<const ET*>(base) + at), V(V) {
    lead = (int)(reinterpret_cast<uintptr_t>(p) / sizeof(ET) % VEC);
  }
  __device__ __forceinline__ int first(int q) const { return q * VEC - lead; }
  __device__ __forceinline__ u32x4 load(int q) const {
    const int id = first(q);
    u32x4 v = {Tr<ET>::NEG_INF_WORD, Tr<ET>::NEG_INF_WORD, Tr<ET>::NEG_INF_WORD, Tr<ET>::NEG_INF_WORD};
    if (id >= 0 && id + VEC <= V) {
      v = *reinterpret_cast<const u32x4*>(p + id);
    } else {
#pragma unroll
      for (int k = 0; k < VEC; ++k)
        if (id + k >= 0 && id + k < V) Tr<ET>::set(v, k, p + id + k);
    }
    return v;
  }
};
template <typename ET>
__device__ __forceinline__ float logit_at(const u32x4& v, int k) {
  return fmaxf(Tr<ET>::at(v, k), NEG_INF);
}

__device__ __forceinline__ double shfl_xor64(double x, int m) { return __shfl_xor(x, m, 64); }

// ---- per chunk ----------------------------------------------------------------

template <typename ET, int NV>
__global__ __launch_bounds__(WG) void sample_stats_kernel(SampleArgs a) {
  constexpr int VEC = Tr<ET>::VEC;
  __shared__ float shf[NWAVE];
  __shared__ int shi[NWAVE];
  __shared__ double shd[NWAVE];
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  const int row = blockIdx.x / a.C, chunk = blockIdx.x % a.C;
  const int b = row / a.P;
  const RowOf<ET> x(a.logits, b * a.row + (int64_t)(row % a.P) * a.pos, a.V);
  const Rules r = rules_of(a, b);
  const int q0 = chunk * WG * NV + t;
  u32x4 v[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) v[j] = x.load(q0 + j * WG);
  float mine = NEG_INF;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int k = 0; k < VEC; ++k) mine = fmaxf(mine, logit_at<ET>(v[j], k));
  const float top = block_max(mine, shf);
  Chunk o = {0.0, top, NEG_INF, INT_MAX, 0};
  Chunk* const put = a.chunks + (int64_t)row * a.C + chunk;
  if (r.greedy || top == NEG_INF) {
    if (top > NEG_INF) {
      int first = INT_MAX;
      if (mine == top) {
#pragma unroll
        for (int j = NV - 1; j >= 0; --j)
#pragma unroll
          for (int k = VEC - 1; k >= 0; --k)
            if (logit_at<ET>(v[j], k) == top) first = x.first(q0 + j * WG) + k;
      }
#pragma unroll
      for (int s = 32; s; s >>= 1) first = min(first, __shfl_xor(first, s, 64));
      if (lane == 0) shi[w] = first;
      __syncthreads();
      for (int k = 0; k < NWAVE; ++k) o.first = min(o.first, shi[k]);
    }
    if (t == 0) *put = o;
    return;
  }
  const bool cut = r.cut();
  const double c = rate(r.T);
  if (r.whole()) {
    double s[NV], all = 0.0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      s[j] = 0.0;
#pragma unroll
      for (int k = 0; k < VEC; ++k) s[j] += weight(logit_at<ET>(v[j], k), top, c);
      all += s[j];
    }
    if (!cut && a.subs) {
      double* subs = a.subs + ((int64_t)row * a.C + chunk) * (NWAVE * NV);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        double z = s[j];
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) z += shfl_xor64(z, m);
        if (lane == 0) subs[j * NWAVE + w] = z;
      }
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) all += shfl_xor64(all, m);
    if (lane == 0) shd[w] = all;
    __syncthreads();
    for (int k = 0; k < NWAVE; ++k) o.sum += shd[k];
  }
  if (cut) {
    float low = NEG_INF;  // no token under it is kept
    if (r.k) {
      // Each wave looks for a logit that a quarter of k of its lanes' maxima
      // reach; the lowest of the four is reached by k.
      const int q = (r.k + NWAVE - 1) / NWAVE;
      uint32_t key = 0;
      if (q <= 64) {
        const uint32_t own = order_of<ET>(mine);
        for (uint32_t bit = sizeof(ET) == 2 ? 1u << 15 : 1u << 31; bit; bit >>= 1)
          if (__popcll(__ballot(own >= (key | bit))) >= q) key |= bit;
      }
      if (lane == 0) shf[w] = key <= order_of<ET>(NEG_INF) ? NEG_INF : logit_of<ET>(key);
      __syncthreads();
      low = fminf(fminf(shf[0], shf[1]), fminf(shf[2], shf[3]));
      o.low = low;
    } else if (r.by_p) {
      low = under(top, r.T, (1.0 - (double)r.p) * o.sum / a.V);
    }
    if (r.m_first()) low = fmaxf(low, under(top, r.T, (double)r.m));
    int n = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        const float l = logit_at<ET>(v[j], k);
        n += (l >= low) & (l > NEG_INF);
      }
    int total;
    __syncthreads();
    int at = block_count_scan(n, shi, total);
    o.listed = total <= a.cap ? total : -1;
    if (o.listed > 0 && n) {
      uint64_t* list = a.lists + ((int64_t)row * a.C + chunk) * a.cap;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const float l = logit_at<ET>(v[j], k);
          if ((l >= low) & (l > NEG_INF))
            list[at++] = (uint64_t)order_of<ET>(l) << 32 | (uint32_t)(x.first(q0 + j * WG) + k);
        }
    }
  }
  if (t == 0) *put = o;
}

// ---- per row ------------------------------------------------------------------

struct RowLds {
  uint64_t mass[BINS];
  uint32_t count[BINS];
  uint64_t held[HELD];
  double upto[MAX_CHUNKS];
  float top[MAX_CHUNKS];
  int listed[MAX_CHUNKS];
  uint64_t sums[RW / 64];
  uint32_t counts[RW / 64];
  uint64_t before;      // what the search found
  uint32_t before_count, bin;
  int found, n;
  float low, max;
};

// Over the work-group's threads, in their order: what lies before this one.
__device__ __forceinline__ uint64_t scan64(uint64_t v, uint64_t* sums, uint64_t& total) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  uint64_t inc = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint64_t u = __shfl_up((unsigned long long)inc, o, 64);
    if (lane >= o) inc += u;
  }
  if (lane == 63) sums[w] = inc;
  __syncthreads();
  uint64_t base = 0;
  total = 0;
#pragma unroll
  for (int k = 0; k < RW / 64; ++k) {
    if (k < w) base += sums[k];
    total += sums[k];
  }
  __syncthreads();
  return base + inc - v;
}

template <typename ET, int NV>
struct RowWork {
  static constexpr int VEC = Tr<ET>::VEC;
  const SampleArgs& a;
  RowLds& sh;
  const RowOf<ET>& x;
  int row;
  float max;
  double c;
  float low;       // no candidate under it
  bool in_lds;
  uint32_t kt;     // kept: order above kt, or kt itself with ids below idlim
  int idlim;

  __device__ __forceinline__ bool kept(uint32_t o, int id) const { return o > kt || (o == kt && id < idlim); }
  __device__ __forceinline__ double w(uint32_t o) const { return weight(logit_of<ET>(o), max, c); }

  // f(order, id) for the row's candidates in chunks [c0, c1).
  template <typename F>
  __device__ __forceinline__ void visit_chunks(int c0, int c1, F f) const {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int ch = c0 + wave; ch < c1; ch += RW / 64) {
      const uint64_t* list = a.lists + ((int64_t)row * a.C + ch) * a.cap;
      for (int i = lane; i < sh.listed[ch]; i += 64) {
        const uint64_t e = list[i];
        if (logit_of<ET>((uint32_t)(e >> 32)) >= low) f((uint32_t)(e >> 32), (int)(uint32_t)e);
      }
    }
    for (int ch = c0; ch < c1; ++ch) {
      if (sh.listed[ch] >= 0) continue;
      for (int q = threadIdx.x; q < WG * NV; q += RW) {
        const u32x4 v = x.load(ch * WG * NV + q);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const float l = logit_at<ET>(v, k);
          if ((l >= low) & (l > NEG_INF)) f(order_of<ET>(l), x.first(ch * WG * NV + q) + k);
        }
      }
    }
  }
  // f(order, id) for the row's candidates with ids in [i0, i1).
  template <typename F>
  __device__ __forceinline__ void visit(int i0, int i1, F f) const {
    if (in_lds) {
      for (int i = threadIdx.x; i < sh.n; i += RW) {
        const uint64_t e = sh.held[i];
        f((uint32_t)(e >> 32), (int)(uint32_t)e);
      }
      return;
    }
    const int per = WG * NV * VEC;
    visit_chunks((i0 + x.lead) / per, min(a.C, (i1 - 1 + x.lead) / per + 1), f);
  }
  __device__ __forceinline__ void clear() {
    for (int i = threadIdx.x; i < BINS; i += RW) {
      sh.mass[i] = 0;
      sh.count[i] = 0;
    }
    __syncthreads();
  }
  // Of the bins, from the last down or from the first up, the one in which the
  // running sum (of counts or masses) reaches `need`: sh.found, sh.bin and what
  // lies before it.  The total of the masses comes back.
  template <bool DOWN, bool MASS>
  __device__ __forceinline__ uint64_t search(uint64_t need) {
    const int t = threadIdx.x;
    __syncthreads();
    if (t == 0) sh.found = 0;
    const int i0 = DOWN ? BINS - 1 - 2 * t : 2 * t, i1 = DOWN ? i0 - 1 : i0 + 1;
    const uint64_t v0 = MASS ? sh.mass[i0] : sh.count[i0], v1 = MASS ? sh.mass[i1] : sh.count[i1];
    uint64_t total;
    const uint64_t before = scan64(v0 + v1, sh.sums, total);
    if (before < need && need <= before + v0 + v1) {
      const bool second = need > before + v0;
      sh.found = 1;
      sh.bin = second ? i1 : i0;
      sh.before = second ? before + v0 : before;
    }
    __syncthreads();
    return total;
  }

  // Cuts the kept set down to its first tokens in the order of logits: as many
  // as `need` (counts), or until their mass reaches it.
  template <bool MASS>
  __device__ __forceinline__ void cut(uint64_t need) {
    uint32_t lo = kt, hi = order_of<ET>(max);
    {
      const uint32_t l = order_of<ET>(low);
      if (l > lo) lo = l;
    }
    uint64_t left = need;
    uint32_t ties = 0;
    for (;;) {
      int shift = 0;
      while ((hi - lo) >> shift >= BINS) ++shift;
      clear();
      visit(0, a.V, [&](uint32_t o, int id) {
        if (o < lo || o > hi || !kept(o, id)) return;
        const uint32_t bin = (o - lo) >> shift;
        atomicAdd(&sh.count[bin], 1u);
        if (MASS) atomicAdd((unsigned long long*)&sh.mass[bin], (unsigned long long)whole_of(w(o)));
      });
      search<true, MASS>(left);
      if (!sh.found) return;  // all of them do not reach it
      left -= sh.before;
      lo += sh.bin << shift;
      if (shift == 0) {
        ties = sh.count[sh.bin];
        break;
      }
      hi = min(hi, lo + ((1u << shift) - 1));
    }
    // Of the tokens with this logit as many as it takes, the lowest ids first.
    uint64_t n = left;
    if (MASS) {
      const uint64_t one = whole_of(w(lo));
      n = one ? (left + one - 1) / one : ties;
    }
    const int limit = lo == kt ? idlim : INT_MAX;
    kt = lo;
    idlim = limit;
    if (n >= ties) return;
    int shift = 0;
    while ((a.V - 1) >> shift >= BINS) ++shift;
    int i0 = 0, i1 = a.V;
    for (int pass = 0; pass < 2; ++pass) {
      __syncthreads();
      clear();
      visit(i0, i1, [&](uint32_t o, int id) {
        if (o == lo && id < limit && id >= i0 && id < i1) atomicAdd(&sh.count[(id - i0) >> shift], 1u);
      });
      search<false, false>(n);
      n -= sh.before;
      i0 += sh.bin << shift;
      i1 = min(a.V, i0 + (1 << shift));
      shift = 0;
    }
    idlim = i0 + 1;
  }
};

template <typename ET, int NV>
__global__ __launch_bounds__(RW) void sample_row_kernel(SampleArgs a) {
  constexpr int VEC = Tr<ET>::VEC, SUBS = NWAVE * NV;
  __shared__ RowLds sh;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int row = blockIdx.x, b = row / a.P;
  const RowOf<ET> x(a.logits, b * a.row + (int64_t)(row % a.P) * a.pos, a.V);
  const Rules r = rules_of(a, b);
  const Chunk* chunks = a.chunks + (int64_t)row * a.C;
  int32_t* tokens = a.tokens ? a.tokens + (int64_t)row * a.n : nullptr;
  float* logprobs = a.logprobs ? a.logprobs + (int64_t)row * a.n : nullptr;

  // The row's maximum, by the first wave.
  if (wave == 0) {
    float top = NEG_INF, low = NEG_INF;
    for (int i = lane; i < a.C; i += 64) {
      const Chunk o = chunks[i];
      sh.top[i] = o.top;
      sh.listed[i] = o.listed;
      sh.upto[i] = o.sum;
      top = fmaxf(top, o.top);
      low = fmaxf(low, o.low);
    }
    top = wave_max(top);
    low = wave_max(low);
    if (lane == 0) {
      sh.max = top;
      sh.low = low;
      sh.n = 0;
    }
  }
  __syncthreads();
  const float max = sh.max;
  if (max == NEG_INF || r.greedy) {
    if (t < a.n) {
      int id = -1;
      if (max > NEG_INF) {
        int i = 0;
        while (sh.top[i] < max) ++i;
        id = chunks[i].first;
      }
      tokens[t] = id;
      if (logprobs) logprobs[t] = id < 0 ? NEG_INF : 0.f;
    }
    if (a.bounds && t == 0) a.bounds[row] = make_uint2(0, INT_MAX);
    return;
  }
  const double c = rate(r.T);
  // Sums of the chunks against the row's maximum, added up in order.
  if (r.whole()) {
    for (int i = t; i < a.C; i += RW)
      sh.upto[i] = sh.top[i] == NEG_INF ? 0.0 : sh.upto[i] * weight(sh.top[i], max, c);
    __syncthreads();
    if (wave == 0) {
      double base = 0.0;
      for (int i0 = 0; i0 < a.C; i0 += 64) {
        double z = i0 + lane < a.C ? sh.upto[i0 + lane] : 0.0;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
          const double u = __shfl_up(z, o, 64);
          if (lane >= o) z += u;
        }
        z += base;
        if (i0 + lane < a.C) sh.upto[i0 + lane] = z;
        base = __shfl(z, 63, 64);
      }
    }
    __syncthreads();
  }

  if (!r.cut()) {
    if (a.bounds && t == 0) a.bounds[row] = make_uint2(0, INT_MAX);
    const double total = sh.upto[a.C - 1];
    for (int d = wave; d < a.n; d += RW / 64) {
      const float u = a.uniforms[(int64_t)row * a.n + d];
      double left = (double)(u > 0.f ? fminf(u, 0x1.fffffep-1f) : 0.f) * total;
      // The first chunk whose running sum passes it; the last with any weight if rounding leaves none.
      int ch = 0, last = 0;
      for (int i0 = 0; i0 < a.C; i0 += 64) {
        const int i = i0 + lane;
        const double z = i < a.C ? sh.upto[i] : total, y = i > 0 && i < a.C ? sh.upto[i - 1] : 0.0;
        const uint64_t some = __ballot(i < a.C && z > (i ? y : 0.0));
        if (some) last = i0 + 63 - __builtin_clzll(some);
        const uint64_t past = __ballot(i < a.C && z > left);
        if (past) {
          ch = i0 + __builtin_ctzll(past);
          break;
        }
        ch = last;
      }
      const float top = sh.top[ch];
      left = (left - (ch ? sh.upto[ch - 1] : 0.0)) / weight(top, max, c);
      const double* subs = a.subs + ((int64_t)row * a.C + ch) * SUBS;
      const double own = lane < SUBS ? subs[lane] : 0.0;
      double z = own;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const double y = __shfl_up(z, o, 64);
        if (lane >= o) z += y;
      }
      uint64_t past = __ballot(own > 0.0 && z > left);
      const uint64_t some = __ballot(own > 0.0);
      const int sub = past ? __builtin_ctzll(past) : 63 - __builtin_clzll(some);
      left -= __shfl(z - own, sub, 64);
      const int q = ch * WG * NV + sub / NWAVE * WG + sub % NWAVE * 64 + lane;
      const u32x4 v = x.load(q);
      double e = 0.0;
#pragma unroll
      for (int k = 0; k < VEC; ++k) e += weight(logit_at<ET>(v, k), top, c);
      z = e;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const double y = __shfl_up(z, o, 64);
        if (lane >= o) z += y;
      }
      past = __ballot(e > 0.0 && z > left);
      const uint64_t any = __ballot(e > 0.0);
      const int who = past ? __builtin_ctzll(past) : 63 - __builtin_clzll(any);
      if (lane == who) {
        double sum = z - e;
        int id = -1;
        float l = 0.f;
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const float y = logit_at<ET>(v, k);
          const double g = weight(y, top, c);
          if (g > 0.0 && (id < 0 || !(sum > left))) {
            id = x.first(q) + k;
            l = y;
          }
          sum += g;
        }
        tokens[d] = id;
        if (logprobs) logprobs[d] = log_part(l, max, r.T, total);
      }
    }
    return;
  }

  RowWork<ET, NV> work{a, sh, x, row, max, c, sh.low, false, 0, INT_MAX};
  const double sum = r.by_p && !r.k ? sh.upto[a.C - 1] : 0.0;
  if (r.by_p && !r.k) work.low = under(max, r.T, (1.0 - (double)r.p) * sum / a.V);
  if (r.m_first()) work.low = fmaxf(work.low, under(max, r.T, (double)r.m));
  // Its candidates come to LDS, if they are few.
  work.visit_chunks(0, a.C, [&](uint32_t o, int id) {
    const int at = atomicAdd(&sh.n, 1);
    if (at < HELD) sh.held[at] = (uint64_t)o << 32 | (uint32_t)id;
  });
  __syncthreads();
  work.in_lds = sh.n <= HELD;

  if (r.k) work.template cut<false>(r.k);
  if (r.by_p) {
    double mass = sum * ONE;
    if (r.k) {
      // The mass of the top k.
      __syncthreads();
      if (t == 0) sh.before = 0;
      __syncthreads();
      uint64_t own = 0;
      work.visit(0, a.V, [&](uint32_t o, int id) {
        if (work.kept(o, id)) own += whole_of(work.w(o));
      });
      uint64_t total;
      scan64(own, sh.sums, total);
      mass = (double)total;
    }
    const double need = ceil((double)r.p * mass);
    work.template cut<true>(need >= 1.0 ? (uint64_t)need : 1);
  }
  if (r.by_m) {
    // The lowest logit whose weight is at least m, by 64 probes at a time.
    uint32_t lo = 0, hi = order_of<ET>(max);  // in (lo, hi]: the maximum's weight is 1
    while (hi - lo > 1) {
      const uint32_t step = (hi - lo + 63) / 64;
      const uint32_t at = lo + min((uint32_t)lane * step + step, hi - lo);
      const uint64_t yes = __ballot(work.w(at) >= (double)r.m);
      const int first = __builtin_ctzll(yes);  // the last probe is hi
      const uint32_t from = lo + (uint32_t)first * step;
      hi = lo + min((uint32_t)first * step + step, hi - lo);
      lo = from;
    }
    if (hi > work.kt) {
      work.kt = hi;
      work.idlim = INT_MAX;
    }
  }
  if (a.bounds) {
    if (t == 0) a.bounds[row] = make_uint2(work.kt, (uint32_t)work.idlim);
    return;
  }

  // The kept tokens' masses by ids, then by the ids of a draw's bin.
  int shift = 0;
  while ((a.V - 1) >> shift >= BINS) ++shift;
  uint64_t* const fine = reinterpret_cast<uint64_t*>(sh.count);  // up to BINS / 2 ids of a bin
  __syncthreads();
  work.clear();
  work.visit(0, a.V, [&](uint32_t o, int id) {
    if (work.kept(o, id)) atomicAdd((unsigned long long*)&sh.mass[id >> shift], (unsigned long long)whole_of(work.w(o)));
  });
  const uint64_t total = work.template search<false, true>(0);
  for (int d = 0; d < a.n; ++d) {
    const float u = a.uniforms[(int64_t)row * a.n + d];
    const double at = floor((double)(u > 0.f ? fminf(u, 0x1.fffffep-1f) : 0.f) * (double)total);
    const uint64_t need = min((uint64_t)at + 1, total);
    work.template search<false, true>(need);
    const int i0 = (int)sh.bin << shift, i1 = min(a.V, i0 + (1 << shift));
    const uint64_t left = need - sh.before;
    for (int i = t; i < 1 << shift; i += RW) fine[i] = 0;
    __syncthreads();
    work.visit(i0, i1, [&](uint32_t o, int id) {
      if (id >= i0 && id < i1 && work.kept(o, id)) fine[id - i0] = (uint64_t)o << 32 | 1u;
    });
    __syncthreads();
    if (wave == 0) {
      // 64 ids at a time.
      uint64_t before = 0;
      for (int i = 0; i < 1 << shift; i += 64) {
        const uint64_t e = i + lane < 1 << shift ? fine[i + lane] : 0;
        const uint64_t own = e ? whole_of(work.w((uint32_t)(e >> 32))) : 0;
        uint64_t z = own;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
          const uint64_t y = __shfl_up((unsigned long long)z, o, 64);
          if (lane >= o) z += y;
        }
        const uint64_t past = __ballot(before + z >= left);
        if (past) {
          if (lane == __builtin_ctzll(past)) {
            tokens[d] = i0 + i + lane;
            if (logprobs) logprobs[d] = log_part(logit_of<ET>((uint32_t)(e >> 32)), max, r.T, (double)total / ONE);
          }
          break;
        }
        before += __shfl((unsigned long long)z, 63, 64);
      }
    }
    __syncthreads();
  }
}

// ---- cut logits ---------------------------------------------------------------

template <typename ET>
__global__ __launch_bounds__(WG) void truncate_kernel(SampleArgs a, int per, int inplace) {
  constexpr int VEC = Tr<ET>::VEC;
  const int row = blockIdx.x / per;
  const int64_t at = (int64_t)(row / a.P) * a.row + (int64_t)(row % a.P) * a.pos;
  const int64_t to = (int64_t)(row / a.P) * a.out_row + (int64_t)(row % a.P) * a.out_pos;
  const RowOf<ET> x(a.logits, at, a.V);
  ET* const y = static_cast<ET*>(a.out) + to;
  const bool aligned = reinterpret_cast<uintptr_t>(y) / sizeof(ET) % VEC == (uintptr_t)x.lead;
  const uint2 bound = a.bounds[row];
  const uint32_t kt = bound.x;
  const int idlim = (int)bound.y;
  if (inplace && kt == 0) return;
#pragma unroll 4
  for (int j = 0; j < 8; ++j) {
    const int q = (blockIdx.x % per * 8 + j) * WG + threadIdx.x;
    const int id = x.first(q);
    if (id >= a.V) return;
    u32x4 v = x.load(q);
    bool any = false;
    uint32_t gone = 0;
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const float l = Tr<ET>::at(v, k);
      const uint32_t o = order_of<ET>(l);
      if (o < kt || (o == kt && id + k >= idlim) || (kt && l != l)) gone |= 1u << k;
    }
    const ET none = sizeof(ET) == 2 ? (ET)0xFF80u : (ET)NEG_INF;
    if (aligned && id >= 0 && id + VEC <= a.V) {
#pragma unroll
      for (int k = 0; k < VEC; ++k)
        if (gone >> k & 1) {
          Tr<ET>::set(v, k, &none);
          any = true;
        }
      if (!inplace || any) *reinterpret_cast<u32x4*>(y + id) = v;
    } else {
#pragma unroll
      for (int k = 0; k < VEC; ++k)
        if (id + k >= 0 && id + k < a.V) {
          if (gone >> k & 1) y[id + k] = none;
          else if (!inplace) y[id + k] = x.p[id + k];
        }
    }
  }
}

// ---- host ---------------------------------------------------------------------

struct Plan {
  int nv, C, cap;
  size_t subs, lists, bounds, total;
};
size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// Chunks of 2 or 8 vectors per thread: small ones where the large ones are too
// few to fill the chip.
int make_plan(int B, int P, int V, int dtype, bool cuts, bool truncate, Plan& pl) {
  const int vec = dtype == SV_BF16 ? 8 : 4;
  const int64_t rows = (int64_t)B * P;
  auto chunks = [&](int nv) { return (V + vec - 1 + WG * nv * vec - 1) / (WG * nv * vec); };
  pl.nv = rows * chunks(8) < 1024 && chunks(2) <= MAX_CHUNKS ? 2 : 8;
  pl.C = chunks(pl.nv);
  pl.cap = cuts ? (pl.nv == 8 ? 1024 : 512) : 0;
  if (rows * pl.C > MAX_ITEMS / WG || rows > MAX_ITEMS / RW) return SV_ERR_UNSUPPORTED;
  const size_t n = (size_t)rows * pl.C;
  pl.subs = align256(n * sizeof(Chunk));
  pl.lists = align256(pl.subs + (truncate ? 0 : n * NWAVE * pl.nv * sizeof(double)));
  pl.bounds = align256(pl.lists + n * pl.cap * sizeof(uint64_t));
  pl.total = align256(pl.bounds + (truncate ? (size_t)rows * sizeof(uint2) : 0));
  return SV_OK;
}

template <typename ET, int NV>
int launch(const SampleArgs& a, bool inplace, hipStream_t st) {
  const int rows = a.B * a.P;
  (void)hipGetLastError();
  hipLaunchKernelGGL((sample_stats_kernel<ET, NV>), dim3((uint32_t)rows * a.C), dim3(WG), 0, st, a);
  if (hipGetLastError() != hipSuccess) return SV_ERR_HIP;
  hipLaunchKernelGGL((sample_row_kernel<ET, NV>), dim3(rows), dim3(RW), 0, st, a);
  if (hipGetLastError() != hipSuccess) return SV_ERR_HIP;
  if (a.out) {
    constexpr int VEC = Tr<ET>::VEC;
    const int per = (a.V + VEC - 1 + WG * 8 * VEC - 1) / (WG * 8 * VEC);
    hipLaunchKernelGGL((truncate_kernel<ET>), dim3((uint32_t)rows * per), dim3(WG), 0, st, a, per, (int)inplace);
    if (hipGetLastError() != hipSuccess) return SV_ERR_HIP;
  }
  return SV_OK;
}
template <typename ET>
int launch_nv(const SampleArgs& a, const Plan& pl, bool inplace, hipStream_t st) {
  return pl.nv == 2 ? launch<ET, 2>(a, inplace, st) : launch<ET, 8>(a, inplace, st);
}

// What both calls check; with no workspace its size is put out.
int prepare(const void* logits, int64_t row_stride, int64_t stride, const float* temperature, const int32_t* top_k,
            const float* top_p, const float* min_p, int B, int P, int V, int dtype, void* workspace,
            size_t* workspace_bytes, bool truncate, Plan& pl, SampleArgs& a) {
  if (!workspace_bytes || B < 1 || P < 1 || V < 1 || (dtype != SV_BF16 && dtype != SV_F32)) return SV_ERR_ARG;
  if (V > MAX_VOCAB || (int64_t)B * P > INT_MAX) return SV_ERR_UNSUPPORTED;
  const int rc = make_plan(B, P, V, dtype, top_k || top_p || min_p, truncate, pl);
  if (rc != SV_OK) return rc;
  if (!workspace) {
    *workspace_bytes = pl.total;
    return SV_OK;
  }
  if (*workspace_bytes < pl.total) return SV_ERR_WORKSPACE;
  if (!logits || !temperature || reinterpret_cast<uintptr_t>(workspace) % 256) return SV_ERR_ARG;
  constexpr int64_t FAR = int64_t(1) << 40;
  if (stride < V || stride > FAR || row_stride < (P - 1) * stride + V || row_stride > FAR) return SV_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(logits) % (dtype == SV_BF16 ? 2 : 4)) return SV_ERR_ARG;
  const void* words[] = {temperature, top_k, top_p, min_p};
  for (const void* p : words)
    if (reinterpret_cast<uintptr_t>(p) % 4) return SV_ERR_ARG;
  a = {};
  a.logits = logits;
  a.row = row_stride;
  a.pos = stride;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.B = B;
  a.P = P;
  a.V = V;
  a.C = pl.C;
  a.cap = pl.cap;
  char* ws = static_cast<char*>(workspace);
  a.chunks = reinterpret_cast<Chunk*>(ws);
  a.subs = truncate ? nullptr : reinterpret_cast<double*>(ws + pl.subs);
  a.lists = reinterpret_cast<uint64_t*>(ws + pl.lists);
  return SV_OK;
}

}  // namespace

extern "C" int spec_verify_sample(const void* logits, int64_t row_stride, int64_t stride, const float* uniforms,
                                  const float* temperature, const int32_t* top_k, const float* top_p,
                                  const float* min_p, int B, int P, int V, int n, int dtype, int32_t* tokens,
                                  float* logprobs, void* workspace, size_t* workspace_bytes, hipStream_t stream) {
  Plan pl;
  SampleArgs a;
  if (n < 1) return SV_ERR_ARG;
  if (n > MAX_DRAWS) return SV_ERR_UNSUPPORTED;
  const int rc = prepare(logits, row_stride, stride, temperature, top_k, top_p, min_p, B, P, V, dtype, workspace,
                         workspace_bytes, false, pl, a);
  if (rc != SV_OK || !workspace) return rc;
  if (!uniforms || !tokens || reinterpret_cast<uintptr_t>(uniforms) % 4 || reinterpret_cast<uintptr_t>(tokens) % 4 ||
      reinterpret_cast<uintptr_t>(logprobs) % 4)
    return SV_ERR_ARG;
  const size_t es = dtype == SV_BF16 ? 2 : 4, draws = (size_t)B * P * n * 4, nb = (size_t)B * 4;
  const Output out[] = {{{tokens, draws}, nullptr}, {{logprobs, draws}, nullptr}, {{workspace, pl.total}, nullptr}};
  const Array in[] = {{logits, (size_t)((B - 1) * row_stride + (P - 1) * stride + V) * es}, {uniforms, draws},
                      {temperature, nb}, {top_k, nb}, {top_p, nb}, {min_p, nb}};
  if (outputs_overlap(out, in)) return SV_ERR_ARG;
  a.uniforms = uniforms;
  a.n = n;
  a.tokens = tokens;
  a.logprobs = logprobs;
  return dtype == SV_BF16 ? launch_nv<uint16_t>(a, pl, false, stream) : launch_nv<float>(a, pl, false, stream);
}

extern "C" int spec_verify_truncate(const void* logits, int64_t row_stride, int64_t stride, const float* temperature,
                                    const int32_t* top_k, const float* top_p, const float* min_p, int B, int P, int V,
                                    int dtype, void* out, int64_t out_row_stride, int64_t out_stride, void* workspace,
                                    size_t* workspace_bytes, hipStream_t stream) {
  Plan pl;
  SampleArgs a;
  const int rc = prepare(logits, row_stride, stride, temperature, top_k, top_p, min_p, B, P, V, dtype, workspace,
                         workspace_bytes, true, pl, a);
  if (rc != SV_OK || !workspace) return rc;
  const size_t es = dtype == SV_BF16 ? 2 : 4, nb = (size_t)B * 4;
  constexpr int64_t FAR = int64_t(1) << 40;
  if (!out || reinterpret_cast<uintptr_t>(out) % es) return SV_ERR_ARG;
  if (out_stride < V || out_stride > FAR || out_row_stride < (P - 1) * out_stride + V || out_row_stride > FAR)
    return SV_ERR_ARG;
  const bool inplace = out == logits;
  if (inplace && (out_row_stride != row_stride || out_stride != stride)) return SV_ERR_ARG;
  const Array whole = {out, (size_t)((B - 1) * out_row_stride + (P - 1) * out_stride + V) * es};
  const Array read = {logits, (size_t)((B - 1) * row_stride + (P - 1) * stride + V) * es};
  if (!inplace && overlap(whole, read)) return SV_ERR_ARG;
  const Output outs[] = {{whole, nullptr}, {{workspace, pl.total}, nullptr}};
  const Array in[] = {{temperature, nb}, {top_k, nb}, {top_p, nb}, {min_p, nb}};
  if (outputs_overlap(outs, in) || overlap({workspace, pl.total}, read)) return SV_ERR_ARG;
  a.out = out;
  a.out_row = out_row_stride;
  a.out_pos = out_stride;
  a.bounds = reinterpret_cast<uint2*>(static_cast<char*>(workspace) + pl.bounds);
  return dtype == SV_BF16 ? launch_nv<uint16_t>(a, pl, inplace, stream) : launch_nv<float>(a, pl, inplace, stream);
}
