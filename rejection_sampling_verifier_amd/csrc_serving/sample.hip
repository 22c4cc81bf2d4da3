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
// their order, so atomics may form them.  A cut or a draw is the one of exact
// weights unless a border lies nearer than what their errors add up to: 2^-39
// of each weight from the series (twice where a chunk's sum is brought to the
// row's maximum), 2^-44 of the largest for each token added up, and that in the
// part of the mass and in the whole.  The sum of a whole row, which draws
// without a cut and top-p without top-k go by, is float64's by chunks: so near
// a border a result may depend on how many chunks there are.
//
// HBM reads bound it.  sample_stats_kernel reads each logit once: per chunk of
// a row the maximum and, where a rule or a draw needs it, the sum.  Where
// rules cut the row it also puts out the chunk's candidates, those that a bound
// from the chunk alone does not exclude: a chunk's top k are found among the k
// largest of its lanes' maxima, its nucleus above (1 - p) / V of its sum, min-p
// below its maximum.  sample_row_kernel finds the row's bound among the
// candidates and draws.  Candidates that fit LDS are a work-group's.  A row
// with more, up to all its tokens, is shared by several where rows are few:
// each counts its chunks (again from the logits, where a chunk's list is too
// short), and the last to arrive adds the counts up and goes on with what
// lies in the bin of the bound.

#include <algorithm>
#include <climits>
#include <cmath>

#include "cache.h"

using namespace sv;
using namespace svr;

namespace {

constexpr int MAX_VOCAB = 1 << 20;   // so that sums of weights of up to 2^43 stay below 2^63
constexpr int MAX_DRAWS = SV_MAX_NODES;
constexpr int MAX_CHUNKS = 512;
constexpr int BINS = 2048;
constexpr int EACH = BINS / WG;      // of a thread
constexpr int HELD = 2048;           // candidates of a row that LDS holds
constexpr int MANY = 16384;          // listed candidates of a row that several work-groups share
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
  uint2* bounds;      // [rows] of spec_verify_truncate; 0 for a row without a rule
  unsigned* arrived;  // [rows] work-groups that have put out their counts
  uint64_t* masses;   // [rows][BINS] of all of them
  uint32_t* counts;   // [rows][1 + share][BINS] of all of them, and of each
  int B, P, V, n, C, cap;
  int share;          // work-groups of a row
  int fill;           // sample_stats_kernel writes -inf to out, sample_row_kernel what is kept
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

// 2^y for -1000 <= y <= 0, to 2^-39 (3e-15 in the mean): y's whole part goes
// into the exponent, the rest r, at most 1/2, into a polynomial of degree 8, the
// interpolation of 2^r at Chebyshev's nodes.  y is rounded off by adding 1.5 *
// 2^52, which leaves its whole part in the sum's low bits.  fp64 additions and
// multiply-adds run at the rate of fp32 ones here.  The factors are held in
// scalar registers: as literals each would take two instructions to every
// multiply-add (256 rows of 201,088 54 us; with the series of 2^r to the 10th
// power and literals 81).
struct Series {
  double k[8];  // of r, r^2, ...; 1 of r^0
  __device__ __forceinline__ Series()
      : k{6.931471805459335e-1, 2.402265069581299e-1, 5.550410941205934e-2, 9.61812915940262e-3,
          1.3333450567999659e-3, 1.5403455852411408e-4, 1.5310079402479794e-5, 1.3255224887698904e-6} {
#pragma unroll
    for (int i = 0; i < 8; ++i) asm volatile("" : "+s"(k[i]));
  }
  __device__ __forceinline__ double exp2(double y) const {
    const double t = y + 0x1.8p52, r = y - (t - 0x1.8p52);
    double s = fma(k[7], r, k[6]);
#pragma unroll
    for (int i = 5; i >= 0; --i) s = fma(s, r, k[i]);
    s = fma(s, r, 1.0);
    return __hiloint2double(__double2hiint(s) + (__double2loint(t) << 20), __double2loint(s));
  }
};
// The weight of a logit against a maximum, c = log2(e) / T.  1 at the maximum,
// whatever it is; 0 for -inf, for all else beside +inf, and under 2^-1000,
// where float64's range ends.
__device__ __forceinline__ double weight(float l, float top, double c) {
  if (l == top) return 1.0;
  const double y = ((double)l - (double)top) * c;
  return y >= -1000.0 ? Series().exp2(y) : 0.0;
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

// Logits by their bits: whole numbers in the order of the logits, -0 just below
// 0, +NaN above everything, -NaN below.  Two bf16 at once, in 16 bits each.
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef short i16x2 __attribute__((ext_vector_type(2)));
template <typename ET>
struct Bits {
  static constexpr uint32_t INF = sizeof(ET) == 2 ? 0xFF80u : 0xFF800000u;   // of +inf; above it is NaN
  static constexpr uint32_t LEAST = sizeof(ET) == 2 ? 0x0080u : 0x00800000u;  // of the lowest finite logit
  __device__ __forceinline__ static uint32_t word(uint32_t w) {
    if (sizeof(ET) == 4) return w ^ ((uint32_t)((int32_t)w >> 31) | 0x80000000u);
    const i16x2 s = __builtin_bit_cast(i16x2, w) >> 15;
    return w ^ (__builtin_bit_cast(uint32_t, s) | 0x80008000u);
  }
  __device__ __forceinline__ static uint32_t most(uint32_t x, uint32_t y) {
    if (sizeof(ET) == 4) return x > y ? x : y;
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, x), __builtin_bit_cast(u16x2, y)));
  }
  // The largest of a vector.
  __device__ __forceinline__ static uint32_t top(const u32x4& v) {
    const uint32_t m = most(most(word(v[0]), word(v[1])), most(word(v[2]), word(v[3])));
    return sizeof(ET) == 4 ? m : (m >> 16 > (m & 0xFFFFu) ? m >> 16 : m & 0xFFFFu);
  }
  __device__ __forceinline__ static uint32_t of(ET e) {
    if constexpr (sizeof(ET) == 2) return word((uint32_t)e) & 0xFFFFu;
    else return word(__float_as_uint(e));
  }
  __device__ __forceinline__ static float logit(uint32_t k) { return logit_of<ET>(k); }
  // The least of the logits at or above a float, none of which is -inf.
  __device__ __forceinline__ static uint32_t at_least(float l) {
    uint32_t k = order_of<ET>(l);
    if (l == 0.f) --k;                                   // -0 counts as 0
    if (sizeof(ET) == 2 && (__float_as_uint(l) & 0xFFFFu)) {  // between two bf16: the next one up
      if (!(__float_as_uint(l) >> 31)) ++k;
    }
    return k > LEAST ? k : LEAST;
  }
};

__device__ __forceinline__ double shfl_xor64(double x, int m) { return __shfl_xor(x, m, 64); }

template <typename T>
__device__ __forceinline__ T wave_upto(T v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const T u = __shfl_up(v, o, 64);
    if (lane >= o) v += u;
  }
  return v;
}
template <typename ET>
__device__ __forceinline__ ET minus_inf() {
  if constexpr (sizeof(ET) == 2) return 0xFF80u;
  else return NEG_INF;
}

// ---- per chunk ----------------------------------------------------------------

constexpr int QUEUE = 512;  // vectors of a chunk that are looked through for candidates

template <typename ET, int NV>
__global__ __launch_bounds__(WG) __attribute__((amdgpu_waves_per_eu(4))) void sample_stats_kernel(SampleArgs a) {
  constexpr int VEC = Tr<ET>::VEC;
  __shared__ uint32_t shk[NWAVE];
  __shared__ int shi[NWAVE];
  __shared__ double shd[NWAVE];
  __shared__ u32x4 queue[QUEUE];
  __shared__ int ids[QUEUE];
  __shared__ int queued, found;
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  const int row = blockIdx.x / a.C, chunk = blockIdx.x % a.C;
  const int b = row / a.P;
  const RowOf<ET> x(a.logits, b * a.row + (int64_t)(row % a.P) * a.pos, a.V);
  const Rules r = rules_of(a, b);
  const int q0 = chunk * WG * NV + t;
  u32x4 v[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) v[j] = x.load(q0 + j * WG);
  const bool cut = !r.greedy && r.cut();
  if (a.fill) {
    // The output's vectors: what is kept of a row that rules cut comes later.
    ET* const y = static_cast<ET*>(a.out) + b * a.out_row + (int64_t)(row % a.P) * a.out_pos;
    const uint32_t none = Tr<ET>::NEG_INF_WORD;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int id = x.first(q0 + j * WG);
      if (id >= 0 && id + VEC <= a.V) {
        *reinterpret_cast<u32x4*>(y + id) = cut ? u32x4{none, none, none, none} : v[j];
      } else {
        for (int k = max(0, -id); k < VEC && id + k < a.V; ++k) y[id + k] = cut ? minus_inf<ET>() : x.p[id + k];
      }
    }
  }
  if (a.arrived) {  // what the row's work-groups will add to
    for (int i = chunk * WG + t; i < BINS; i += a.C * WG) {
      a.masses[(int64_t)row * BINS + i] = 0;
      a.counts[(int64_t)row * (a.share + 1) * BINS + i] = 0;
    }
    if (chunk == 0 && t == 0) a.arrived[row] = 0;
  }
  if (t == 0) queued = found = 0;
  uint32_t top_of[NV], mine = 0;
  for (bool again = true; again;) {
    mine = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      top_of[j] = Bits<ET>::top(v[j]);
      mine = mine > top_of[j] ? mine : top_of[j];
    }
    again = mine > Bits<ET>::INF;
    if (again) {  // NaN: as -inf
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (sizeof(ET) == 4) {
            if (Bits<ET>::word(v[j][k]) > Bits<ET>::INF) v[j][k] = Tr<ET>::NEG_INF_WORD;
          } else {
            if ((Bits<ET>::word(v[j][k]) & 0xFFFFu) > Bits<ET>::INF) v[j][k] = (v[j][k] & 0xFFFF0000u) | 0xFF80u;
            if (Bits<ET>::word(v[j][k]) >> 16 > Bits<ET>::INF) v[j][k] = (v[j][k] & 0xFFFFu) | 0xFF800000u;
          }
        }
    }
  }
  uint32_t key = mine;
#pragma unroll
  for (int s = 32; s; s >>= 1) key = max(key, (uint32_t)__shfl_xor((int)key, s, 64));
  if (lane == 0) shk[w] = key;
  __syncthreads();
  for (int k = 0; k < NWAVE; ++k) key = max(key, shk[k]);
  const float top = key < Bits<ET>::LEAST ? NEG_INF : Bits<ET>::logit(key);
  Chunk o = {0.0, top, NEG_INF, INT_MAX, 0};
  Chunk* const put = a.chunks + (int64_t)row * a.C + chunk;
  if (r.greedy || top == NEG_INF) {
    if (top > NEG_INF) {
      int first = INT_MAX;
      if (Bits<ET>::logit(mine) == top) {
#pragma unroll
        for (int j = NV - 1; j >= 0; --j)
#pragma unroll
          for (int k = VEC - 1; k >= 0; --k)
            if (Tr<ET>::at(v[j], k) == top) first = x.first(q0 + j * WG) + k;
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
  const double c = rate(r.T);
  if (r.whole()) {
    double all = 0.0;
    const Series series;
    const double from = top;
    double* const subs = cut || !a.subs ? nullptr : a.subs + ((int64_t)row * a.C + chunk) * (NWAVE * NV);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      double z = 0.0;
      if (top == INFINITY) {  // beside it the others weigh nothing
#pragma unroll
        for (int k = 0; k < VEC; ++k) z += Tr<ET>::at(v[j], k) == top ? 1.0 : 0.0;
      } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          if (k % 4 == 0) __builtin_amdgcn_sched_barrier(0);  // four at a time: more would not fit the registers
          z += series.exp2(fmax(((double)Tr<ET>::at(v[j], k) - from) * c, -1000.0));  // NaN too
        }
      }
      all += z;
      if (subs) {
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
      // W waves look for a logit that a W-th of k of their lanes' maxima reach;
      // the lowest of theirs is reached by k.  W is 4, fewer where waves have
      // fewer lanes with logits (a row's last chunk, a masked vocabulary).
      const int lanes = __popcll(__ballot(mine >= Bits<ET>::LEAST));
      if (lane == 0) shi[w] = lanes;
      __syncthreads();
      int q = INT_MAX;
      for (int W = NWAVE; W > 0 && q == INT_MAX; --W) {
        const int each = (r.k + W - 1) / W;
        if ((shi[0] >= each) + (shi[1] >= each) + (shi[2] >= each) + (shi[3] >= each) >= W) q = each;
      }
      uint32_t reached = q == INT_MAX ? 0 : UINT32_MAX;
      if (shi[w] >= q) {
        reached = 0;
        for (uint32_t bit = sizeof(ET) == 2 ? 1u << 15 : 1u << 31; bit; bit >>= 1)
          if (__popcll(__ballot(mine >= (reached | bit))) >= q) reached |= bit;
      }
      if (lane == 0) shk[w] = reached;
      __syncthreads();
      reached = min(min(shk[0], shk[1]), min(shk[2], shk[3]));
      if (reached >= Bits<ET>::LEAST) low = Bits<ET>::logit(reached);
      o.low = low;
    } else if (r.by_p) {
      low = under(top, r.T, (1.0 - (double)r.p) * o.sum / a.V);
    }
    if (r.m_first()) low = fmaxf(low, under(top, r.T, (double)r.m));
    // Vectors that hold a candidate stand in line in LDS, where each element is looked at by one lane.
    const uint32_t least = Bits<ET>::at_least(low);
    int n = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) n += top_of[j] >= least;
    const int upto = wave_upto(n), waves = __builtin_amdgcn_readlane(upto, 63);
    int at = 0;
    if (lane == 0 && waves) at = atomicAdd(&queued, waves);
    at = __builtin_amdgcn_readfirstlane(at) + upto - n;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (top_of[j] >= least) {
        if (at < QUEUE) {
          queue[at] = v[j];
          ids[at] = x.first(q0 + j * WG);
        }
        ++at;
      }
    __syncthreads();
    const int vectors = queued;
    if (vectors <= QUEUE) {
      uint64_t* const list = a.lists + ((int64_t)row * a.C + chunk) * a.cap;
      for (int e0 = 0; e0 < vectors * VEC; e0 += WG) {
        const int e = e0 + t;
        uint32_t k = 0;
        if (e < vectors * VEC) k = Bits<ET>::of(reinterpret_cast<const ET*>(queue)[e]);
        const bool hit = k >= least;
        const uint64_t hits = __ballot(hit);
        if (!hits) continue;
        int to = 0;
        if (lane == 0) to = atomicAdd(&found, (int)__popcll(hits));
        to = __builtin_amdgcn_readfirstlane(to) + __builtin_amdgcn_mbcnt_hi((uint32_t)(hits >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)hits, 0));
        if (hit && to < a.cap)
          list[to] = (uint64_t)order_of<ET>(Bits<ET>::logit(k)) << 32 | (uint32_t)(ids[e / VEC] + e % VEC);
      }
      __syncthreads();
      o.listed = found <= a.cap ? found : -1;
    } else {
      o.listed = -1;
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
  uint64_t sums[NWAVE];
  uint64_t before;      // what a search found
  uint32_t bin;
  int found, n, last;
};

// Over the work-group's threads, in their order: what lies before this one.
__device__ __forceinline__ uint64_t before_me(uint64_t v, uint64_t* sums, uint64_t& total) {
  const int w = threadIdx.x >> 6;
  const uint64_t inc = wave_upto((unsigned long long)v);
  if ((threadIdx.x & 63) == 63) sums[w] = inc;
  __syncthreads();
  uint64_t base = 0;
  total = 0;
#pragma unroll
  for (int k = 0; k < NWAVE; ++k) {
    if (k < w) base += sums[k];
    total += sums[k];
  }
  __syncthreads();
  return base + inc - v;
}

template <typename T>
__device__ __forceinline__ T max_of(T x, T y) { return x > y ? x : y; }

template <typename ET, int NV>
struct RowWork {
  static constexpr int VEC = Tr<ET>::VEC;
  const SampleArgs& a;
  RowLds& sh;
  const RowOf<ET>& x;
  int row;
  float top;       // the row's maximum
  double c;
  float low;       // no candidate under it
  bool lists;      // the candidates are in the chunks' lists, or else among all logits
  bool in_lds;     // the candidates are sh.held
  bool shared;     // the first counts are several work-groups'
  uint32_t kt;     // kept: order above kt, or kt itself with ids below idlim
  int idlim;

  __device__ __forceinline__ bool kept(uint32_t o, int id) const { return o > kt || (o == kt && id < idlim); }
  __device__ __forceinline__ double w(uint32_t o) const { return weight(logit_of<ET>(o), top, c); }

  // f(order, id) for the row's candidates in chunks [c0, c1).
  template <typename F>
  __device__ __forceinline__ void visit_chunks(int c0, int c1, F f) const {
    if (lists) {
      // A wave takes every fourth chunk, the lists of eight of them side by side.
      constexpr int SIDE = 8;
      const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
      const uint32_t least = order_of<ET>(low);
      const uint64_t* const list = a.lists + (int64_t)row * a.C * a.cap;
      for (int ch = c0 + wave; ch < c1; ch += NWAVE * SIDE) {
        int n[SIDE], most = 0;
#pragma unroll
        for (int j = 0; j < SIDE; ++j) {
          n[j] = ch + j * NWAVE < c1 ? __builtin_amdgcn_readfirstlane(sh.listed[ch + j * NWAVE]) : 0;
          most = max_of(most, n[j]);
        }
        for (int i = lane; i - lane < most; i += 64) {
          uint64_t e[SIDE];
#pragma unroll
          for (int j = 0; j < SIDE; ++j) {
            e[j] = 0;  // of no logit
            if (i < n[j]) e[j] = list[(int64_t)(ch + j * NWAVE) * a.cap + i];
          }
#pragma unroll
          for (int j = 0; j < SIDE; ++j)
            if (i < n[j] && (uint32_t)(e[j] >> 32) >= least) f((uint32_t)(e[j] >> 32), (int)(uint32_t)e[j]);
        }
      }
      return;
    }
    constexpr int AHEAD = 8;
    const uint32_t least = Bits<ET>::at_least(low);
#pragma unroll 1
    for (int q = c0 * NV * WG + (int)threadIdx.x; q < c1 * NV * WG; q += AHEAD * WG) {
      u32x4 v[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) v[j] = x.load(q + j * WG);
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        if (Bits<ET>::top(v[j]) < least || q + j * WG >= c1 * NV * WG) continue;
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const float l = Tr<ET>::at(v[j], k);
          if ((l >= low) & (l > NEG_INF)) f(order_of<ET>(l), x.first(q + j * WG) + k);
        }
      }
    }
  }
  // f(order, id) for the row's candidates, those with ids in [i0, i1) at least.
  template <typename F>
  __device__ __forceinline__ void visit(int i0, int i1, F f) const {
    if (in_lds) {
      for (int i = threadIdx.x; i < sh.n; i += WG) {
        const uint64_t e = sh.held[i];
        f((uint32_t)(e >> 32), (int)(uint32_t)e);
      }
      return;
    }
    const int per = WG * NV * VEC;
    visit_chunks((i0 + x.lead) / per, min(a.C, (i1 - 1 + x.lead) / per + 1), f);
  }
  // The candidates that `keep` takes, n of them at most, come to LDS if it has room.
  template <typename F>
  __device__ __forceinline__ void hold(uint64_t n, int c0, int c1, F keep) {
    if (in_lds || n > HELD) return;
    __syncthreads();
    if (threadIdx.x == 0) sh.n = 0;
    __syncthreads();
    visit_chunks(c0, c1, [&](uint32_t o, int id) {
      if (!keep(o, id)) return;
      // One addition for the lanes that are here together: each by itself would wait for the others'.
      const uint64_t here = __ballot(1);
      const int before = __builtin_amdgcn_mbcnt_hi((uint32_t)(here >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)here, 0));
      int at = 0;
      if (before == 0) at = atomicAdd(&sh.n, (int)__popcll(here));
      at = __builtin_amdgcn_readfirstlane(at) + before;
      if (at < HELD) sh.held[at] = (uint64_t)o << 32 | (uint32_t)id;
    });
    __syncthreads();
    in_lds = sh.n <= HELD;
  }
  __device__ __forceinline__ void clear() {
    __syncthreads();
    for (int i = threadIdx.x; i < BINS; i += WG) {
      sh.mass[i] = 0;
      sh.count[i] = 0;
    }
    __syncthreads();
  }
  // Of the bins, from the last down or from the first up, the one in which the
  // running sum (of counts or masses) reaches `need`: sh.found, sh.bin and what
  // lies before it.  The total comes back.
  template <bool DOWN, bool MASS>
  __device__ __forceinline__ uint64_t search(uint64_t need) {
    const int t = threadIdx.x;
    __syncthreads();
    if (t == 0) sh.found = 0;
    uint64_t v[EACH], own = 0;
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
      const int i = DOWN ? BINS - 1 - (t * EACH + k) : t * EACH + k;
      v[k] = MASS ? sh.mass[i] : sh.count[i];
      own += v[k];
    }
    uint64_t total;
    uint64_t before = before_me(own, sh.sums, total);
    if (before < need && need <= before + own) {
#pragma unroll
      for (int k = 0; k < EACH; ++k) {
        if (before < need && need <= before + v[k]) {
          sh.found = 1;
          sh.bin = DOWN ? BINS - 1 - (t * EACH + k) : t * EACH + k;
          sh.before = before;
        }
        before += v[k];
      }
    }
    __syncthreads();
    return total;
  }
  // The orders that a cut looks at first, and how many of them make a bin.
  __device__ __forceinline__ void range(uint32_t& lo, uint32_t& hi, int& shift) const {
    lo = max_of(kt, order_of<ET>(low));
    hi = order_of<ET>(top);
    shift = 0;
    while ((hi - lo) >> shift >= BINS) ++shift;
  }
  // A bin of one order has a mass of so many times its weight.
  template <bool MASS>
  __device__ __forceinline__ void add(uint32_t o, uint32_t lo, int shift) {
    const uint32_t bin = (o - lo) >> shift;
    atomicAdd(&sh.count[bin], 1u);
    if (MASS && shift) atomicAdd((unsigned long long*)&sh.mass[bin], (unsigned long long)whole_of(w(o)));
  }
  template <bool MASS>
  __device__ __forceinline__ void fill(uint32_t lo, int shift) {
    __syncthreads();
    if (!MASS || shift) return;
    for (int i = threadIdx.x; i < BINS; i += WG)
      if (sh.count[i]) sh.mass[i] = sh.count[i] * whole_of(w(lo + i));
  }
  // The first counts of a cut, of chunks [c0, c1).
  template <bool MASS>
  __device__ __forceinline__ void count(int c0, int c1) {
    uint32_t lo, hi;
    int shift;
    range(lo, hi, shift);
    clear();
    if (in_lds) visit(0, a.V, [&](uint32_t o, int id) { if (o >= lo && kept(o, id)) add<MASS>(o, lo, shift); });
    else visit_chunks(c0, c1, [&](uint32_t o, int id) { if (o >= lo && kept(o, id)) add<MASS>(o, lo, shift); });
    if (!shared) fill<MASS>(lo, shift);
    else __syncthreads();
  }
  __device__ __forceinline__ int part_begin(int part) const { return (int)((int64_t)a.C * part / a.share); }
  // The counts of a row's work-groups, each put out and added up; the last of them to arrive has the sums.
  template <bool MASS>
  __device__ __forceinline__ bool share_counts(int part) {
    const int t = threadIdx.x;
    uint32_t lo, hi;
    int shift;
    range(lo, hi, shift);
    uint32_t* const all = a.counts + (int64_t)row * (a.share + 1) * BINS;
    uint64_t* const mass = a.masses + (int64_t)row * BINS;
    for (int i = t; i < BINS; i += WG) {
      const uint32_t n = sh.count[i];
      __hip_atomic_store(all + (int64_t)(part + 1) * BINS + i, n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (!n) continue;
      __hip_atomic_fetch_add(all + i, n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (MASS && shift) __hip_atomic_fetch_add(mass + i, sh.mass[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    wait_vmem();
    __syncthreads();
    if (t == 0)
      sh.last = __hip_atomic_fetch_add(a.arrived + row, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                (unsigned)a.share - 1;
    __syncthreads();
    if (!sh.last) return false;
    uint32_t n[EACH];
    uint64_t m[EACH];
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
      n[k] = __hip_atomic_load(all + k * WG + t, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      m[k] = MASS && shift ? __hip_atomic_load(mass + k * WG + t, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0;
    }
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
      sh.count[k * WG + t] = n[k];
      sh.mass[k * WG + t] = m[k];
    }
    fill<MASS>(lo, shift);
    return true;
  }
  // Of the work-groups whose counts of this bin, one after the other, reach n:
  // its chunks, and what is left of n.  By every wave for itself.
  __device__ __forceinline__ void part_of(uint32_t bin, uint64_t& n, int& c0, int& c1) const {
    const int lane = threadIdx.x & 63;
    const uint32_t* const own = a.counts + ((int64_t)row * (a.share + 1) + 1) * BINS + bin;
    for (int p0 = 0; p0 < a.share; p0 += 64) {
      uint32_t v = 0;
      if (p0 + lane < a.share) v = __hip_atomic_load(own + (int64_t)(p0 + lane) * BINS, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      const uint32_t upto = wave_upto(v);
      const uint64_t past = __ballot(upto >= n);
      if (past) {
        const int at = __builtin_ctzll(past);
        n -= __builtin_amdgcn_readlane(upto - v, at);
        c0 = part_begin(p0 + at);
        c1 = part_begin(p0 + at + 1);
        return;
      }
      n -= __builtin_amdgcn_readlane(upto, 63);
    }
  }

  // The bound among the kept tokens of orders [from, to], WG of them at most: a
  // thread adds up what comes before its own (the row's kernel for 64 x 6 rows cut
  // by top-k and top-p 29 -> 23 us, against bins down to equal logits and ids).
  template <bool MASS>
  __device__ __forceinline__ void rank(uint32_t from, uint32_t to, uint64_t need) {
    uint64_t* const key = sh.mass;  // order << 32 | ~id: larger ones come first
    uint64_t* const mass = sh.mass + WG;
    const int t = threadIdx.x;
    __syncthreads();
    if (t == 0) sh.found = sh.last = 0;
    __syncthreads();
    visit(0, a.V, [&](uint32_t o, int id) {
      if (o < from || o > to || !kept(o, id)) return;
      const int at = atomicAdd(&sh.found, 1);
      key[at] = (uint64_t)o << 32 | (uint32_t)~id;
      if (MASS) mass[at] = whole_of(w(o));
    });
    __syncthreads();
    const int n = sh.found;
    if (t < n) {
      const uint64_t own = key[t], size = MASS ? mass[t] : 1;
      uint64_t before = 0;
#pragma unroll 4
      for (int j = 0; j < n; ++j)
        if (key[j] > own) before += MASS ? mass[j] : 1;
      if (before < need && need <= before + size) {
        sh.before = own;
        sh.last = 1;
      }
    }
    __syncthreads();
    if (!sh.last) return;
    kt = (uint32_t)(sh.before >> 32);
    idlim = (int)~(uint32_t)sh.before + 1;
  }

  // Cuts the kept set down to its first tokens in the order of logits: as many
  // as `need` (counts), or until their mass reaches it.  The first counts are
  // in the bins.
  template <bool MASS>
  __device__ __forceinline__ void cut(uint64_t need) {
    const bool all = in_lds;
    cut_down<MASS>(need);
    in_lds = all;  // what it held meanwhile were the candidates around the bound
  }
  template <bool MASS>
  __device__ __forceinline__ void cut_down(uint64_t need) {
    uint32_t lo, hi;
    int shift;
    range(lo, hi, shift);
    uint64_t left = need;
    for (bool first = true;; first = false) {
      search<true, MASS>(left);
      if (!sh.found) return;  // all of them do not reach it
      left -= sh.before;
      const uint32_t bin = sh.bin, ties = sh.count[bin];
      lo += bin << shift;
      if (shift) hi = min(hi, lo + ((1u << shift) - 1));
      if (shift == 0) {
        // Of the tokens with this logit as many as it takes, the lowest ids first.
        uint64_t n = left;
        if (MASS) {
          const uint64_t one = whole_of(w(lo));
          n = one ? (left + one - 1) / one : ties;
        }
        if (lo != kt) idlim = INT_MAX;
        kt = lo;
        if (n >= ties) return;
        if (ties <= WG && !(shared && first)) {
          rank<false>(lo, lo, n);
          return;
        }
        const int limit = idlim;
        int c0 = 0, c1 = a.C;
        if (shared && first) part_of(bin, n, c0, c1);
        hold(c0 || c1 < a.C ? 0 : ties, c0, c1, [&](uint32_t o, int id) { return o == lo && id < limit; });
        const int per = WG * NV * VEC;
        int i0 = max(0, c0 * per - x.lead), i1 = min(a.V, c1 * per - x.lead);
        const int last = i1;
        while ((i1 - i0 - 1) >> shift >= BINS) ++shift;
        for (int pass = 0; pass < 2; ++pass) {
          clear();
          visit(i0, i1, [&](uint32_t o, int id) {
            if (o == lo && id < limit && id >= i0 && id < i1) atomicAdd(&sh.count[(id - i0) >> shift], 1u);
          });
          search<false, false>(n);
          n -= sh.before;
          i0 += sh.bin << shift;
          i1 = min(last, i0 + (1 << shift));
          shift = 0;
        }
        idlim = i0 + 1;
        return;
      }
      if (ties <= WG) {
        rank<MASS>(lo, hi, left);
        return;
      }
      shift = 0;
      while ((hi - lo) >> shift >= BINS) ++shift;
      const uint32_t from = lo, to = hi;
      hold(ties, 0, a.C, [&](uint32_t o, int id) { return o >= from && o <= to && kept(o, id); });
      clear();
      visit(0, a.V, [&](uint32_t o, int id) {
        if (o >= from && o <= to && kept(o, id)) add<MASS>(o, from, shift);
      });
      fill<MASS>(from, shift);
    }
  }
};

template <typename ET, int NV>
__global__ __launch_bounds__(WG) __attribute__((amdgpu_waves_per_eu(3))) void sample_row_kernel(SampleArgs a) {
  constexpr int VEC = Tr<ET>::VEC, SUBS = NWAVE * NV;
  __shared__ RowLds sh;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int row = blockIdx.x / a.share, part = blockIdx.x % a.share, b = row / a.P;
  const Rules r = rules_of(a, b);
  if (part && (r.greedy || !r.cut())) return;
  const RowOf<ET> x(a.logits, b * a.row + (int64_t)(row % a.P) * a.pos, a.V);
  const Chunk* chunks = a.chunks + (int64_t)row * a.C;
  int32_t* tokens = a.tokens ? a.tokens + (int64_t)row * a.n : nullptr;
  float* logprobs = a.logprobs ? a.logprobs + (int64_t)row * a.n : nullptr;

  // The row's maximum, by every wave for itself.
  float max = NEG_INF, low = NEG_INF;
  int listed = 0;  // -1: more than the lists hold
  for (int i0 = 0; i0 < a.C; i0 += 64) {
    const int i = i0 + lane;
    Chunk o = {0.0, NEG_INF, NEG_INF, INT_MAX, 0};
    if (i < a.C) o = chunks[i];
    if (i < a.C && wave == 0) {
      sh.top[i] = o.top;
      sh.listed[i] = o.listed;
      sh.upto[i] = o.sum;
    }
    max = fmaxf(max, o.top);
    low = fmaxf(low, o.low);
    const uint64_t over = __ballot(o.listed < 0);
    int n = o.listed;
#pragma unroll
    for (int s = 32; s; s >>= 1) n += __shfl_xor(n, s, 64);
    listed = over || listed < 0 ? -1 : listed + n;
  }
  max = wave_max(max);
  low = wave_max(low);
  // Lists of up to MANY are gone through by one work-group, and those of them that the row's own bound leaves held in LDS.
  const bool large = listed < 0 || listed > MANY;
  if (part && !large) return;
  if (max == NEG_INF || r.greedy) {
    if (part) return;
    __syncthreads();
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
    if (a.bounds && t == 0) a.bounds[row] = make_uint2(r.greedy || !r.cut() ? 0 : Bits<ET>::LEAST, INT_MAX);
    return;
  }
  const double c = rate(r.T);
  __syncthreads();
  // Sums of the chunks against the row's maximum, added up in order.
  if (r.whole()) {
    if (wave == 0) {
      double base = 0.0;
      for (int i0 = 0; i0 < a.C; i0 += 64) {
        const int i = i0 + lane;
        double z = 0.0;
        if (i < a.C && sh.top[i] > NEG_INF) z = sh.upto[i] * weight(sh.top[i], max, c);
        z = wave_upto(z) + base;
        if (i < a.C) sh.upto[i] = z;
        base = __shfl(z, 63, 64);
      }
    }
    __syncthreads();
  }

  if (!r.cut()) {
    if (a.bounds && t == 0) a.bounds[row] = make_uint2(0, INT_MAX);
    const double total = sh.upto[a.C - 1];
    for (int d = wave; d < a.n; d += NWAVE) {
      const float u = a.uniforms[(int64_t)row * a.n + d];
      double left = (double)(u > 0.f ? fminf(u, 0x1.fffffep-1f) : 0.f) * total;
      // The first chunk whose running sum passes it; the last with any weight if rounding leaves none.
      int ch = 0;
      for (int i0 = 0; i0 < a.C; i0 += 64) {
        const int i = i0 + lane;
        const double z = i < a.C ? sh.upto[i] : 0.0, y = i > 0 && i < a.C ? sh.upto[i - 1] : 0.0;
        const uint64_t some = __ballot(z > y);
        if (some) ch = i0 + 63 - __builtin_clzll(some);
        const uint64_t past = __ballot(z > left);
        if (past) {
          ch = i0 + __builtin_ctzll(past);
          break;
        }
      }
      const float top = sh.top[ch];
      const double of = weight(top, max, c), least = 0x1p-1000 / of;  // what weighs less against the chunk's maximum weighs nothing
      left = (left - (ch ? sh.upto[ch - 1] : 0.0)) / of;
      const double own = lane < SUBS ? a.subs[((int64_t)row * a.C + ch) * SUBS + lane] : 0.0;
      const double upto = wave_upto(own);
      // Of the wave's vectors whose running sum passes what is left, the first that hold a token with a weight; if
      // there are none, the last that do.  A sum alone does not tell: 2^-1000 is in it for each -inf.  The chunk's
      // maximum is in one of them.
      const uint64_t may = __ballot(own >= least);
      uint64_t up = __ballot(upto > left) & may, down = may & ~up, any = 0;
      u32x4 v;
      int q = 0;
      double e = 0.0, before = 0.0;
      while (!any && (up | down)) {
        const int sub = up ? __builtin_ctzll(up) : 63 - __builtin_clzll(down);
        up &= ~(1ull << sub);
        down &= ~(1ull << sub);
        q = ch * WG * NV + sub / NWAVE * WG + sub % NWAVE * 64 + lane;
        v = x.load(q);
        e = 0.0;
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const double g = weight(logit_at<ET>(v, k), top, c);
          e += g >= least ? g : 0.0;
        }
        any = __ballot(e > 0.0);
        before = __shfl(upto - own, sub, 64);
      }
      left -= before;
      const double z = wave_upto(e);
      const uint64_t past = __ballot(e > 0.0 && z > left);
      const int who = past ? __builtin_ctzll(past) : any ? 63 - __builtin_clzll(any) : 0;
      if (lane == who) {
        double sum = z - e;
        int id = -1;
        float l = 0.f;
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const float y = logit_at<ET>(v, k);
          const double w = weight(y, top, c), g = w >= least ? w : 0.0;
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

  RowWork<ET, NV> work{a, sh, x, row, max, c, low, listed >= 0, false, false, 0, INT_MAX};
  const bool mass_first = r.by_p && !r.k;
  const double sum = mass_first ? sh.upto[a.C - 1] : 0.0;
  if (mass_first) work.low = under(max, r.T, (1.0 - (double)r.p) * sum / a.V);
  if (r.m_first()) work.low = fmaxf(work.low, under(max, r.T, (double)r.m));
  if (part && !r.k && !r.by_p) return;
  if (work.lists && (!large || a.share == 1)) work.hold(0, 0, a.C, [](uint32_t, int) { return true; });
  if (r.k || r.by_p) {
    work.shared = large && a.share > 1;
    const int c0 = work.shared ? work.part_begin(part) : 0, c1 = work.shared ? work.part_begin(part + 1) : a.C;
    if (mass_first) work.template count<true>(c0, c1);
    else work.template count<false>(c0, c1);
    if (work.shared && !(mass_first ? work.template share_counts<true>(part) : work.template share_counts<false>(part)))
      return;
    if (mass_first) {
      const double need = ceil((double)r.p * (sum * ONE));
      work.template cut<true>(need >= 1.0 ? (uint64_t)need : 1);
    } else {
      work.template cut<false>(r.k);
      work.hold(r.k, 0, a.C, [&](uint32_t o, int id) { return work.kept(o, id); });
    }
    work.shared = false;
    if (r.by_p && r.k) {
      work.template count<true>(0, a.C);
      const uint64_t total = work.template search<true, true>(0);
      const double need = ceil((double)r.p * (double)total);
      work.template cut<true>(need >= 1.0 ? (uint64_t)need : 1);
    }
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
    // -inf, and NaN as it, is left out by any rule, also by one that leaves all else.
    const bool all = work.kt < Bits<ET>::LEAST;
    if (t == 0) a.bounds[row] = all ? make_uint2(Bits<ET>::LEAST, INT_MAX) : make_uint2(work.kt, (uint32_t)work.idlim);
    return;
  }
  if (logit_of<ET>(work.kt) > work.low) work.low = logit_of<ET>(work.kt);
  if (a.fill) {
    ET* const y = static_cast<ET*>(a.out) + b * a.out_row + (int64_t)(row % a.P) * a.out_pos;
    work.visit(0, a.V, [&](uint32_t o, int id) {
      if (work.kept(o, id)) y[id] = x.p[id];
    });
    return;
  }

  // The kept tokens' masses by ids, then by the ids of a draw's bin.
  int shift = 0;
  while ((a.V - 1) >> shift >= BINS) ++shift;
  uint64_t* const fine = reinterpret_cast<uint64_t*>(sh.count);  // up to BINS / 2 ids of a bin
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
    for (int i = t; i < 1 << shift; i += WG) fine[i] = 0;
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
        const uint64_t z = wave_upto((unsigned long long)own);
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

template <typename ET, int NV>
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
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int q = (blockIdx.x % per * NV + j) * WG + threadIdx.x;
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
    const ET none = minus_inf<ET>();
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
  int nv, C, cap, share;
  bool fill;
  size_t subs, lists, bounds, arrived, masses, counts, total;
};
size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// Work-groups of a row in truncate_kernel, which takes half a chunk.
int cut_groups(int nv, int V, int vec) { return (V + vec - 1 + WG * (nv / 2) * vec - 1) / (WG * (nv / 2) * vec); }

// Chunks of 8 vectors per thread, or of 2 for few rows, whose chunks would be
// too few: six rows of 128,256 cut by top-p 33 us against 106, both kernels, as
// four times as many work-groups count a row; but 16 rows of 151,936 with top-k
// 44 against 23, as the k-th largest of a small chunk leaves more candidates.
int make_plan(int B, int P, int V, int dtype, bool cuts, bool truncate, Plan& pl) {
  const int vec = dtype == SV_BF16 ? 8 : 4;
  const int64_t rows = (int64_t)B * P;
  auto chunks = [&](int nv) { return (V + vec - 1 + WG * nv * vec - 1) / (WG * nv * vec); };
  pl.nv = rows * chunks(8) < 64 && chunks(2) <= MAX_CHUNKS ? 2 : 8;
  pl.fill = truncate && rows * chunks(8) >= 1024;
  pl.C = chunks(pl.nv);
  pl.cap = cuts ? (pl.nv == 8 ? 1024 : 512) : 0;
  if (rows * (truncate ? cut_groups(pl.nv, V, vec) : pl.C) > MAX_ITEMS / WG) return SV_ERR_UNSUPPORTED;
  // Work-groups of a row for the case that it has many candidates: two to a CU.
  pl.share = cuts ? (int)std::max<int64_t>(1, std::min<int64_t>(pl.C, 512 / rows)) : 1;
  const size_t n = (size_t)rows * pl.C;
  pl.subs = align256(n * sizeof(Chunk));
  pl.lists = align256(pl.subs + (truncate ? 0 : n * NWAVE * pl.nv * sizeof(double)));
  pl.bounds = align256(pl.lists + n * pl.cap * sizeof(uint64_t));
  pl.arrived = align256(pl.bounds + (truncate ? (size_t)rows * sizeof(uint2) : 0));
  const size_t bins = pl.share > 1 ? (size_t)rows * BINS : 0;
  pl.masses = align256(pl.arrived + (bins ? (size_t)rows * sizeof(unsigned) : 0));
  pl.counts = pl.masses + bins * sizeof(uint64_t);
  pl.total = pl.counts + bins * (1 + pl.share) * sizeof(uint32_t);
  return SV_OK;
}

template <typename ET, int NV>
int launch(const SampleArgs& a, bool inplace, hipStream_t st) {
  const int rows = a.B * a.P;
  (void)hipGetLastError();
  hipLaunchKernelGGL((sample_stats_kernel<ET, NV>), dim3((uint32_t)rows * a.C), dim3(WG), 0, st, a);
  if (hipGetLastError() != hipSuccess) return SV_ERR_HIP;
  hipLaunchKernelGGL((sample_row_kernel<ET, NV>), dim3((uint32_t)rows * a.share), dim3(WG), 0, st, a);
  if (hipGetLastError() != hipSuccess) return SV_ERR_HIP;
  if (a.bounds) {
    const int per = cut_groups(NV, a.V, Tr<ET>::VEC);
    hipLaunchKernelGGL((truncate_kernel<ET, NV / 2>), dim3((uint32_t)rows * per), dim3(WG), 0, st, a, per, (int)inplace);
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
  a.share = pl.share;
  if (pl.share > 1) {
    a.arrived = reinterpret_cast<unsigned*>(ws + pl.arrived);
    a.masses = reinterpret_cast<uint64_t*>(ws + pl.masses);
    a.counts = reinterpret_cast<uint32_t*>(ws + pl.counts);
  }
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
  // Large batches get -inf written as they are read, and the kept logits after that, where vectors of both are alike
  // (64 x 6 rows of 151,936: the third kernel alone takes 42 us).  In small ones that kernel takes 4, and a row with many tokens left would be gone through by one work-group.
  const int64_t vec = 16 / es;
  const int64_t apart = (reinterpret_cast<intptr_t>(out) - reinterpret_cast<intptr_t>(logits)) / (int64_t)es;
  a.fill = pl.fill && !inplace && apart % vec == 0 && (out_row_stride - row_stride) % vec == 0 &&
           (out_stride - stride) % vec == 0;
  if (!a.fill) a.bounds = reinterpret_cast<uint2*>(static_cast<char*>(workspace) + pl.bounds);
  return dtype == SV_BF16 ? launch_nv<uint16_t>(a, pl, inplace, stream) : launch_nv<float>(a, pl, inplace, stream);
}
