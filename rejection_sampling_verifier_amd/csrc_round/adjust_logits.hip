// Penalties for repeated tokens, biases and grammar masks on the logits of a
// verification round (spec_verify_adjust_logits), for gfx950.
//
// Mathematics: per logit at most one division or product, two subtractions
// and one addition, on few tokens; every other logit is copied or set to
// -inf.  The call is bound by HBM: it reads and writes each logit once
// (where a mask forbids all of a vector's tokens, it is not read).
//
// One work-group per (row, chunk of CH token ids, group of positions).  It
// first counts the row's history inside its chunk: a direct-addressed table
// of counts in LDS, built by integer atomics, so the order of the tokens
// does not matter and there is nothing to sort or to clear in memory.  The
// history is read again by each of a row's chunks, out of L2.  Then it
// streams its chunk of every position, 16 bytes per lane; a bit per id says
// which vectors hold a counted or biased token and take the slow path.
// Drafted tokens are not counted in the table: a position's own are those
// of its path (a 64-bit mask over the drafted tokens) that fall into the
// chunk, usually none or one, and the slow path adds them, so positions
// need no barrier between them.

#include <cstdint>

#include "spec_verify.h"
#include "sv_device.h"

using namespace sv;

namespace {

constexpr int CH = 4096;                 // token ids per chunk
constexpr int GRID_WANTED = 1024;        // work-groups that fill the chip; below, positions are split too
constexpr uint32_t IN_PROMPT = 1u << 31; // table entry: occurs in the prompt; the rest counts n(x)

struct AdjustArgs {
  const void* in;
  void* out;
  int64_t in_row, in_pos, out_row, out_pos;
  const int32_t* tokens;
  const int32_t* parents;
  int64_t tokens_stride;
  sv_controls c;
  int P, V, C, PG;  // positions, ids, chunks, position groups
  int words;        // words of a mask row
  int penalties, inplace;
};

// 16-byte access at any element alignment (the memory system splits what
// crosses a line).
typedef u32x4 u32x4_u __attribute__((aligned(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef i32x4 i32x4_u __attribute__((aligned(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

template <typename ET> struct Out;
template <> struct Out<uint16_t> {
  static constexpr uint16_t NEG = 0xFF80u;
  // Round to nearest even, the conversion's own rounding.
  __device__ __forceinline__ static void pack(u32x4& v, const float (&x)[8]) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      v[k] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x[2 * k], x[2 * k + 1]}, bf16x2));
  }
  __device__ __forceinline__ static uint16_t one(const u32x4& v, int k) { return (uint16_t)(v[k >> 1] >> (16 * (k & 1))); }
  // Words whose two tokens are cut by the allowed bits.
  __device__ __forceinline__ static void cut(u32x4& v, uint32_t allow) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t w = v[k];
      if (!((allow >> (2 * k)) & 1)) w = (w & 0xFFFF0000u) | 0xFF80u;
      if (!((allow >> (2 * k + 1)) & 1)) w = (w & 0x0000FFFFu) | 0xFF800000u;
      v[k] = w;
    }
  }
};
template <> struct Out<float> {
  static constexpr float NEG = NEG_INF;
  __device__ __forceinline__ static void pack(u32x4& v, const float (&x)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = __float_as_uint(x[k]);
  }
  __device__ __forceinline__ static float one(const u32x4& v, int k) { return __uint_as_float(v[k]); }
  __device__ __forceinline__ static void cut(u32x4& v, uint32_t allow) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (!((allow >> k) & 1)) v[k] = 0xFF800000u;
  }
};

// LDS: the chunk's tables.  `bias` holds 1 + the number of the last entry of
// the bias list for the id.
template <bool BIAS>
struct Tables {
  alignas(16) uint32_t count[CH];
  alignas(16) int32_t bias[BIAS ? CH : 1];
  uint32_t touched[CH / 32];
  int32_t local[64];     // drafted tokens' places in the chunk
  uint64_t path[64];     // tree: nodes on the path root .. v
  uint64_t here;         // drafted tokens inside the chunk
};

// The path masks of a tree, by one wave: lane v starts with itself and its
// parent, and each step doubles the length of the paths known.  The root's
// bit is left out of the masks.
__device__ __forceinline__ uint64_t path_mask(const int32_t* par, int N) {
  const int v = threadIdx.x & 63;
  int up = -1;
  if (v > 0 && v < N) {
    const int p = par[v];
    up = p >= 0 && p < v ? p : -1;
  }
  uint64_t m = v > 0 ? 1ull << v : 0;
#pragma unroll
  for (int s = 0; s < 6; ++s) {
    const int src = up < 0 ? v : up;
    const uint32_t lo = __shfl((uint32_t)m, src, 64), hi = __shfl((uint32_t)(m >> 32), src, 64);
    const int next = __shfl(up, src, 64);
    if (up >= 0) {
      m |= ((uint64_t)hi << 32) | lo;
      up = next;
    }
  }
  return m;
}

template <typename ET, bool BIAS>
__global__ __launch_bounds__(WG) void adjust_logits_kernel(AdjustArgs a) {
  constexpr int VEC = Tr<ET>::VEC;
  constexpr int NV = CH / (WG * VEC);  // vectors per thread and position
  __shared__ Tables<BIAS> sh;
  const int t = threadIdx.x;
  const int pg = blockIdx.x % a.PG;
  const int chunk = (blockIdx.x / a.PG) % a.C;
  const int b = blockIdx.x / a.PG / a.C;
  const int lo = chunk * CH, len = min(CH, a.V - lo);

  for (int i = t; i < CH / 4; i += WG) {
    reinterpret_cast<u32x4*>(sh.count)[i] = u32x4{0, 0, 0, 0};
    if (BIAS) reinterpret_cast<u32x4*>(sh.bias)[i] = u32x4{0, 0, 0, 0};
  }
  if (t < CH / 32) sh.touched[t] = 0;
  const int drafted = a.penalties && a.tokens ? (a.parents ? a.P : a.P - 1) : 0;
  if (t < 64) {
    int at = -1;
    if (t < drafted && (!a.parents || t > 0)) {
      const uint32_t d = (uint32_t)a.tokens[b * a.tokens_stride + t] - (uint32_t)lo;
      at = d < (uint32_t)len ? (int)d : -1;
    }
    sh.local[t] = at;
    const uint64_t m = __ballot(at >= 0);
    if (t == 0) sh.here = m;
    if (a.parents) sh.path[t] = path_mask(a.parents + (int64_t)b * a.P, a.P);
  }
  __syncthreads();
  if (t < 64 && sh.local[t] >= 0) atomicOr(&sh.touched[sh.local[t] >> 5], 1u << (sh.local[t] & 31));
  if (a.penalties && a.c.history) {
    const int32_t* h = a.c.history + b * a.c.history_stride;
    const int64_t n = min((int64_t)max(a.c.history_lens[b], 0), a.c.history_stride);
    const int64_t np = a.c.prompt_lens ? (int64_t)max(a.c.prompt_lens[b], 0) : 0;
    auto take = [&](int tok, int64_t j) {
      const uint32_t d = (uint32_t)tok - (uint32_t)lo;
      if (d < (uint32_t)len) {
        if (j < np) atomicOr(&sh.count[d], IN_PROMPT);
        else atomicAdd(&sh.count[d], 1u);
        atomicOr(&sh.touched[d >> 5], 1u << (d & 31));
      }
    };
    const int64_t n4 = n / 4;
    for (int64_t j = t; j < n4; j += WG) {
      const i32x4 w = *reinterpret_cast<const i32x4_u*>(h + 4 * j);
#pragma unroll
      for (int k = 0; k < 4; ++k) take(w[k], 4 * j + k);
    }
    if (4 * n4 + t < n) take(h[4 * n4 + t], 4 * n4 + t);
  }
  if (BIAS) {
    const int32_t* ids = a.c.bias_ids + b * a.c.bias_stride;
    const int n = (int)(a.c.bias_lens ? min((int64_t)max(a.c.bias_lens[b], 0), a.c.bias_stride) : a.c.bias_stride);
    for (int e = t; e < n; e += WG) {
      const uint32_t d = (uint32_t)ids[e] - (uint32_t)lo;
      if (d < (uint32_t)len) {
        atomicMax(&sh.bias[d], e + 1);
        atomicOr(&sh.touched[d >> 5], 1u << (d & 31));
      }
    }
  }
  __syncthreads();

  const float r = a.c.repetition ? a.c.repetition[b] : 1.f;
  const float freq = a.c.frequency ? a.c.frequency[b] : 0.f;
  const float pres = a.c.presence ? a.c.presence[b] : 0.f;
  const uint64_t here = sh.here;
  constexpr uint32_t ALL = (1u << VEC) - 1;
  const int p0 = (int)((int64_t)a.P * pg / a.PG), p1 = (int)((int64_t)a.P * (pg + 1) / a.PG);

  for (int i = p0; i < p1; ++i) {
    const ET* src = static_cast<const ET*>(a.in) + b * a.in_row + i * a.in_pos + lo;
    ET* dst = static_cast<ET*>(a.out) + b * a.out_row + i * a.out_pos + lo;
    const uint32_t* mask = nullptr;
    if (a.c.mask) {
      const int64_t row = a.c.mask_rows ? (int64_t)a.c.mask_rows[(int64_t)b * a.P + i] : (int64_t)b * a.P + i;
      if (row >= 0 && row < a.c.num_masks) mask = a.c.mask + row * a.words + lo / 32;
    }
    const uint64_t path = here & (a.parents ? sh.path[i & 63] : i >= 64 ? ~0ull : (1ull << i) - 1);

    u32x4 v[NV];
    uint32_t allow[NV], touch[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = (j * WG + t) * VEC;
      allow[j] = ALL;
      touch[j] = 0;
      if (e < len) {
        if (mask) allow[j] = (mask[e >> 5] >> (e & 31)) & ALL;
        touch[j] = (sh.touched[e >> 5] >> (e & 31)) & ALL;
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = (j * WG + t) * VEC;
      const bool need = allow[j] && (!a.inplace || touch[j] || allow[j] != ALL);
      if (need) {
        if (e + VEC <= len) v[j] = *reinterpret_cast<const u32x4_u*>(src + e);
        else {
          v[j] = u32x4{0, 0, 0, 0};
#pragma unroll
          for (int k = 0; k < VEC; ++k)
            if (e + k < len) Tr<ET>::set(v[j], k, src + e + k);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = (j * WG + t) * VEC;
      if (e >= len || (a.inplace && !touch[j] && allow[j] == ALL)) continue;
      if (!allow[j]) {
        const uint32_t f = Tr<ET>::NEG_INF_WORD;
        v[j] = u32x4{f, f, f, f};
      } else {
        if (touch[j]) {
          float x[VEC];
          uint64_t more = 0;  // drafted tokens: a byte per id of the vector
          for (uint64_t m = path; m; m &= m - 1) {
            const uint32_t d = (uint32_t)sh.local[__builtin_ctzll(m)] - (uint32_t)e;
            if (d < (uint32_t)VEC) more += 1ull << (8 * d);
          }
#pragma unroll
          for (int k = 0; k < VEC; ++k) {
            x[k] = Tr<ET>::at(v[j], k);
            if (!((touch[j] >> k) & 1)) continue;
            const uint32_t c = sh.count[e + k];
            const uint32_t d = (uint32_t)(more >> (8 * k)) & 0xFFu;
            const uint32_t n = (c & ~IN_PROMPT) + d;
            if (c | d) x[k] = x[k] > 0.f ? x[k] / r : x[k] * r;
            if (n) x[k] = (x[k] - freq * (float)n) - pres;
            if (BIAS) {
              const int at = sh.bias[e + k];
              if (at) x[k] = x[k] + a.c.bias_values[b * a.c.bias_stride + at - 1];
            }
          }
          Out<ET>::pack(v[j], x);
        }
        if (allow[j] != ALL) Out<ET>::cut(v[j], allow[j]);
      }
      if (e + VEC <= len) *reinterpret_cast<u32x4_u*>(dst + e) = v[j];
      else {
#pragma unroll
        for (int k = 0; k < VEC; ++k)
          if (e + k < len) dst[e + k] = Out<ET>::one(v[j], k);
      }
    }
  }
}

// Bytes [first, last] that a strided [B, P, V] tensor spans.
struct Span { uintptr_t lo, hi; };
Span span(const void* p, int64_t row, int64_t pos, int B, int P, int V, int64_t es) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + (uintptr_t)(((B - 1) * row + (P - 1) * pos + V) * es)};
}

}  // namespace

extern "C" int spec_verify_adjust_logits(const void* logits, int64_t row_stride, int64_t stride, const int32_t* tokens,
                                         int64_t tokens_stride, const int32_t* parents, const sv_controls* controls,
                                         int B, int P, int V, int dtype, void* out, int64_t out_row_stride,
                                         int64_t out_stride, hipStream_t stream) {
  if (!logits || !out || !controls || B < 1 || P < 1 || V < 1 || (dtype != SV_BF16 && dtype != SV_F32))
    return SV_ERR_ARG;
  if (P > (parents ? SV_MAX_NODES : SV_MAX_K + 1)) return SV_ERR_UNSUPPORTED;
  const int64_t es = dtype == SV_BF16 ? 2 : 4;
  constexpr int64_t FAR = int64_t(1) << 56;  // strides whose offsets stay inside 64 bits
  if (stride < V || out_stride < V || stride > FAR / (P * es) || out_stride > FAR / (P * es)) return SV_ERR_ARG;
  if (B > 1 && (row_stride < (P - 1) * stride + V || out_row_stride < (P - 1) * out_stride + V ||
                row_stride > FAR / (B * es) || out_row_stride > FAR / (B * es)))
    return SV_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(logits) % es || reinterpret_cast<uintptr_t>(out) % es) return SV_ERR_ARG;
  AdjustArgs a;
  a.c = *controls;
  a.inplace = logits == out;
  if (a.inplace) {
    if ((P > 1 && stride != out_stride) || (B > 1 && row_stride != out_row_stride)) return SV_ERR_ARG;
  } else {
    const Span x = span(logits, row_stride, stride, B, P, V, es);
    const Span y = span(out, out_row_stride, out_stride, B, P, V, es);
    if (x.lo < y.hi && y.lo < x.hi) return SV_ERR_ARG;
  }
  a.penalties = a.c.repetition || a.c.presence || a.c.frequency;
  if (a.penalties) {
    if (a.c.history && (!a.c.history_lens || a.c.history_stride < 0 || a.c.history_stride > INT32_MAX)) return SV_ERR_ARG;
    if (P > 1 && (!tokens || tokens_stride < (parents ? P : P - 1) || tokens_stride > INT32_MAX)) return SV_ERR_ARG;
  }
  if (a.c.bias_ids && (!a.c.bias_values || a.c.bias_stride < 0 || a.c.bias_stride > INT32_MAX - 1)) return SV_ERR_ARG;
  if (a.c.mask && (a.c.num_masks < 0 || (!a.c.mask_rows && a.c.num_masks < (int64_t)B * P))) return SV_ERR_ARG;
  a.in = logits;
  a.out = out;
  a.in_row = row_stride;
  a.in_pos = stride;
  a.out_row = out_row_stride;
  a.out_pos = out_stride;
  a.tokens = P > 1 ? tokens : nullptr;
  a.parents = a.penalties && P > 1 ? parents : nullptr;
  a.tokens_stride = tokens_stride;
  a.P = P;
  a.V = V;
  a.C = (V - 1) / CH + 1;
  a.words = (V - 1) / 32 + 1;
  const int64_t groups = (int64_t)B * a.C;
  a.PG = (int)(groups >= GRID_WANTED ? 1 : (GRID_WANTED + groups - 1) / groups);
  if (a.PG > P) a.PG = P;
  if (groups * a.PG > INT32_MAX) return SV_ERR_UNSUPPORTED;
  const bool bias = a.c.bias_ids && a.c.bias_stride > 0;
  void (*const k)(AdjustArgs) =
      dtype == SV_BF16 ? (bias ? adjust_logits_kernel<uint16_t, true> : adjust_logits_kernel<uint16_t, false>)
                       : (bias ? adjust_logits_kernel<float, true> : adjust_logits_kernel<float, false>);
  (void)hipGetLastError();
  hipLaunchKernelGGL(k, dim3((uint32_t)(groups * a.PG)), dim3(WG), 0, stream, a);
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
}
