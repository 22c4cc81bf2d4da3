// Penalties for repeated tokens, biases and grammar masks on the logits of a
// verification step (spec_verify_adjust_logits), for gfx950.
//
// Mathematics: per logit at most one division or product, two subtractions
// and one addition, on few tokens; every other logit is copied or set to
// -inf.  The call is bound by HBM: it reads and writes each logit once
// (where a mask forbids all of a vector's tokens, it is not read).
//
// One work-group per (row, chunk of token ids, group of positions).  It
// first counts the row's history inside its chunk: a direct-addressed table
// of counts in LDS, built by integer atomics, so the order of the tokens
// does not matter and there is nothing to sort or to clear in memory.  The
// history is read again by each of a row's chunks, out of L2.  A bit per id
// tells which ids are counted, drafted or biased, and their list is made of
// it.  Then it streams its chunk of every position, 16 bytes per lane and
// eight such loads at once.  A wave whose window of 64 vectors holds listed
// ids puts those vectors into LDS, changes the ids there, one lane each, and
// takes the vectors back: doing it in place, all lanes for all ids of a
// vector, made the kernel bound by its arithmetic (538 against 450 us on 256
// rows of 8 positions of 201,088 ids with every control).  The next positions'
// loads are issued before the present ones are changed, the first before the
// tables are made (450 -> 402 us), and loads and stores pass the caches by
// (402 -> 391 us; 64 rows of 6 positions of 151,936 ids: 57 -> 51 us, 4.6 TB/s,
// where a large copy reaches 4.9).  Drafted tokens are
// not counted in the table: a position's own are those of its path (a 64-bit
// mask over the drafted tokens) that fall into the chunk, usually none or
// one, so positions need no barrier between them.
//
// A token's bias is its last entry's: a bit per id and the bits' ranks give
// each biased id a place in LDS, where a maximum over entry numbers settles
// it once per work-group.  (A search of the chunk's entries by each listed id
// at each position: 388 against 306 us with every control, 300 entries a row,
// and 52.9 ms against 48 us with 20,000 entries side by side in 8 rows of 8
// positions of 131,072 ids.)  Rows with more entries than places get chunks of
// as many ids as there are places, which takes half of the lanes.

#include <cstdint>

#include "spec_verify.h"
#include "sv_device.h"

using namespace sv;

namespace {

constexpr int CH = 4096;                 // token ids per chunk at most
constexpr int64_t MAX_GROUPS = UINT32_MAX / WG;  // a launch has fewer than 2^32 work-items
constexpr int GRID_WANTED = 1024;        // work-groups that fill the chip; below, positions are split too
constexpr uint32_t IN_PROMPT = 1u << 31; // table entry: occurs in the prompt;
constexpr uint32_t BIASED = 1u << 30;    // has a bias; the rest counts n(x)
constexpr int64_t MAX_ENTRIES = (1 << 30) - 1024;  // of a row's history or biases: a count stays below BIASED, an index in 32 bits
constexpr int BIASES = 2048;             // biased ids of a chunk that LDS holds; rows with more entries get chunks of so many

struct AdjustArgs {
  const void* in;
  void* out;
  int64_t in_row, in_pos, out_row, out_pos;
  const int32_t* tokens;
  const int32_t* parents;
  int64_t tokens_stride;
  sv_controls c;
  int P, V, C, PG;  // positions, ids, chunks, position groups
  int chunk;        // ids of a chunk
  int words;        // words of a mask row
  int penalties, inplace;
};

// 16-byte access at any element alignment (the memory system splits what
// crosses a line).
typedef u32x4 u32x4_u __attribute__((aligned(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef i32x4 i32x4_u __attribute__((aligned(4)));

template <typename ET> struct Out;
template <> struct Out<uint16_t> {
  __device__ __forceinline__ static float widen(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
  // Round to nearest even, the conversion's own rounding.
  __device__ __forceinline__ static uint16_t narrow(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }
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
  __device__ __forceinline__ static float widen(float x) { return x; }
  __device__ __forceinline__ static float narrow(float x) { return x; }
  __device__ __forceinline__ static float one(const u32x4& v, int k) { return __uint_as_float(v[k]); }
  __device__ __forceinline__ static void cut(u32x4& v, uint32_t allow) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (!((allow >> k) & 1)) v[k] = 0xFF800000u;
  }
};

// LDS: the chunk's tables.
struct Tables {
  alignas(16) uint32_t count[CH];
  alignas(16) u32x4 stage[WG];  // a wave's window, while listed ids change
  uint32_t touched[CH / 32];
  int before[CH / 32 + 1];      // listed ids before each word of `touched`
  uint16_t list[CH];
  uint32_t biased[CH / 32];
  int rank[CH / 32 + 1];        // biased ids before each word of `biased`
  union {                       // of each biased id, in order: 1 + its last entry, then
    int entry[BIASES];
    float bias[BIASES];         // that entry's value
  };
  int local[64];                // drafted tokens' places in the chunk
  uint64_t path[64];            // tree: nodes on the path root .. v
  uint64_t here[CH / 256];      // drafted tokens inside each window of a wave's 64 vectors
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

// Vectors of U positions, NV per thread each.
template <int NV, int U>
struct Group {
  u32x4 v[U][NV];
  uint32_t allow[U][NV];
};

template <typename ET>
__global__ __launch_bounds__(WG) __attribute__((amdgpu_waves_per_eu(4))) void adjust_logits_kernel(AdjustArgs a) {
  constexpr int VEC = Tr<ET>::VEC;
  constexpr int NV = CH / (WG * VEC);  // vectors per thread and position
  constexpr int U = 8 / NV;            // positions at once
  __shared__ Tables sh;
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  const int pg = blockIdx.x % a.PG;
  const int chunk = (blockIdx.x / a.PG) % a.C;
  const int b = blockIdx.x / a.PG / a.C;
  const int lo = chunk * a.chunk, len = min(a.chunk, a.V - lo);

  constexpr uint32_t ALL = (1u << VEC) - 1;
  const int p0 = (int)((int64_t)a.P * pg / a.PG), p1 = (int)((int64_t)a.P * (pg + 1) / a.PG);

  // The vectors of positions i0 .. i0 + U - 1 that are needed, and what their
  // masks allow.
  auto fetch = [&](Group<NV, U>& r, int i0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u;
      const uint32_t* mask = nullptr;
      if (a.c.mask && i < p1) {
        const int64_t row = a.c.mask_rows ? (int64_t)a.c.mask_rows[(int64_t)b * a.P + i] : (int64_t)b * a.P + i;
        if (row >= 0 && row < a.c.num_masks) mask = a.c.mask + row * a.words + lo / 32;
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int e = (j * WG + t) * VEC;
        r.allow[u][j] = mask && e < len ? (mask[e >> 5] >> (e & 31)) & ALL : ALL;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const ET* src = static_cast<const ET*>(a.in) + b * a.in_row + (i0 + u) * a.in_pos + lo;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int e = (j * WG + t) * VEC;
        bool need = i0 + u < p1 && e < len && r.allow[u][j];
        if (a.inplace && r.allow[u][j] == ALL) need = need && ((sh.touched[e >> 5] >> (e & 31)) & ALL);
        if (!need) continue;
        if (e + VEC <= len) r.v[u][j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_u*>(src + e));
        else {
          r.v[u][j] = u32x4{0, 0, 0, 0};
#pragma unroll
          for (int k = 0; k < VEC; ++k)
            if (e + k < len) Tr<ET>::set(r.v[u][j], k, src + e + k);
        }
      }
    }
  };
  // The first of them are on their way while the tables are made (in place,
  // what is needed depends on the tables).
  Group<NV, U> now;
  if (!a.inplace) fetch(now, p0);

  for (int i = t; i < CH / 4; i += WG) reinterpret_cast<u32x4*>(sh.count)[i] = u32x4{0, 0, 0, 0};
  if (t < CH / 32) sh.touched[t] = sh.biased[t] = 0;
  const int drafted = a.penalties && a.tokens ? (a.parents ? a.P : a.P - 1) : 0;
  if (t < 64) {
    int at = -1;
    if (t < drafted && (!a.parents || t > 0)) {
      const uint32_t d = (uint32_t)a.tokens[b * a.tokens_stride + t] - (uint32_t)lo;
      at = d < (uint32_t)len ? (int)d : -1;
    }
    sh.local[t] = at;
#pragma unroll
    for (int k = 0; k < CH / (64 * VEC); ++k) {
      const uint64_t m = __ballot(at >= 0 && at / (64 * VEC) == k);
      if (t == 0) sh.here[k] = m;
    }
    if (a.parents) sh.path[t] = path_mask(a.parents + (int64_t)b * a.P, a.P);
  }
  __syncthreads();
  if (t < 64 && sh.local[t] >= 0) atomicOr(&sh.touched[sh.local[t] >> 5], 1u << (sh.local[t] & 31));
  if (a.penalties && a.c.history) {
    const int32_t* h = a.c.history + b * a.c.history_stride;
    const int n = (int)min((int64_t)max(a.c.history_lens[b], 0), a.c.history_width);
    const int np = a.c.prompt_lens ? max(a.c.prompt_lens[b], 0) : 0;
    auto take = [&](int tok, int j) {
      const uint32_t d = (uint32_t)tok - (uint32_t)lo;
      if (d < (uint32_t)len) {
        if (j < np) atomicOr(&sh.count[d], IN_PROMPT);
        else atomicAdd(&sh.count[d], 1u);
        atomicOr(&sh.touched[d >> 5], 1u << (d & 31));
      }
    };
    const int n4 = n / 4;
    for (int j = t; j < n4; j += 4 * WG) {
      i32x4 x[4];
#pragma unroll
      for (int s = 0; s < 4; ++s)
        x[s] = j + s * WG < n4 ? *reinterpret_cast<const i32x4_u*>(h + 4 * (int64_t)(j + s * WG)) : i32x4{-1, -1, -1, -1};
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int k = 0; k < 4; ++k) take(x[s][k], 4 * (j + s * WG) + k);
    }
    if (4 * n4 + t < n) take(h[4 * n4 + t], 4 * n4 + t);
  }
  const int32_t* bias_ids = a.c.bias_ids + b * a.c.bias_stride;
  const float* bias_values = a.c.bias_values + b * a.c.bias_stride;
  const int nbias = !a.c.bias_ids ? 0
                    : (int)(a.c.bias_lens ? min((int64_t)max(a.c.bias_lens[b], 0), a.c.bias_stride) : a.c.bias_stride);
  for (int e = t; e < nbias; e += WG) {
    const uint32_t d = (uint32_t)bias_ids[e] - (uint32_t)lo;
    if (d < (uint32_t)len) {
      atomicOr(&sh.count[d], BIASED);
      atomicOr(&sh.touched[d >> 5], 1u << (d & 31));
      atomicOr(&sh.biased[d >> 5], 1u << (d & 31));
    }
  }
  if (nbias > 0)
    for (int k = t; k < BIASES; k += WG) sh.entry[k] = 0;
  __syncthreads();

  // The places of touched ids in their list, and of biased ones in theirs, by
  // a wave each.
  if (t < 128) {
    const uint32_t* bits = t < 64 ? sh.touched : sh.biased;
    int* before = t < 64 ? sh.before : sh.rank;
    const uint32_t w0 = bits[2 * lane], w1 = bits[2 * lane + 1];
    const int n0 = __popc(w0), n = n0 + __popc(w1);
    int inc = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(inc, o, 64);
      if (lane >= o) inc += u;
    }
    before[2 * lane] = inc - n;
    before[2 * lane + 1] = inc - n + n0;
    if (lane == 63) before[128] = inc;
  }
  __syncthreads();
  auto bias_place = [&](int d) { return sh.rank[d >> 5] + __popc(sh.biased[d >> 5] & ((1u << (d & 31)) - 1)); };
  if (nbias > 0) {
    // A token's last entry counts, whatever order they come in here.
    for (int e = t; e < nbias; e += WG) {
      const uint32_t d = (uint32_t)bias_ids[e] - (uint32_t)lo;
      if (d < (uint32_t)len) atomicMax(&sh.entry[bias_place(d)], e + 1);
    }
    __syncthreads();
    for (int k = t; k < sh.rank[CH / 32]; k += WG) sh.bias[k] = bias_values[sh.entry[k] - 1];
  }
  if (t < CH / 32) {
    int k = sh.before[t];
    for (uint32_t m = sh.touched[t]; m; m &= m - 1) sh.list[k++] = (uint16_t)(t * 32 + __ffs(m) - 1);
  }
  __syncthreads();

  const float r = a.c.repetition ? a.c.repetition[b] : 1.f;
  const float freq = a.c.frequency ? a.c.frequency[b] : 0.f;
  const float pres = a.c.presence ? a.c.presence[b] : 0.f;
  // For each of the thread's vectors: its listed ids, and its wave's window:
  // the part of the list and the drafted tokens in it.
  uint32_t touch[NV];
  int k0[NV], k1[NV];
  uint64_t here[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = (j * WG + t) * VEC, win = __builtin_amdgcn_readfirstlane((j * WG + w * 64) * VEC);
    touch[j] = (sh.touched[e >> 5] >> (e & 31)) & ALL;
    k0[j] = __builtin_amdgcn_readfirstlane(sh.before[win / 32]);
    k1[j] = __builtin_amdgcn_readfirstlane(sh.before[win / 32 + 2 * VEC]);
    here[j] = sh.here[win / (64 * VEC)];
  }
  // Changes listed id d's logit, where something applies to it (a NaN's bits
  // would not pass through the conversions); path: the position's drafted
  // tokens near it.
  const uint32_t applies = BIASED | (a.c.repetition ? IN_PROMPT : 0);
  auto adjust = [&](ET& logit, int d, uint64_t path) {
    const uint32_t c = sh.count[d];
    uint32_t n = c & ~(IN_PROMPT | BIASED);
    for (uint64_t m = path; m; m &= m - 1) n += sh.local[__builtin_ctzll(m)] == d;
    if (!(n | (c & applies))) return;
    float x = Out<ET>::widen(logit);
    if (n | (c & IN_PROMPT)) x = x > 0.f ? x / r : x * r;
    if (n) x = (x - freq * (float)n) - pres;
    if (c & BIASED) x = x + sh.bias[bias_place(d)];
    logit = Out<ET>::narrow(x);
  };

  if (a.inplace) fetch(now, p0);
  for (int i0 = p0; i0 < p1; i0 += U) {
    Group<NV, U> next;
    if (i0 + U < p1) fetch(next, i0 + U);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u;
      if (i >= p1) break;
      ET* dst = static_cast<ET*>(a.out) + b * a.out_row + i * a.out_pos + lo;
      const uint64_t path = a.parents ? sh.path[i & 63] : i >= 64 ? ~0ull : (1ull << i) - 1;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int e = (j * WG + t) * VEC;
        const int win = (j * WG + w * 64) * VEC;
        if (k1[j] > k0[j]) {
          const uint64_t on = path & here[j];
          ET* stage = reinterpret_cast<ET*>(sh.stage + w * 64);
          if (touch[j]) sh.stage[t] = now.v[u][j];
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
          __builtin_amdgcn_wave_barrier();
          for (int k = k0[j] + lane; k < k1[j]; k += 64) {
            const int d = sh.list[k];
            adjust(stage[d - win], d, on);
          }
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
          __builtin_amdgcn_wave_barrier();
          if (touch[j]) now.v[u][j] = sh.stage[t];
        }
        if (e >= len || (a.inplace && !touch[j] && now.allow[u][j] == ALL)) continue;
        if (!now.allow[u][j]) {
          const uint32_t f = Tr<ET>::NEG_INF_WORD;
          now.v[u][j] = u32x4{f, f, f, f};
        } else if (now.allow[u][j] != ALL) {
          Out<ET>::cut(now.v[u][j], now.allow[u][j]);
        }
        if (e + VEC <= len) __builtin_nontemporal_store(now.v[u][j], reinterpret_cast<u32x4_u*>(dst + e));
        else {
#pragma unroll
          for (int k = 0; k < VEC; ++k)
            if (e + k < len) dst[e + k] = Out<ET>::one(now.v[u][j], k);
        }
      }
    }
    now = next;
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
    if (a.c.history && (!a.c.history_lens || a.c.history_stride < 0 || a.c.history_stride > INT32_MAX ||
                        a.c.history_width < 0 || a.c.history_width > a.c.history_stride))
      return SV_ERR_ARG;
    if (a.c.history_width == 0) a.c.history_width = a.c.history_stride;
    if (a.c.history && a.c.history_width > MAX_ENTRIES) return SV_ERR_UNSUPPORTED;
    if (P > 1 && (!tokens || tokens_stride < (parents ? P : P - 1) || tokens_stride > INT32_MAX)) return SV_ERR_ARG;
  }
  if (a.c.bias_ids && (!a.c.bias_values || a.c.bias_stride < 0 || a.c.bias_stride > INT32_MAX - 1)) return SV_ERR_ARG;
  if (a.c.bias_ids && a.c.bias_stride > MAX_ENTRIES) return SV_ERR_UNSUPPORTED;
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
  a.chunk = a.c.bias_ids && a.c.bias_stride > BIASES ? BIASES : CH;
  a.C = (V - 1) / a.chunk + 1;
  a.words = (V - 1) / 32 + 1;
  const int64_t groups = (int64_t)B * a.C;
  a.PG = (int)(groups >= GRID_WANTED ? 1 : (GRID_WANTED + groups - 1) / groups);
  if (a.PG > P) a.PG = P;
  if (groups * a.PG > MAX_GROUPS) return SV_ERR_UNSUPPORTED;
  if (a.c.bias_stride <= 0) a.c.bias_ids = nullptr;
  void (*const k)(AdjustArgs) = dtype == SV_BF16 ? adjust_logits_kernel<uint16_t> : adjust_logits_kernel<float>;
  (void)hipGetLastError();
  hipLaunchKernelGGL(k, dim3((uint32_t)(groups * a.PG)), dim3(WG), 0, stream, a);
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
}
