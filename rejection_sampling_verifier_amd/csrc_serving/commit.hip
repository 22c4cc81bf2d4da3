// The accepted path's keys and values enter the paged 8-bit cache
// (spec_verify_commit), for gfx950.
//
// Mathematics: per completed block and head one maximum over page * D bf16
// values, then code = round_half_even(x / scale).  A power-of-two scale makes
// the e4m3 quotient exact; an int8 quotient is rounded from its float32
// value and put right by the sign of x - (r +- 1/2) scale, which one fma
// gives exactly.  Bytes bound it: few rows complete a block in a step, the
// others copy n rows of D values; small batches are bound by latency.
//
// Three kinds of work-groups: one per (row, K or V) copies the committed
// tokens of all heads, which lie side by side, to the tail; one per (row, kv
// head, K or V) quantises a head's completed blocks, and leaves at once where
// there are none (the counters are on the device); the rest add the weights
// of the committed tokens to the blocks' totals.  A block is read once: its
// values wait in registers for their maximum (256 rows of up to 9 tokens:
// 16.7 us with one kind that did a head's copy and blocks both, 14.5 us so; two
// or four heads to a work-group: 17 and 26 us).

#include <climits>

#include "cache.h"

using namespace sv;
using namespace svr;

namespace {

struct CommitArgs {
  const uint16_t* kn;
  const uint16_t* vn;
  int64_t kv_row, kv_tok;
  sv_cache c;
  const int32_t* num;
  const int32_t* nodes;
  int64_t nodes_stride;
  const int32_t* positions;
  const int32_t* blocks;
  int32_t* positions_out;
  int32_t* blocks_out;
  const float* weights;
  const float* totals;
  float* totals_out;
  int T, quant_groups, total_groups;  // work-groups per row, beside the two that copy
  int inplace;                       // the counters are updated by a kernel of their own
};

// What row b commits.  n = 0: the row is left as it was.
struct Commit {
  int n, filled, blocks, tail, start, pos;
};

__device__ __forceinline__ Commit row_counters(const CommitArgs& a, int b) {
  Commit r;
  r.pos = a.positions[b];
  r.blocks = a.blocks[b];
  r.n = a.num[b];
  r.n = r.n < 0 || r.n >= a.T || r.pos < 0 || r.pos > INT_MAX - r.n - 1 || r.blocks < 0 || r.blocks > a.c.max_blocks
            ? 0 : r.n + 1;
  r.tail = r.n ? r.pos % a.c.page : 0;
  r.start = r.n ? (r.pos - r.tail) % a.c.tail : 0;
  r.filled = (r.tail + r.n) / a.c.page;
  return r;
}

// By the whole work-group (of more than SV_MAX_K threads): path[] gets the
// committed tokens; a bad one, or a missing page, undoes the row's commit.
__device__ __forceinline__ void row_path(const CommitArgs& a, int b, Commit& r, int* path, int* bad) {
  const int t = threadIdx.x;
  if (t == 0) *bad = 0;
  __syncthreads();
  if (t < r.n) {
    const int node = t == 0 || !a.nodes ? t : a.nodes[b * a.nodes_stride + t - 1];
    if ((uint32_t)node >= (uint32_t)a.T) *bad = 1;
    path[t] = min(max(node, 0), a.T - 1);
  }
  if (t < r.filled) {
    const int j = r.blocks + t;
    if (j >= a.c.max_blocks || (uint32_t)a.c.block_table[(int64_t)b * a.c.max_blocks + j] >= (uint32_t)a.c.num_pages)
      *bad = 1;
  }
  __syncthreads();
  if (*bad) r.n = r.filled = 0;
}

__device__ __forceinline__ float bf16_at(const u32x4& v, int k) { return Tr<uint16_t>::at(v, k); }

// The scale of a block whose largest magnitude has these bf16 bits.
template <int KIND>
__device__ __forceinline__ float scale_of(uint32_t top) {
  if (top >= 0x7F80u) return __uint_as_float(0x7FC00000u);
  if (top == 0) return 1.f;
  const float a = __uint_as_float(top << 16);
  if (KIND == SV_INT8) return fmaxf(a / 127.f, 0x1p-126f);
  // a = 1.m 2^e and 448 = 1.75 2^8
  const int e = (int)(top >> 7) - 127 - ((top & 0x7Fu) <= 0x60u ? 8 : 7);
  return ldexpf(1.f, max(e, -126));
}

template <int KIND>
__device__ __forceinline__ uint32_t code8(float x, float scale, float inv) {
  if (KIND == SV_E4M3) return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x * inv, 0.f, 0, false) & 0xFFu;
  float r = rintf(x / scale);
  const float d = fmaf(-r, scale, x), h = 0.5f * scale;  // both exact
  const bool odd = ((int)r & 1) != 0;
  if (d > h || (d == h && odd)) r += 1.f;
  else if (d < -h || (d == -h && odd)) r -= 1.f;
  return (uint32_t)(int)r & 0xFFu;
}

constexpr int TPAD = 16;  // bytes between the channels of the transposing buffer

template <int KIND, int D, int PAGE>
__global__ __launch_bounds__(WG) void cache_commit_kernel(CommitArgs a) {
  constexpr int PER = D / 8;                                   // 16-byte pieces of a head's token
  constexpr int NV = PAGE * PER < WG ? 1 : PAGE * PER / WG;    // those of a block, per thread
  __shared__ int path[SV_MAX_K + 1];
  __shared__ int bad;
  __shared__ uint32_t tops[NWAVE];
  __shared__ alignas(16) uint8_t codes[D * (PAGE + TPAD)];     // V: its channels' tokens side by side
  const int t = threadIdx.x;
  const int per = 2 + a.total_groups + a.quant_groups;
  const int b = blockIdx.x / per, part = blockIdx.x % per;
  Commit r = row_counters(a, b);
  const bool quant = part >= 2 + a.total_groups;
  if (quant && r.filled == 0) return;
  row_path(a, b, r, path, &bad);

  if (part == 0 && t == 0 && !a.inplace) {
    a.positions_out[b] = r.pos + r.n;
    a.blocks_out[b] = r.blocks + r.filled;
  }
  if (part >= 2 && !quant) {
    const int j = (part - 2) * WG + t;
    if (j < a.c.max_blocks) {
      float x = 0.f;
      if (j < r.blocks) {
        if (a.weights) {
          const float* w = a.weights + (int64_t)b * a.T * a.c.max_blocks + j;
          for (int i = 0; i < r.n; i += 8) {  // eight loads at once
            float y[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = i + k < r.n ? w[(int64_t)path[i + k] * a.c.max_blocks] : 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) x += y[k];
          }
        }
        x = a.totals[(int64_t)b * a.c.max_blocks + j] + x;
      }
      a.totals_out[(int64_t)b * a.c.max_blocks + j] = x;
    }
    return;
  }
  if (r.n == 0) return;
  const bool val = part & 1;
  const int64_t slot = (int64_t)a.c.Hkv * D;
  uint16_t* ring = (val ? a.c.v_tail : a.c.k_tail) + (int64_t)b * a.c.tail * slot;
  const uint16_t* fresh = (val ? a.vn : a.kn) + b * a.kv_row;
  auto place = [&](int j) {  // ring slot of the row's j-th token since its last full block
    const int s = r.start + j;
    return s < a.c.tail ? s : s - a.c.tail;
  };

  if (!quant) {
    const int j0 = max(r.tail, r.filled * PAGE), all = a.c.Hkv * PER;
    const int pieces = (r.tail + r.n - j0) * all;
    for (int e0 = t; e0 < pieces; e0 += 4 * WG) {
      u32x4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int e = min(e0 + k * WG, pieces - 1);
        v[k] = *reinterpret_cast<const u32x4*>(fresh + path[j0 + e / all - r.tail] * a.kv_tok + e % all * 8);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int e = e0 + k * WG;
        if (e < pieces) *reinterpret_cast<u32x4*>(ring + place(j0 + e / all) * slot + e % all * 8) = v[k];
      }
    }
    return;
  }

  const int h = (part - 2 - a.total_groups) >> 1;
  for (int m = 0; m < r.filled; ++m) {
    const int pid = a.c.block_table[(int64_t)b * a.c.max_blocks + r.blocks + m];
    const int64_t at = (int64_t)pid * a.c.Hkv + h;
    u32x4 v[NV];
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int e = k * WG + t, j = m * PAGE + e / PER, d = h * D + e % PER * 8;
      v[k] = u32x4{0, 0, 0, 0};
      if (e < PAGE * PER)
        v[k] = *reinterpret_cast<const u32x4*>(j < r.tail ? ring + place(j) * slot + d
                                                          : fresh + path[j - r.tail] * a.kv_tok + d);
    }
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = max(top, max(v[k][i] & 0x7FFFu, (v[k][i] >> 16) & 0x7FFFu));
#pragma unroll
    for (int o = 32; o; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o, 64));
    if ((t & 63) == 0) tops[t >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NWAVE; ++k) top = max(top, tops[k]);
    const float scale = scale_of<KIND>(top);
    const bool finite = top < 0x7F80u;
    const float inv = KIND == SV_E4M3 && finite ? 1.f / scale : 0.f;  // a power of two: exact
    if (t == 0) (val ? a.c.v_scale : a.c.k_scale)[at] = scale;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int e = k * WG + t, j = e / PER, d = e % PER * 8;
      if (e >= PAGE * PER) continue;
      uint32_t w[2] = {0, 0};
      if (finite) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i >> 2] |= code8<KIND>(bf16_at(v[k], i), scale, inv) << (8 * (i & 3));
      }
      if (!val) {
        *reinterpret_cast<uint2*>(a.c.k_pages + (at * PAGE + j) * D + d) = make_uint2(w[0], w[1]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) codes[(d + i) * (PAGE + TPAD) + j] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
      }
    }
    __syncthreads();
    if (val) {
      for (int e = t; e < D * PAGE / 16; e += WG) {
        const int d = e / (PAGE / 16), j = e % (PAGE / 16) * 16;
        *reinterpret_cast<u32x4*>(a.c.v_pages + (at * D + d) * PAGE + j) =
            *reinterpret_cast<const u32x4*>(codes + d * (PAGE + TPAD) + j);
      }
      __syncthreads();
    }
  }
}

// Counters updated in place: after every work-group has read them.
__global__ __launch_bounds__(128) void commit_counters_kernel(CommitArgs a) {
  __shared__ int path[SV_MAX_K + 1];
  __shared__ int bad;
  const int b = blockIdx.x;
  Commit r = row_counters(a, b);
  row_path(a, b, r, path, &bad);
  if (threadIdx.x == 0) {
    a.positions_out[b] = r.pos + r.n;
    a.blocks_out[b] = r.blocks + r.filled;
  }
}

template <int KIND, int D>
auto kernel_of_page(int page) -> void (*)(CommitArgs) {
  return page == 16 ? cache_commit_kernel<KIND, D, 16> : page == 32 ? cache_commit_kernel<KIND, D, 32>
         : page == 64 ? cache_commit_kernel<KIND, D, 64> : page == 128 ? cache_commit_kernel<KIND, D, 128>
                                                                       : cache_commit_kernel<KIND, D, 256>;
}
auto kernel_of(const sv_cache& c) -> void (*)(CommitArgs) {
  return c.kind == SV_E4M3 ? (c.D == 64 ? kernel_of_page<SV_E4M3, 64>(c.page) : kernel_of_page<SV_E4M3, 128>(c.page))
                           : (c.D == 64 ? kernel_of_page<SV_INT8, 64>(c.page) : kernel_of_page<SV_INT8, 128>(c.page));
}

}  // namespace

extern "C" int spec_verify_commit(const void* k_new, const void* v_new, int64_t kv_row, int64_t kv_tok, int T,
                                  const int32_t* num_accepted, const int32_t* nodes, int64_t nodes_stride,
                                  const sv_cache* cache, const int32_t* positions, const int32_t* blocks,
                                  int32_t* positions_out, int32_t* blocks_out, const float* weights,
                                  const float* totals, float* totals_out, hipStream_t stream) {
  const int bad = check_cache(cache);
  if (bad != SV_OK) return bad;
  const sv_cache& c = *cache;
  if (!k_new || !v_new || !num_accepted || !positions || !blocks || !positions_out || !blocks_out || T < 1)
    return SV_ERR_ARG;
  if (T > SV_MAX_K + 1) return SV_ERR_UNSUPPORTED;
  if (c.tail < c.page - 1 + T) return SV_ERR_ARG;
  const size_t nb = (size_t)c.B * 4, nt = nb * c.max_blocks;
  if ((positions == positions_out) != (blocks == blocks_out)) return SV_ERR_ARG;
  if ((totals == nullptr) != (totals_out == nullptr) || (weights && !totals)) return SV_ERR_ARG;
  if (nodes && (nodes_stride < T - 1 || nodes_stride > INT_MAX)) return SV_ERR_ARG;
  // What some work-groups still read when others write.
  const Output out[] = {{{positions_out, nb}, positions}, {{blocks_out, nb}, blocks}, {{totals_out, nt}, totals}};
  const Array in[] = {{positions, nb}, {blocks, nb}, {num_accepted, nb}, {totals, nt}, {c.block_table, nt},
                      {weights, nt * T}, {nodes, 4 * ((size_t)nodes_stride * (c.B - 1) + T - 1)}};
  if (outputs_overlap(out, in)) return SV_ERR_ARG;
  const void* aligned[] = {k_new, v_new};
  for (const void* p : aligned)
    if (reinterpret_cast<uintptr_t>(p) % 16) return SV_ERR_ARG;
  constexpr int64_t FAR = int64_t(1) << 40;
  const int64_t strides[] = {kv_row, kv_tok};
  for (int64_t s : strides)
    if (s < 0 || s > FAR || s % 8) return SV_ERR_ARG;
  CommitArgs a;
  a.kn = static_cast<const uint16_t*>(k_new);
  a.vn = static_cast<const uint16_t*>(v_new);
  a.kv_row = kv_row;
  a.kv_tok = kv_tok;
  a.c = c;
  a.num = num_accepted;
  a.nodes = nodes;
  a.nodes_stride = nodes_stride;
  a.positions = positions;
  a.blocks = blocks;
  a.positions_out = positions_out;
  a.blocks_out = blocks_out;
  a.weights = weights;
  a.totals = totals;
  a.totals_out = totals_out;
  a.T = T;
  a.quant_groups = 2 * c.Hkv;
  a.total_groups = totals ? (c.max_blocks + WG - 1) / WG : 0;
  a.inplace = positions == positions_out;
  const int64_t grid = (int64_t)c.B * (2 + a.quant_groups + a.total_groups);
  if (grid > MAX_ITEMS / WG) return SV_ERR_UNSUPPORTED;
  (void)hipGetLastError();
  hipLaunchKernelGGL(kernel_of(c), dim3((uint32_t)grid), dim3(WG), 0, stream, a);
  if (hipGetLastError() != hipSuccess) return SV_ERR_HIP;
  if (a.inplace) {
    hipLaunchKernelGGL(commit_counters_kernel, dim3(c.B), dim3(128), 0, stream, a);
    if (hipGetLastError() != hipSuccess) return SV_ERR_HIP;
  }
  return SV_OK;
}
