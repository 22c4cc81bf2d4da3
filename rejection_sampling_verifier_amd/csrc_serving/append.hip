// A prompt's keys and values enter the paged 8-bit cache, the keys rotated by
// their positions on the way (spec_verify_append), for gfx950.
//
// Mathematics: rotation (rotary.h), then per completed block and head what a
// commit does (quantise.h).  Bytes bound it: two are read and one is written
// for each element.  A work-group takes one block of a row with some of its
// heads, a head at a time: its values wait in registers, rotated, for their
// largest magnitude, while the values of the head's other half are on their
// way.  A thread has the same pairs of the same tokens in every head, so it
// forms their cosines and sines once and keeps them: 124 registers, four
// work-groups to a CU, at pages of 64 tokens and D = 128 (16 prompts of up to
// 4096 tokens 109 us; in LDS, 32 KB of it, they leave room for three: 142), 210
// and two at pages of 128 (175 us), 427 and one at 256 (248 us).  V's codes are turned in LDS in words of four tokens, which one lane
// has read.  The tokens after the last full block go to the tail by the
// work-group of the row's first block, which is also the one that reads the
// tail's old tokens, so that a ring of a single block will do.

#include <climits>

#include "quantise.h"
#include "rotary.h"

using namespace sv;
using namespace svr;

namespace {

struct AppendArgs {
  const uint16_t* k;
  const uint16_t* v;
  int64_t kv_row, kv_tok;
  uint16_t* k_out;
  int64_t ko_row, ko_tok;
  sv_rotary rot;  // dims 0: keys are taken as they are
  sv_cache c;
  const int32_t* lens;
  const int32_t* positions;
  const int32_t* blocks;
  int32_t* positions_out;
  int32_t* blocks_out;
  int T, units, groups, heads;  // work-groups per row: units times groups of heads
  int inplace;                  // the counters are updated by a kernel of their own
};

// What row b appends.  n = 0: the row is left as it was.
struct Append {
  int n, filled, blocks, tail, start, pos;
};

// By the whole work-group: a missing page undoes the row's append.
__device__ __forceinline__ Append row_append(const AppendArgs& a, int b, int* bad) {
  Append r;
  r.pos = a.positions[b];
  r.blocks = a.blocks[b];
  r.n = a.lens ? a.lens[b] : a.T;
  if (r.n < 0 || r.n > a.T || r.pos < 0 || r.pos > INT_MAX - r.n || r.blocks < 0 || r.blocks > a.c.max_blocks) r.n = 0;
  r.tail = r.n ? r.pos & (a.c.page - 1) : 0;
  r.start = r.n ? (r.pos - r.tail) % a.c.tail : 0;
  r.filled = r.n ? (r.tail + r.n) / a.c.page : 0;
  if (threadIdx.x == 0) *bad = r.filled > a.c.max_blocks - r.blocks;
  __syncthreads();
  if (!*bad)
    for (int j = threadIdx.x; j < r.filled; j += blockDim.x)
      if ((uint32_t)a.c.block_table[(int64_t)b * a.c.max_blocks + r.blocks + j] >= (uint32_t)a.c.num_pages) *bad = 2;
  __syncthreads();
  if (*bad) r.n = r.filled = 0;
  return r;
}

template <int KIND, int D, int PAGE>
__global__ __launch_bounds__(WG) void cache_append_kernel(AppendArgs a) {
  constexpr int PER = D / 16;                                  // pairs of 16-byte pieces of a head's token
  constexpr int NV = PAGE * PER < WG ? 1 : PAGE * PER / WG;    // those of a block's keys, per thread
  constexpr int QP = D / 8;                                    // pieces of a token
  constexpr int NQ = PAGE / 4 * QP < WG ? 1 : PAGE / 4 * QP / WG;  // pieces of four tokens' values, per thread
  constexpr int ROW = PAGE + 4;                                // bytes of a channel in LDS: rows in different banks
  __shared__ int bad;
  __shared__ uint32_t tops[2][NWAVE];
  __shared__ alignas(16) uint32_t codes[D * ROW / 4];          // V: its channels' tokens side by side
  const int t = threadIdx.x;
  const int b = blockIdx.x / (a.units * a.groups), unit = blockIdx.x / a.groups % a.units, group = blockIdx.x % a.groups;
  const Append r = row_append(a, b, &bad);
  if (unit == 0 && group == 0 && t == 0 && !a.inplace) {
    a.positions_out[b] = r.pos + r.n;
    a.blocks_out[b] = r.blocks + r.filled;
  }
  if (r.n == 0 || unit >= max(r.filled, 1)) return;
  const int h0 = group * a.heads, h1 = min(h0 + a.heads, a.c.Hkv);
  const int64_t slot = (int64_t)a.c.Hkv * D;
  auto place = [&](int j) {  // ring slot of the row's j-th token since its last full block before the call
    const int s = r.start + j % a.c.tail;
    return s < a.c.tail ? s : s - a.c.tail;
  };
  auto token = [&](bool val, int j) -> const uint16_t* {
    return j < r.tail ? (val ? a.c.v_tail : a.c.k_tail) + ((int64_t)b * a.c.tail + place(j)) * slot
                      : (val ? a.v : a.k) + b * a.kv_row + (j - r.tail) * a.kv_tok;
  };
  // The thread's pairs of the window of PAGE tokens that begins with the row's
  // j0-th: their cos and sin, as far as they are new.
  float2 cs[NV][8];
  auto turns = [&](int j0) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int e = k * WG + t, at = j0 + e / PER - r.tail, c = e % PER;  // its number among the new ones
      if (e < PAGE * PER && at >= 0 && at < r.n && c < a.rot.dims / 16)
#pragma unroll
        for (int i = 0; i < 8; ++i) cs[k][i] = turn_of(a.rot, a.c.B, a.T, b, at, c * 8 + i, (int64_t)r.pos + at);
    }
  };
  // Keys rotated, and put out, where they are new.
  auto turn = [&](int k, int h, int j, u32x4& u, u32x4& w) {
    const int c = (k * WG + t) % PER;
    if (c < a.rot.dims / 16) rotate_pieces(u, w, a.rot.interleaved, cs[k]);
    if (a.k_out) {
      const Pieces p = pieces_of(c, a.rot.dims, a.rot.interleaved);
      uint16_t* to = a.k_out + b * a.ko_row + (j - r.tail) * a.ko_tok + h * D;
      *reinterpret_cast<u32x4*>(to + p.p0 * 8) = u;
      *reinterpret_cast<u32x4*>(to + p.p1 * 8) = w;
    }
  };
  auto top_of = [&](const u32x4& v, uint32_t top) {
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, max(v[i] & 0x7FFFu, (v[i] >> 16) & 0x7FFFu));
    return top;
  };
  auto all_tops = [&](uint32_t top, uint32_t* place) {
#pragma unroll
    for (int o = 32; o; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o, 64));
    if ((t & 63) == 0) place[t >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NWAVE; ++k) top = max(top, place[k]);
    return top;
  };

  if (unit < r.filled) {
    const int j0 = unit * PAGE;
    const int pid = a.c.block_table[(int64_t)b * a.c.max_blocks + r.blocks + unit];
    u32x4 kv[NV][2], vv[NQ][4];
    // Where the thread's pieces of head 0 are: what is divided and looked up is so once.
    const uint16_t* kp[NV];
    const uint16_t* vp[NQ][4];
#pragma unroll
    for (int k = 0; k < NV; ++k) kp[k] = token(false, j0 + min((k * WG + t) / PER, PAGE - 1));
#pragma unroll
    for (int k = 0; k < NQ; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        vp[k][i] = token(true, j0 + min((k * WG + t) / QP * 4, PAGE - 4) + i) + (k * WG + t) % QP * 8;
    auto load_k = [&](int h) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        kv[k][0] = kv[k][1] = u32x4{0, 0, 0, 0};
        if (k * WG + t >= PAGE * PER) continue;
        const Pieces p = pieces_of((k * WG + t) % PER, a.rot.dims, a.rot.interleaved);
        kv[k][0] = *reinterpret_cast<const u32x4*>(kp[k] + h * D + p.p0 * 8);
        kv[k][1] = *reinterpret_cast<const u32x4*>(kp[k] + h * D + p.p1 * 8);
      }
    };
    auto load_v = [&](int h) {
#pragma unroll
      for (int k = 0; k < NQ; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          vv[k][i] = u32x4{0, 0, 0, 0};
          if (k * WG + t < PAGE / 4 * QP) vv[k][i] = *reinterpret_cast<const u32x4*>(vp[k][i] + h * D);
        }
    };
    load_k(h0);
    turns(j0);
    for (int h = h0; h < h1; ++h) {
      const int64_t at = (int64_t)pid * a.c.Hkv + h;
      load_v(h);
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int e = k * WG + t, j = j0 + e / PER;
        if (e < PAGE * PER && j >= r.tail) turn(k, h, j, kv[k][0], kv[k][1]);
        top = top_of(kv[k][1], top_of(kv[k][0], top));
      }
      top = all_tops(top, tops[0]);
      {
        const float scale = scale_of<KIND>(top);
        const bool finite = top < 0x7F80u;
        const float inv = KIND == SV_E4M3 && finite ? 1.f / scale : 0.f;  // a power of two: exact
        if (t == 0) a.c.k_scale[at] = scale;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          const int e = k * WG + t, j = e / PER;
          if (e >= PAGE * PER) continue;
          const Pieces p = pieces_of(e % PER, a.rot.dims, a.rot.interleaved);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t w[2] = {0, 0};
            if (finite) {
#pragma unroll
              for (int i = 0; i < 2; ++i)
                w[i] = code32<KIND>(bf16_at(kv[k][half], 4 * i), bf16_at(kv[k][half], 4 * i + 1),
                                    bf16_at(kv[k][half], 4 * i + 2), bf16_at(kv[k][half], 4 * i + 3), scale, inv);
            }
            *reinterpret_cast<uint2*>(a.c.k_pages + (at * PAGE + j) * D + (half ? p.p1 : p.p0) * 8) = make_uint2(w[0], w[1]);
          }
        }
      }
      if (h + 1 < h1) load_k(h + 1);
      top = 0;
#pragma unroll
      for (int k = 0; k < NQ; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = top_of(vv[k][i], top);
      top = all_tops(top, tops[1]);
      {
        const float scale = scale_of<KIND>(top);
        const bool finite = top < 0x7F80u;
        const float inv = KIND == SV_E4M3 && finite ? 1.f / scale : 0.f;
        if (t == 0) a.c.v_scale[at] = scale;
#pragma unroll
        for (int k = 0; k < NQ; ++k) {
          const int f = k * WG + t;
          if (f >= PAGE / 4 * QP) continue;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            codes[((f % QP * 8 + i) * ROW) / 4 + f / QP] =
                finite ? code32<KIND>(bf16_at(vv[k][0], i), bf16_at(vv[k][1], i), bf16_at(vv[k][2], i), bf16_at(vv[k][3], i), scale, inv)
                       : 0;
        }
      }
      __syncthreads();
      for (int e = t; e < D * PAGE / 16; e += WG) {
        const int d = e / (PAGE / 16), j = e % (PAGE / 16) * 16;
        const uint32_t* from = codes + (d * ROW + j) / 4;
        *reinterpret_cast<u32x4*>(a.c.v_pages + (at * D + d) * PAGE + j) = u32x4{from[0], from[1], from[2], from[3]};
      }
    }
  }
  if (unit) return;
  __syncthreads();  // the tail's old tokens have been read
  // The window of the tokens after the last full block.
  const int j0 = r.filled * PAGE, all = r.tail + r.n;
  turns(j0);
  for (int h = h0; h < h1; ++h)
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int e = k * WG + t, j = j0 + e / PER;
      if (e >= PAGE * PER || j < r.tail || j >= all) continue;
      const Pieces p = pieces_of(e % PER, a.rot.dims, a.rot.interleaved);
      const uint16_t* from = token(false, j) + h * D;
      const uint16_t* fresh = token(true, j) + h * D;
      u32x4 u = *reinterpret_cast<const u32x4*>(from + p.p0 * 8), w = *reinterpret_cast<const u32x4*>(from + p.p1 * 8);
      const u32x4 x = *reinterpret_cast<const u32x4*>(fresh + p.p0 * 8), y = *reinterpret_cast<const u32x4*>(fresh + p.p1 * 8);
      turn(k, h, j, u, w);
      const int64_t to = ((int64_t)b * a.c.tail + place(j)) * slot + h * D;
      *reinterpret_cast<u32x4*>(a.c.k_tail + to + p.p0 * 8) = u;
      *reinterpret_cast<u32x4*>(a.c.k_tail + to + p.p1 * 8) = w;
      *reinterpret_cast<u32x4*>(a.c.v_tail + to + p.p0 * 8) = x;
      *reinterpret_cast<u32x4*>(a.c.v_tail + to + p.p1 * 8) = y;
    }
}

// Counters updated in place: after every work-group has read them.
__global__ __launch_bounds__(WG) void append_counters_kernel(AppendArgs a) {
  __shared__ int bad;
  const int b = blockIdx.x;
  const Append r = row_append(a, b, &bad);
  if (threadIdx.x == 0) {
    a.positions_out[b] = r.pos + r.n;
    a.blocks_out[b] = r.blocks + r.filled;
  }
}

template <int KIND, int D>
auto kernel_of_page(int page) -> void (*)(AppendArgs) {
  return page == 16 ? cache_append_kernel<KIND, D, 16> : page == 32 ? cache_append_kernel<KIND, D, 32>
         : page == 64 ? cache_append_kernel<KIND, D, 64> : page == 128 ? cache_append_kernel<KIND, D, 128>
                                                                       : cache_append_kernel<KIND, D, 256>;
}
auto kernel_of(const sv_cache& c) -> void (*)(AppendArgs) {
  return c.kind == SV_E4M3 ? (c.D == 64 ? kernel_of_page<SV_E4M3, 64>(c.page) : kernel_of_page<SV_E4M3, 128>(c.page))
                           : (c.D == 64 ? kernel_of_page<SV_INT8, 64>(c.page) : kernel_of_page<SV_INT8, 128>(c.page));
}

constexpr int MAX_TOKENS = 1 << 24;

}  // namespace

extern "C" int spec_verify_append(const void* k, const void* v, int64_t kv_row, int64_t kv_tok, int T,
                                  const int32_t* lens, const sv_rotary* rotary, const sv_cache* cache,
                                  const int32_t* positions, const int32_t* blocks, int32_t* positions_out,
                                  int32_t* blocks_out, void* k_out, int64_t ko_row, int64_t ko_tok,
                                  hipStream_t stream) {
  const int bad = check_cache(cache);
  if (bad != SV_OK) return bad;
  const sv_cache& c = *cache;
  if (!k || !v || !positions || !blocks || !positions_out || !blocks_out || T < 1) return SV_ERR_ARG;
  if (T > MAX_TOKENS) return SV_ERR_UNSUPPORTED;
  if (rotary) {
    const int rc = check_rotary(rotary, c.D);
    if (rc != SV_OK) return rc;
  }
  if ((positions == positions_out) != (blocks == blocks_out)) return SV_ERR_ARG;
  const size_t nb = (size_t)c.B * 4, pages = (size_t)c.num_pages * c.Hkv, tail = (size_t)c.B * c.tail * c.Hkv * c.D * 2;
  const size_t ids = rotary && rotary->ids ? nb * T * rotary->num_axes : 0;
  const size_t words = rotary ? (size_t)rotary->dims * 2 : 0;
  const Array lists[] = {{positions, nb}, {blocks, nb}, {lens, nb}, {c.block_table, nb * c.max_blocks},
                         {rotary ? rotary->freqs : nullptr, words}, {rotary ? rotary->axes : nullptr, words},
                         {rotary ? rotary->ids : nullptr, ids}};
  const Output counters[] = {{{positions_out, nb}, positions}, {{blocks_out, nb}, blocks}};
  if (outputs_overlap(counters, lists)) return SV_ERR_ARG;
  const void* aligned[] = {k, v, k_out};
  for (const void* p : aligned)
    if (reinterpret_cast<uintptr_t>(p) % 16) return SV_ERR_ARG;
  constexpr int64_t FAR = int64_t(1) << 40;
  const int64_t strides[] = {kv_row, kv_tok, ko_row, ko_tok};
  for (int64_t s : strides)
    if (s < 0 || s > FAR || s % 8) return SV_ERR_ARG;
  const int64_t width = (int64_t)c.Hkv * c.D * 2;
  const View in[] = {{k, kv_row * 2, kv_tok * 2, width}, {v, kv_row * 2, kv_tok * 2, width}};
  // Work-groups write the cache and the counters while others still read the prompt and the lists.
  const Array written[] = {{positions_out, nb}, {blocks_out, nb}, {c.k_pages, pages * c.page * c.D},
                           {c.v_pages, pages * c.page * c.D}, {c.k_scale, pages * 4}, {c.v_scale, pages * 4},
                           {c.k_tail, tail}, {c.v_tail, tail}};
  for (const Array& o : written) {
    for (const View& i : in)
      if (overlap({i.p, (size_t)((c.B - 1) * i.row + (T - 1) * i.tok + i.width)}, o)) return SV_ERR_ARG;
    if (&o < written + 2) continue;  // the counters: above
    for (const Array& i : lists)
      if (overlap(i, o)) return SV_ERR_ARG;
    for (const Output& i : counters)
      if (overlap(i.a, o)) return SV_ERR_ARG;
  }
  if (k_out) {
    const View out = {k_out, ko_row * 2, ko_tok * 2, width};
    const Array whole = {k_out, (size_t)((c.B - 1) * out.row + (T - 1) * out.tok + out.width)};
    if (view_overlaps_itself(out, c.B, T) || views_clash(in[0], out, c.B, T, true) ||
        views_clash(in[1], out, c.B, T, false))
      return SV_ERR_ARG;
    for (const Array& o : written)
      if (overlap(whole, o)) return SV_ERR_ARG;
    for (const Array& i : lists)
      if (overlap(whole, i)) return SV_ERR_ARG;
  }
  AppendArgs a = {};
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.kv_row = kv_row;
  a.kv_tok = kv_tok;
  a.k_out = static_cast<uint16_t*>(k_out);
  a.ko_row = ko_row;
  a.ko_tok = ko_tok;
  if (rotary) a.rot = *rotary;
  a.c = c;
  a.lens = lens;
  a.positions = positions;
  a.blocks = blocks;
  a.positions_out = positions_out;
  a.blocks_out = blocks_out;
  a.T = T;
  a.units = (c.page - 1 + T) / c.page;  // blocks that T tokens complete at most
  const int64_t rows = (int64_t)c.B * a.units;
  // Heads that share a work-group's cosines: as many as leave 4096 work-groups
  // (16 prompts of up to 4096 tokens: 112 us with two of eight heads, 115 with
  // four, 129 with all).
  a.heads = 1;
  while (a.heads < c.Hkv && rows * ((c.Hkv + 2 * a.heads - 1) / (2 * a.heads)) >= 4096) a.heads *= 2;
  a.groups = (c.Hkv + a.heads - 1) / a.heads;
  a.inplace = positions == positions_out;
  if (rows * a.groups > MAX_ITEMS / WG) return SV_ERR_UNSUPPORTED;
  (void)hipGetLastError();
  hipLaunchKernelGGL(kernel_of(c), dim3((uint32_t)(rows * a.groups)), dim3(WG), 0, stream, a);
  if (hipGetLastError() != hipSuccess) return SV_ERR_HIP;
  if (a.inplace) {
    hipLaunchKernelGGL(append_counters_kernel, dim3(c.B), dim3(WG), 0, stream, a);
    if (hipGetLastError() != hipSuccess) return SV_ERR_HIP;
  }
  return SV_OK;
}
