// A prompt's keys and values enter the paged 8-bit cache, the keys rotated by
// their positions on the way (spec_verify_append), for gfx950.
//
// Mathematics: rotation (rotary.h), then per completed block and head what a
// commit does (quantise.h).  Bytes bound it: two are read and one is written
// for each element.  A work-group takes one block of a row with some of its
// heads, a head at a time: its values wait in registers, rotated, for their
// largest magnitude.  Cos and sin of up to 64 tokens lie in LDS for all heads
// of the work-group.  The tokens after the last full block go to the tail by
// the work-group of the row's first block, which is also the one that reads
// the tail's old tokens, so that a ring of a single block will do.

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
  constexpr int NV = PAGE * PER < WG ? 1 : PAGE * PER / WG;    // those of a block, per thread
  constexpr int CH = PAGE < 64 ? PAGE : 64;                    // tokens whose cos and sin are in LDS
  constexpr int STEPS = CH * PER < WG ? 1 : CH * PER / WG;     // of a thread's pairs in as many tokens
  __shared__ int bad;
  __shared__ uint32_t tops[NWAVE];
  __shared__ alignas(16) float2 cs[CH * (D / 2)];
  __shared__ alignas(16) uint8_t codes[D * (PAGE + TPAD)];     // V: its channels' tokens side by side
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
  const int pairs = a.rot.dims / 2;
  auto place = [&](int j) {  // ring slot of the row's j-th token since its last full block before the call
    const int s = (r.start + j % a.c.tail);
    return s < a.c.tail ? s : s - a.c.tail;
  };
  // The row's tokens j0 .. j0 + CH - 1: their cos and sin, as far as they are new.
  auto turns = [&](int j0) {
    if (!pairs) return;
    __syncthreads();
    for (int e = t; e < CH * pairs; e += WG) {
      const int at = j0 + e / pairs - r.tail;  // its number among the new ones
      if (at >= 0 && at < r.n) cs[e] = turn_of(a.rot, a.c.B, a.T, b, at, e % pairs, (int64_t)r.pos + at);
    }
    __syncthreads();
  };
  // Piece pair c of head h of token j, which is jc-th of those in LDS: rotated and put out, if it is a new key.
  auto take = [&](bool val, int h, int j, int jc, int c, u32x4& u, u32x4& w) {
    const Pieces p = pieces_of(c, a.rot.dims, a.rot.interleaved);
    const uint16_t* from = j < r.tail
        ? (val ? a.c.v_tail : a.c.k_tail) + ((int64_t)b * a.c.tail + place(j)) * slot + h * D
        : (val ? a.v : a.k) + b * a.kv_row + (j - r.tail) * a.kv_tok + h * D;
    u = *reinterpret_cast<const u32x4*>(from + p.p0 * 8);
    w = *reinterpret_cast<const u32x4*>(from + p.p1 * 8);
    if (val || j < r.tail) return;
    if (pairs) rotate_pieces(u, w, c, a.rot.dims, a.rot.interleaved, cs + jc * pairs);
    if (a.k_out) {
      uint16_t* to = a.k_out + b * a.ko_row + (j - r.tail) * a.ko_tok + h * D;
      *reinterpret_cast<u32x4*>(to + p.p0 * 8) = u;
      *reinterpret_cast<u32x4*>(to + p.p1 * 8) = w;
    }
  };

  if (unit < r.filled) {
    const int j0 = unit * PAGE;
    if (PAGE == CH) turns(j0);
    const int pid = a.c.block_table[(int64_t)b * a.c.max_blocks + r.blocks + unit];
    for (int hv = h0 * 2; hv < h1 * 2; ++hv) {
      const int h = hv >> 1;
      const bool val = hv & 1;
      const int64_t at = (int64_t)pid * a.c.Hkv + h;
      u32x4 v[NV][2];
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (PAGE != CH && !val && k % STEPS == 0) turns(j0 + k / STEPS * CH);
        const int e = k * WG + t, j = e / PER;
        v[k][0] = v[k][1] = u32x4{0, 0, 0, 0};
        if (e < PAGE * PER) take(val, h, j0 + j, j % CH, e % PER, v[k][0], v[k][1]);
      }
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t w = v[k][i >> 2][i & 3];
          top = max(top, max(w & 0x7FFFu, (w >> 16) & 0x7FFFu));
        }
#pragma unroll
      for (int o = 32; o; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o, 64));
      __syncthreads();  // what the head before left in LDS has been read
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
        const int e = k * WG + t, j = e / PER;
        if (e >= PAGE * PER) continue;
        const Pieces p = pieces_of(e % PER, a.rot.dims, a.rot.interleaved);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int d = (half ? p.p1 : p.p0) * 8;
          uint32_t w[2] = {0, 0};
          if (finite) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i >> 2] |= code8<KIND>(bf16_at(v[k][half], i), scale, inv) << (8 * (i & 3));
          }
          if (!val) {
            *reinterpret_cast<uint2*>(a.c.k_pages + (at * PAGE + j) * D + d) = make_uint2(w[0], w[1]);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) codes[(d + i) * (PAGE + TPAD) + j] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
          }
        }
      }
      if (!val) continue;
      __syncthreads();
      for (int e = t; e < D * PAGE / 16; e += WG) {
        const int d = e / (PAGE / 16), j = e % (PAGE / 16) * 16;
        *reinterpret_cast<u32x4*>(a.c.v_pages + (at * D + d) * PAGE + j) =
            *reinterpret_cast<const u32x4*>(codes + d * (PAGE + TPAD) + j);
      }
    }
  }
  if (unit) return;
  __syncthreads();  // the tail's old tokens have been read
  const int all = r.tail + r.n;
  for (int j0 = max(r.tail, r.filled * PAGE); j0 < all; j0 += CH) {
    turns(j0);
    const int n = min(CH, all - j0) * (h1 - h0) * 2 * PER;
    for (int e = t; e < n; e += WG) {
      const int c = e % PER, h = h0 + (e / PER >> 1) % (h1 - h0), jc = e / (PER * 2) / (h1 - h0);
      const bool val = e / PER & 1;
      u32x4 u, w;
      take(val, h, j0 + jc, jc, c, u, w);
      const Pieces p = pieces_of(c, a.rot.dims, a.rot.interleaved);
      uint16_t* to = (val ? a.c.v_tail : a.c.k_tail) + ((int64_t)b * a.c.tail + place(j0 + jc)) * slot + h * D;
      *reinterpret_cast<u32x4*>(to + p.p0 * 8) = u;
      *reinterpret_cast<u32x4*>(to + p.p1 * 8) = w;
    }
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
  // Work-groups write the cache and the counters while others still read the prompt.
  const Array written[] = {{c.k_pages, pages * c.page * c.D}, {c.v_pages, pages * c.page * c.D}, {c.k_scale, pages * 4},
                           {c.v_scale, pages * 4}, {c.k_tail, tail}, {c.v_tail, tail}, {positions_out, nb},
                           {blocks_out, nb}};
  for (const View& i : in)
    for (const Array& o : written)
      if (overlap({i.p, (size_t)((c.B - 1) * i.row + (T - 1) * i.tok + i.width)}, o)) return SV_ERR_ARG;
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
  a.heads = 1;
  while (a.heads < c.Hkv && rows * ((c.Hkv + 2 * a.heads - 1) / (2 * a.heads)) >= 2048) a.heads *= 2;
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
