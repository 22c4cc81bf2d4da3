// Queries and keys of a step rotated by their positions (spec_verify_rotate),
// for gfx950.
//
// Mathematics: a pair of channels (a, b) becomes (a cos - b sin, b cos +
// a sin) of its position times its frequency.  Bytes bound it: each element
// is read and written once.  A work-group takes TT tokens with all their
// heads, so that a cos and sin, 60 instructions of float64, serve every head
// of the token from LDS; fewer tokens to a work-group where there are too few
// to fill the chip.

#include <climits>

#include "rotary.h"

using namespace sv;
using namespace svr;

namespace {

constexpr int MAX_DIM = 512;
constexpr int AHEAD = 4;  // pairs of pieces that a thread has on their way

struct RotateArgs {
  const uint16_t* q;
  const uint16_t* k;
  uint16_t* qo;
  uint16_t* ko;
  int64_t q_row, q_tok, k_row, k_tok, qo_row, qo_tok, ko_row, ko_tok;
  sv_rotary rot;
  const int32_t* positions;
  const int32_t* parents;
  const int32_t* qlens;
  int B, T, H, Hkv, D;
};

// Steps from the root to this lane's node of row b's tree (0 where its path
// starts elsewhere), for up to 64 nodes, a wave at once: each round doubles
// the steps taken.
__device__ __forceinline__ int depth_of(const int32_t* parents, int T) {
  const int t = threadIdx.x & 63;
  int up = -1, depth = 0;
  if (t > 0 && t < T) {
    const int p = parents[t];
    up = p >= 0 && p < t ? p : -1;
  }
  depth = up >= 0;
#pragma unroll
  for (int s = 0; s < 6; ++s) {
    const int src = up < 0 ? t : up;
    const int more = __shfl(depth, src, 64), next = __shfl(up, src, 64);
    if (up >= 0) {
      depth += more;
      up = next;
    }
  }
  return depth;
}

template <int TT>
__global__ __launch_bounds__(WG) void rotate_kernel(RotateArgs a, int groups) {
  __shared__ alignas(16) float2 cs[TT * (MAX_DIM / 2)];
  __shared__ int depth[64];
  const int t = threadIdx.x, b = blockIdx.x / groups, first = blockIdx.x % groups * TT;
  const int live = a.qlens ? min(max(a.qlens[b], 0), a.T) : a.T;
  const int n = min(TT, live - first);
  if (n <= 0) return;
  if (a.parents && !a.rot.ids) {
    if (t < 64) depth[t] = depth_of(a.parents + (int64_t)b * a.T, a.T);
    __syncthreads();
  }
  const int pairs = a.rot.dims / 2;
  const int64_t start = a.positions && !a.rot.ids ? a.positions[b] : 0;
  for (int e = t; e < n * pairs; e += WG) {
    const int j = e / pairs, i = e % pairs, at = first + j;
    cs[e] = turn_of(a.rot, a.B, a.T, b, at, i, start + (a.parents && !a.rot.ids ? depth[at] : at));
  }
  __syncthreads();
  const int per = a.D / 16, heads = a.H + a.Hkv, all = n * heads * per;
  for (int e0 = t; e0 < all; e0 += AHEAD * WG) {
    u32x4 u[AHEAD], v[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int e = min(e0 + k * WG, all - 1), head = e / per % heads, c = e % per;
      const Pieces p = pieces_of(c, a.rot.dims, a.rot.interleaved);
      const int64_t tok = first + e / per / heads;
      const uint16_t* from = head < a.H ? a.q + b * a.q_row + tok * a.q_tok + (int64_t)head * a.D
                                        : a.k + b * a.k_row + tok * a.k_tok + (int64_t)(head - a.H) * a.D;
      u[k] = *reinterpret_cast<const u32x4*>(from + p.p0 * 8);
      v[k] = *reinterpret_cast<const u32x4*>(from + p.p1 * 8);
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int e = e0 + k * WG, head = e / per % heads, c = e % per, j = e / per / heads;
      if (e >= all) break;
      const Pieces p = pieces_of(c, a.rot.dims, a.rot.interleaved);
      if (c < a.rot.dims / 16) rotate_pieces(u[k], v[k], a.rot.interleaved, cs + j * pairs + c * 8);
      const int64_t tok = first + j;
      uint16_t* to = head < a.H ? a.qo + b * a.qo_row + tok * a.qo_tok + (int64_t)head * a.D
                                : a.ko + b * a.ko_row + tok * a.ko_tok + (int64_t)(head - a.H) * a.D;
      *reinterpret_cast<u32x4*>(to + p.p0 * 8) = u[k];
      *reinterpret_cast<u32x4*>(to + p.p1 * 8) = v[k];
    }
  }
}

template <int TT>
int launch(const RotateArgs& a, hipStream_t st) {
  const int64_t groups = ((int64_t)a.T + TT - 1) / TT;
  if (a.B * groups > MAX_ITEMS / WG) return SV_ERR_UNSUPPORTED;
  (void)hipGetLastError();
  hipLaunchKernelGGL(rotate_kernel<TT>, dim3((uint32_t)(a.B * groups)), dim3(WG), 0, st, a, (int)groups);
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
}

}  // namespace

extern "C" int spec_verify_rotate(const void* q, int64_t q_row, int64_t q_tok, const void* k, int64_t k_row,
                                  int64_t k_tok, const sv_rotary* rotary, const int32_t* positions,
                                  const int32_t* parents, const int32_t* query_lens, int B, int T, int H, int Hkv,
                                  int D, void* q_out, int64_t qo_row, int64_t qo_tok, void* k_out, int64_t ko_row,
                                  int64_t ko_tok, hipStream_t stream) {
  if (!q || !k || !q_out || !k_out || B < 1 || T < 1 || H < 1 || Hkv < 1 || D < 1) return SV_ERR_ARG;
  if (D % 16 || D > MAX_DIM || H > 65536 || Hkv > 65536 || (parents && T > SV_MAX_NODES)) return SV_ERR_UNSUPPORTED;
  const int bad = check_rotary(rotary, D);
  if (bad != SV_OK) return bad;
  if (!positions && !rotary->ids) return SV_ERR_ARG;
  constexpr int64_t FAR = int64_t(1) << 40;
  const int64_t strides[] = {q_row, q_tok, k_row, k_tok, qo_row, qo_tok, ko_row, ko_tok};
  for (int64_t s : strides)
    if (s < 0 || s > FAR || s % 8) return SV_ERR_ARG;
  const void* aligned[] = {q, k, q_out, k_out};
  for (const void* p : aligned)
    if (reinterpret_cast<uintptr_t>(p) % 16) return SV_ERR_ARG;
  const int64_t qw = (int64_t)H * D * 2, kw = (int64_t)Hkv * D * 2;
  const View in[] = {{q, q_row * 2, q_tok * 2, qw}, {k, k_row * 2, k_tok * 2, kw}};
  const View out[] = {{q_out, qo_row * 2, qo_tok * 2, qw}, {k_out, ko_row * 2, ko_tok * 2, kw}};
  const size_t n = (size_t)B * 4;
  const View lists[] = {{positions, 0, 0, (int64_t)n},
                        {parents, 0, 0, (int64_t)(n * T)},
                        {query_lens, 0, 0, (int64_t)n},
                        {rotary->freqs, 0, 0, rotary->dims * 2},
                        {rotary->axes, 0, 0, rotary->dims * 2},
                        {rotary->ids, 0, 0, (int64_t)(n * T * (rotary->ids ? rotary->num_axes : 0))}};
  for (const View& o : out) {
    if (view_overlaps_itself(o, B, T)) return SV_ERR_ARG;
    for (const View& i : in)
      if (views_clash(i, o, B, T, (&o == out) == (&i == in))) return SV_ERR_ARG;
    // A list counts as lying over the output where it lies between its first byte and its last.
    const size_t whole = (size_t)((B - 1) * o.row + (T - 1) * o.tok + o.width);
    for (const View& l : lists)
      if (overlap({o.p, whole}, {l.p, (size_t)l.width})) return SV_ERR_ARG;
  }
  if (views_clash(out[0], out[1], B, T, false)) return SV_ERR_ARG;
  RotateArgs a = {static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k), static_cast<uint16_t*>(q_out),
                  static_cast<uint16_t*>(k_out), q_row, q_tok, k_row, k_tok, qo_row, qo_tok, ko_row, ko_tok, *rotary,
                  positions, parents, query_lens, B, T, H, Hkv, D};
  // 384 tokens of 40 heads: 5.6 us one to a work-group, 7.4 four; 2048: 12.5 and 10.6; 4096: 19.6 and 15.6.  Of 16
  // heads 4.8 and 4.9, 9.2 and 7.0, 13.8 and 9.9; of 136 9.2 and 15.7, 23.7 and 26.2, 44.6 and 46.2.
  const int64_t tokens = (int64_t)B * T;
  return tokens <= 2048 ? launch<1>(a, stream) : launch<4>(a, stream);
}
