// The rotation of queries and keys by their positions (see sv_rotary in
// spec_verify.h).
#pragma once

#include "cache.h"

namespace svr {

constexpr int MAX_ROTARY_AXES = 16;

// Checks of the description that every entry point makes.
inline int check_rotary(const sv_rotary* r, int D) {
  if (!r || !r->freqs || reinterpret_cast<uintptr_t>(r->freqs) % 4) return SV_ERR_ARG;
  if (r->dims < 1 || r->dims > D || (r->interleaved != 0 && r->interleaved != 1)) return SV_ERR_ARG;
  if (r->dims % 16) return SV_ERR_UNSUPPORTED;
  if (r->ids) {
    if (r->num_axes < 1 || reinterpret_cast<uintptr_t>(r->ids) % 4) return SV_ERR_ARG;
    if (r->num_axes > MAX_ROTARY_AXES) return SV_ERR_UNSUPPORTED;
    if (reinterpret_cast<uintptr_t>(r->axes) % 4) return SV_ERR_ARG;
  } else if (r->axes) {
    return SV_ERR_ARG;
  }
  return SV_OK;
}

// cos and sin of x, |x| <= 2^52, each to less than 2^-51: x is brought to
// [-pi/4, pi/4] by fused multiply-adds with pi/2 in two parts, which lose
// nothing of it, and the Taylor series there end with terms below 2^-54.
// All in float64 because a far position's angle has more turns than float32
// has bits to spare; fp64 instructions cost no more than fp32 ones here.
__device__ __forceinline__ float2 cos_sin(double x) {
  const double k = rint(x * 0.63661977236758134308);
  double r = fma(-k, 1.5707963267948965580, x);
  r = fma(-k, 6.1232339957367658860e-17, r);
  const double z = r * r;
  double s = -1.0 / 1307674368000.0;
  s = fma(s, z, 1.0 / 6227020800.0);
  s = fma(s, z, -1.0 / 39916800.0);
  s = fma(s, z, 1.0 / 362880.0);
  s = fma(s, z, -1.0 / 5040.0);
  s = fma(s, z, 1.0 / 120.0);
  s = fma(s, z, -1.0 / 6.0);
  s = fma(s * z, r, r);
  double c = 1.0 / 20922789888000.0;
  c = fma(c, z, -1.0 / 87178291200.0);
  c = fma(c, z, 1.0 / 479001600.0);
  c = fma(c, z, -1.0 / 3628800.0);
  c = fma(c, z, 1.0 / 40320.0);
  c = fma(c, z, -1.0 / 720.0);
  c = fma(c, z, 1.0 / 24.0);
  c = fma(c, z, -0.5);
  c = fma(c, z, 1.0);
  // The quadrant: k modulo 4, k a whole number of float64.
  const int quarter = (int)(k - 4.0 * floor(k * 0.25));
  const float cf = (float)c, sf = (float)s;
  const float a = quarter & 1 ? sf : cf, b = quarter & 1 ? cf : sf;
  return make_float2(quarter == 1 || quarter == 2 ? -a : a, quarter & 2 ? -b : b);
}

// cos and sin for pair i of token t of row b, whose position is `at` unless
// positions are given by axis.
__device__ __forceinline__ float2 turn_of(const sv_rotary& r, int B, int T, int b, int t, int i, int64_t at) {
  if (r.ids) {
    const int axis = r.axes ? min(max(r.axes[i], 0), r.num_axes - 1) : 0;
    at = r.ids[((int64_t)axis * B + b) * T + t];
  }
  return cos_sin((double)at * (double)r.freqs[i]);
}

// Of a token's D / 8 pieces of 8 channels (16 bytes), the two that thread c of
// D / 16 takes: those whose channels are paired where the pairs are half of
// the rotated channels apart, neighbours elsewhere.
struct Pieces {
  int p0, p1;
};
__device__ __forceinline__ Pieces pieces_of(int c, int dims, int interleaved) {
  const int half = dims / 16;
  if (!interleaved && c < half) return {c, c + half};
  return {2 * c, 2 * c + 1};  // past the rotated ones too: 2 half + 2 (c - half)
}

__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x, y}, bf16x2));
}

// Rotates the two pieces of thread c; cs: cos and sin of the token's pairs 8 c
// .. 8 c + 7.  Products and sums are rounded to float32 one by one, the results
// once to bf16.
__device__ __forceinline__ void rotate_pieces(u32x4& u, u32x4& v, int interleaved, const float2* cs) {
  if (!interleaved) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 w0 = cs[2 * k], w1 = cs[2 * k + 1];
      const float a0 = __uint_as_float(u[k] << 16), a1 = __uint_as_float(u[k] & 0xFFFF0000u);
      const float b0 = __uint_as_float(v[k] << 16), b1 = __uint_as_float(v[k] & 0xFFFF0000u);
      u[k] = pack_bf16(a0 * w0.x - b0 * w0.y, a1 * w1.x - b1 * w1.y);
      v[k] = pack_bf16(b0 * w0.x + a0 * w0.y, b1 * w1.x + a1 * w1.y);
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {  // words of the two pieces are pairs
    const float2 w = cs[k];
    const uint32_t x = k < 4 ? u[k & 3] : v[k & 3];
    const float a = __uint_as_float(x << 16), b = __uint_as_float(x & 0xFFFF0000u);
    (k < 4 ? u : v)[k & 3] = pack_bf16(a * w.x - b * w.y, b * w.x + a * w.y);
  }
}

// The elements [0, width) of every token of a [B, T] view, strides in bytes.
struct View {
  const void* p;
  int64_t row, tok, width;
};
// Whether `out` shares bytes with `in`, other than by being it, element for
// element, where it may be (`same`).  Views of one tensor (the parts of a fused projection) may lie
// between each other: where both have one stride from token to token, rows a
// multiple of it, they are apart if they are within one stride.  Other views
// whose first and last bytes enclose each other count as sharing.
inline bool views_clash(const View& in, const View& out, int B, int64_t T, bool same) {
  if (!in.p || !out.p) return false;
  const bool rows = B > 1, toks = T > 1;
  if (in.p == out.p && in.width == out.width && (!rows || in.row == out.row) && (!toks || in.tok == out.tok)) return !same;
  auto span = [&](const View& v) { return (rows ? (B - 1) * v.row : 0) + (toks ? (T - 1) * v.tok : 0) + v.width; };
  const int64_t d = reinterpret_cast<intptr_t>(out.p) - reinterpret_cast<intptr_t>(in.p);
  if (d >= span(in) || -d >= span(out)) return false;
  const int64_t s = toks ? in.tok : in.row;
  if (s <= 0 || (toks ? out.tok : out.row) != s) return true;
  if (toks && rows && (in.row != out.row || in.row % s)) return true;
  const int64_t at = ((d % s) + s) % s;
  return at < in.width || at + out.width > s;
}
// Whether two tokens of an output share bytes.
inline bool view_overlaps_itself(const View& v, int B, int64_t T) {
  if (T > 1 && v.tok < v.width) return true;
  return B > 1 && v.row < (T > 1 ? (T - 1) * v.tok : 0) + v.width;
}

}  // namespace svr
