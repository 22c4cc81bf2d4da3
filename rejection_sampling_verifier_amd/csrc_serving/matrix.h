// What the attention kernels over the 8-bit cache share: lanes that stand
// apart, codes widened to matrix operands, value scales.
#pragma once

#include "cache.h"

namespace svr {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float VMIN = 0x1p-126f;  // smallest value scale told apart (see spec_verify.h)
constexpr float GROW = 4.f;    // a maximum may lag this much (a factor of 16) before the sums are rescaled
constexpr float ALIKE = 4.f;   // value scales of one tile that differ by 2^5 and more need more range than f16 has
constexpr float LOW = -110.f;  // scores further below the maximum count as this far, so that 2^x stays in float32's range
constexpr float FAR = 0x1p127f;  // in place of an infinite -m, where every score is -inf
constexpr int TOP = 100;       // sums are not raised above 2^TOP
constexpr int LOST = -40;

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

// A block's value scale as 2^e f, 1 <= f < 2.
struct ValueScale {
  int e;
  float log, inv;  // log2 f, 1 / f; -inf and 0 where there is no block
};
__device__ __forceinline__ ValueScale value_scale(float v, bool any) {
  v = !any ? 1.f : v < VMIN ? VMIN : v;
  const float f = 2.f * __builtin_amdgcn_frexp_mantf(v);
  return {__builtin_amdgcn_frexp_expf(v) - 1, any ? __builtin_amdgcn_logf(f) : sv::NEG_INF, any ? __builtin_amdgcn_rcpf(f) : 0.f};
}

}  // namespace svr
