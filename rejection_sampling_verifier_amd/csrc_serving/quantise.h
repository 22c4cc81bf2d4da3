// How a block of bf16 values becomes 8-bit codes and a scale (see
// spec_verify_commit in spec_verify.h).
#pragma once

#include "cache.h"

namespace svr {

__device__ __forceinline__ float bf16_at(const u32x4& v, int k) { return sv::Tr<uint16_t>::at(v, k); }

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

// Four codes in a word.
template <int KIND>
__device__ __forceinline__ uint32_t code32(float x0, float x1, float x2, float x3, float scale, float inv) {
  if (KIND == SV_E4M3) {
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(x0 * inv, x1 * inv, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x2 * inv, x3 * inv, lo, true);
  }
  return code8<KIND>(x0, scale, inv) | code8<KIND>(x1, scale, inv) << 8 | code8<KIND>(x2, scale, inv) << 16 |
         code8<KIND>(x3, scale, inv) << 24;
}

constexpr int TPAD = 16;  // bytes between the channels of a buffer that transposes a block's codes

}  // namespace svr
