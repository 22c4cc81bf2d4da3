// What the kernels over the paged 8-bit cache share.
#pragma once

#include <cstdint>

#include "spec_verify.h"
#include "sv_device.h"

namespace svr {

using sv::u32x4;
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int64_t MAX_ITEMS = UINT32_MAX;  // a launch has fewer than 2^32 work-items

// The counters of one row, brought into range: full blocks kept and tokens
// in the tail (its first token's ring slot is `start`).
struct RowState {
  int blocks, tail, start;
};
__device__ __forceinline__ RowState row_state(const sv_cache& c, const int32_t* positions, const int32_t* blocks, int b) {
  RowState s;
  s.blocks = min(max(blocks[b], 0), c.max_blocks);
  const int pos = max(positions[b], 0);
  s.tail = pos & (c.page - 1);
  s.start = (pos - s.tail) % c.tail;
  return s;
}

// An argument's array.
struct Array {
  const void* p;
  size_t bytes;
};
// Whether an output shares bytes with another output, or with an input other
// than the one that it may be itself (updated in place).
struct Output {
  Array a;
  const void* in;
};
inline bool overlap(const Array& a, const Array& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && x < y + b.bytes && y < x + a.bytes;
}
template <size_t NO, size_t NI>
inline bool outputs_overlap(const Output (&out)[NO], const Array (&in)[NI]) {
  for (size_t i = 0; i < NO; ++i) {
    for (size_t j = 0; j < i; ++j)
      if (overlap(out[i].a, out[j].a)) return true;
    for (const Array& a : in)
      if (!(a.p == out[i].a.p && a.p == out[i].in) && overlap(out[i].a, a)) return true;
  }
  return false;
}

// Checks of the cache's description that every entry point makes.
inline int check_cache(const sv_cache* c) {
  if (!c || !c->k_pages || !c->v_pages || !c->k_scale || !c->v_scale || !c->k_tail || !c->v_tail || !c->block_table)
    return SV_ERR_ARG;
  if (c->B < 1 || c->num_pages < 1 || c->Hkv < 1 || c->max_blocks < 1 || c->page < 1 || c->tail < 1 ||
      (c->kind != SV_E4M3 && c->kind != SV_INT8))
    return SV_ERR_ARG;
  if ((c->D != 64 && c->D != 128) || c->page < 16 || c->page > 256 || (c->page & (c->page - 1)) || c->Hkv > 4096 ||
      c->max_blocks > SV_MAX_BLOCKS || c->B > 65536)
    return SV_ERR_UNSUPPORTED;
  if (c->tail % c->page || c->tail > (1 << 20)) return SV_ERR_ARG;
  const void* aligned[] = {c->k_pages, c->v_pages, c->k_tail, c->v_tail};
  for (const void* p : aligned)
    if (reinterpret_cast<uintptr_t>(p) % 16) return SV_ERR_ARG;
  const void* words[] = {c->k_scale, c->v_scale, c->block_table};
  for (const void* p : words)
    if (reinterpret_cast<uintptr_t>(p) % 4) return SV_ERR_ARG;
  return SV_OK;
}

}  // namespace svr
