// Attention over a prefix that rows share, and its join with what the rows
// have of their own.
#pragma once

#include "cache.h"

namespace svr {

struct PrefixArgs {
  const uint16_t* q;
  int64_t q_row, q_tok;
  sv_cache c;
  sv_prefix p;
  const int32_t* qlens;
  int T, H, G, pshift;
  int qtiles, splits;   // tiles of queries at most, parts of a prefix's keys
  float scale2;         // scale * log2(e)
  float* part_o;        // [splits][B][T][H][D] means of a part's values
  float* part_ml;       // [splits][B][T][H][2] its maximum and sum
  const float* own;     // [B][T][H][D] what the rows have of their own
  float* lse;           // [B][Hkv][mpad] log2 of its softmax denominator; then of the whole one
  int mpad;
  uint16_t* out;
};

struct PrefixPlan {
  int qtiles, splits;
  size_t o, ml, own, total;  // from the start of the prefix's part of the workspace
};

int check_prefix(const sv_prefix* p);
int prefix_plan(const sv_cache& c, const sv_prefix& p, int T, int H, PrefixPlan& pl);
int prefix_launch(const PrefixArgs& a, hipStream_t st);
int prefix_join(const PrefixArgs& a, hipStream_t st);

}  // namespace svr
