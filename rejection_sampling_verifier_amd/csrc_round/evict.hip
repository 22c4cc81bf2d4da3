// Blocks of least accumulated attention leave the cache (spec_verify_evict),
// for gfx950.
//
// Mathematics: the e smallest of a row's totals, ties to the earlier block: a
// radix selection over order-preserving keys finds the e-th smallest key, and
// one stable pass parts the row's table by it.  Integer counts only, so the
// result does not depend on any order of arrival.  It reads a row's totals
// and table once from memory (again from cache) and is bound by latency.
//
// One work-group per row.

#include <climits>

#include "cache.h"

using namespace sv;
using svr::overlap;

namespace {

constexpr int ET = 1024;               // threads
constexpr int EW = ET / 64;            // waves
constexpr int INPLACE_BLOCKS = 16384;  // evicted pages that LDS can hold while the table is rewritten

struct EvictArgs {
  const float* totals;
  const int32_t* table;
  const int32_t* blocks;
  float* totals_out;
  int32_t* table_out;
  int32_t* blocks_out;
  int32_t* evicted;
  int most, budget, first, last;
  int staged;  // table_out is the table: evicted pages wait in LDS
};

__device__ __forceinline__ uint32_t key_of(float x) { return x != x ? 0xFFFFFFFFu : order_key(x); }

// Exclusive prefix of v over the work-group's threads, and the total.
__device__ __forceinline__ int scan(int v, int* sh, int& total) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(inc, o, 64);
    if (lane >= o) inc += u;
  }
  if (lane == 63) sh[w] = inc;
  __syncthreads();
  int base = 0, all = 0;
#pragma unroll
  for (int k = 0; k < EW; ++k) {
    if (k < w) base += sh[k];
    all += sh[k];
  }
  __syncthreads();
  total = all;
  return base + inc - v;
}

__global__ __launch_bounds__(ET) void cache_evict_kernel(EvictArgs a) {
  __shared__ int hist[256];
  __shared__ int sums[EW];
  __shared__ uint32_t found[2];
  extern __shared__ int32_t staged[];
  const int t = threadIdx.x, b = blockIdx.x;
  const float* tot = a.totals + (int64_t)b * a.most;
  const int32_t* table = a.table + (int64_t)b * a.most;
  float* tot_out = a.totals_out + (int64_t)b * a.most;
  int32_t* table_out = a.table_out + (int64_t)b * a.most;
  const int n = min(max(a.blocks[b], 0), a.most);
  const int lo = min(a.first, n), hi = max(n - min(a.last, n), lo);
  const int e = min(max(n - a.budget, 0), hi - lo);

  // The e-th smallest key, and how many of the keys equal to it leave.
  uint32_t key = 0;
  int ties = 0;
  if (e > 0) {
    int want = e;
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (t < 256) hist[t] = 0;
      __syncthreads();
      for (int j = lo + t; j < hi; j += ET) {
        const uint32_t k = key_of(tot[j]);
        if (shift == 24 || (k >> (shift + 8)) == (key >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255], 1);
      }
      __syncthreads();
      int all;
      const int c = t < 256 ? hist[t] : 0;
      const int before = scan(c, sums, all);
      if (before < want && want <= before + c) {
        found[0] = (uint32_t)t;
        found[1] = (uint32_t)(want - before);
      }
      __syncthreads();
      key |= found[0] << shift;
      want = (int)found[1];
      __syncthreads();
    }
    ties = want;
  }

  // Kept blocks to the front, evicted ones behind them, in order.
  int kept = 0, gone = 0, equal = 0;
  for (int j0 = 0; j0 < n; j0 += ET) {
    const int j = j0 + t;
    float x = 0.f;
    int32_t p = 0;
    bool may = false;
    uint32_t k = 0;
    if (j < n) {
      x = tot[j];
      p = table[j];
      k = key_of(x);
      may = e > 0 && j >= lo && j < hi;
    }
    int all;
    const int eq = scan(may && k == key, sums, all);
    const bool out = may && (k < key || (k == key && equal + eq < ties));
    equal += all;
    const int rank = scan(out, sums, all);
    if (j < n) {
      if (!out) {
        const int to = kept + (t - rank);
        table_out[to] = p;
        tot_out[to] = x;
      } else if (a.staged) {
        staged[gone + rank] = p;
      } else {
        table_out[n - e + gone + rank] = p;
      }
    }
    gone += all;
    kept += min(ET, n - j0) - all;
  }
  __syncthreads();
  if (a.staged)
    for (int j = t; j < e; j += ET) table_out[n - e + j] = staged[j];
  else
    for (int j = n + t; j < a.most; j += ET) table_out[j] = table[j];
  for (int j = n - e + t; j < a.most; j += ET) tot_out[j] = 0.f;
  if (t == 0) {
    a.blocks_out[b] = n - e;
    a.evicted[b] = e;
  }
}

}  // namespace

extern "C" int spec_verify_evict(const float* totals, const int32_t* block_table, const int32_t* blocks, int B,
                                 int max_blocks, int budget, int keep_first, int keep_last, float* totals_out,
                                 int32_t* table_out, int32_t* blocks_out, int32_t* evicted, hipStream_t stream) {
  if (!totals || !block_table || !blocks || !totals_out || !table_out || !blocks_out || !evicted || B < 1 ||
      max_blocks < 1 || budget < 0 || keep_first < 0 || keep_last < 0)
    return SV_ERR_ARG;
  if (max_blocks > SV_MAX_BLOCKS) return SV_ERR_UNSUPPORTED;
  const size_t n = (size_t)B * max_blocks * 4;
  if ((totals_out != totals && overlap(totals_out, totals, n)) ||
      (table_out != block_table && overlap(table_out, block_table, n)) || overlap(totals_out, block_table, n) ||
      overlap(table_out, totals, n) || overlap(totals_out, table_out, n) ||
      (blocks_out != blocks && overlap(blocks_out, blocks, (size_t)B * 4)) || overlap(evicted, blocks, (size_t)B * 4) ||
      overlap(evicted, blocks_out, (size_t)B * 4))
    return SV_ERR_ARG;
  const bool staged = table_out == block_table;
  if (staged && max_blocks > INPLACE_BLOCKS) return SV_ERR_UNSUPPORTED;
  const EvictArgs a{totals, block_table, blocks, totals_out, table_out, blocks_out, evicted, max_blocks, budget,
                    keep_first, keep_last, staged};
  (void)hipGetLastError();
  hipLaunchKernelGGL(cache_evict_kernel, dim3(B), dim3(ET), staged ? (size_t)max_blocks * 4 : 0, stream, a);
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
}
