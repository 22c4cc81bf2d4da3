// Blocks of least accumulated attention leave the cache (spec_verify_evict),
// for gfx950.
//
// Mathematics: the e smallest of a row's totals, ties to the earlier block: a
// radix selection over order-preserving keys (digits of 11, 11 and 10 bits:
// the first holds the whole exponent, so few totals share a counter) finds
// the e-th smallest key, and one stable pass parts the row's table by it.
// Integer counts only, so the result does not depend on any order of arrival.
// It is bound by latency: the steps of a selection follow each other.
//
// One work-group per row.  Up to 16384 blocks the threads hold the totals and
// pages in registers, neighbouring blocks in neighbouring lanes: memory is read
// once, a block's rank is a count over its wave's ballot and one prefix sum
// over the waves' counts, and nothing needs to be kept aside when the table is
// rewritten in place.  Longer rows are streamed (256 rows of up to 8191
// blocks: 31 us streamed, 18 us from registers).  Each kernel up to the size
// that it holds, against the next larger one at that size (one row, us):
// 256 blocks 6.0 and 6.7, 1024 8.0 and 7.8, 4096 9.7 and 10.7, 8192 13.2 and
// 14.7, 12288 17.3 and 18.9; of 256 rows 6.5 and 7.1, 8.6 and 8.6, 11.4 and
// 12.3, 17.4 and 18.5, 22.3 and 23.2.

#include <climits>

#include "cache.h"

using namespace sv;
using namespace svr;

namespace {

constexpr int ET = 1024;             // threads at most
constexpr int HELD_BLOCKS = 16384;   // rows that registers hold
constexpr int BINS = 2048;

struct EvictArgs {
  const float* totals;
  const int32_t* table;
  const int32_t* blocks;
  float* totals_out;
  int32_t* table_out;
  int32_t* blocks_out;
  int32_t* evicted;
  int most, budget, first, last;
};

// Row b's range of blocks that may leave, and how many do.
struct Row {
  int n, lo, hi, e;
};
__device__ __forceinline__ Row row_of(const EvictArgs& a, int b) {
  Row r;
  r.n = min(max(a.blocks[b], 0), a.most);
  r.lo = min(a.first, r.n);
  r.hi = max(r.n - min(a.last, r.n), r.lo);
  r.e = min(max(r.n - a.budget, 0), r.hi - r.lo);
  return r;
}

__device__ __forceinline__ uint32_t key_of(float x) { return x != x ? 0xFFFFFFFFu : order_key(x); }

// Exclusive prefix of v over the work-group's NT threads, and the total.
template <int NT>
__device__ __forceinline__ int scan(int v, int* sh, int& total) {
  constexpr int NW = NT / 64;
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
  for (int k = 0; k < NW; ++k) {
    if (k < w) base += sh[k];
    all += sh[k];
  }
  __syncthreads();
  total = all;
  return base + inc - v;
}

struct SelectLds {
  int hist[BINS];
  int sums[ET / 64];
  int found[2];
};

// The want-th smallest key (from 1) of those that `each` calls its argument
// with, and which of the keys equal to it that is.
template <int NT, typename F>
__device__ __forceinline__ uint32_t select(SelectLds& sh, int want, const F& each, int& rank) {
  const int t = threadIdx.x;
  uint32_t key = 0;
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    for (int k = t; k < BINS; k += NT) sh.hist[k] = 0;
    __syncthreads();
    each([&](uint32_t k) {
      if (pass == 0 || (k >> (shift + bits)) == (key >> (shift + bits)))
        atomicAdd(&sh.hist[(k >> shift) & ((1u << bits) - 1)], 1);
    });
    __syncthreads();
    constexpr int PER = BINS / NT;
    int c[PER], sum = 0, all;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      c[k] = sh.hist[t * PER + k];
      sum += c[k];
    }
    int before = scan<NT>(sum, sh.sums, all);
    if (before < want && want <= before + sum) {
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        if (before < want && want <= before + c[k]) {
          sh.found[0] = t * PER + k;
          sh.found[1] = want - before;
        }
        before += c[k];
      }
    }
    __syncthreads();
    key |= (uint32_t)sh.found[0] << shift;
    want = sh.found[1];
    __syncthreads();
  }
  rank = want;
  return key;
}

// How many of the flags before each of the thread's own, block i NT + t of the
// row being bit i's, are set: base[i] plus the lanes below.
template <int NT, int IPT>
__device__ __forceinline__ void ranks(const bool (&flag)[IPT], int* groups, int* sums, int (&rank)[IPT]) {
  constexpr int NW = NT / 64, G = IPT * NW;  // groups of 64 blocks, in order
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
#pragma unroll
  for (int i = 0; i < IPT; ++i) {
    const uint64_t m = __ballot(flag[i]);
    rank[i] = __popcll(m & ((1ull << lane) - 1));
    if (lane == 0) groups[i * NW + w] = __popcll(m);
  }
  __syncthreads();
  int all;
  const int before = scan<NT>(t < G ? groups[t] : 0, sums, all);
  if (t < G) groups[t] = before;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < IPT; ++i) rank[i] += groups[i * NW + w];
  __syncthreads();
}

// NT threads hold IPT blocks each.
template <int NT, int IPT>
__global__ __launch_bounds__(NT) void cache_evict_kernel(EvictArgs a) {
  static_assert(IPT * (NT / 64) <= NT, "a group of 64 blocks has a thread of its own");
  __shared__ SelectLds sh;
  const int t = threadIdx.x, b = blockIdx.x;
  const float* tot = a.totals + (int64_t)b * a.most;
  const int32_t* table = a.table + (int64_t)b * a.most;
  float* tot_out = a.totals_out + (int64_t)b * a.most;
  int32_t* table_out = a.table_out + (int64_t)b * a.most;
  float x[IPT];
  int32_t p[IPT];
#pragma unroll
  for (int i = 0; i < IPT; ++i) x[i] = i * NT + t < a.most ? tot[i * NT + t] : 0.f;
#pragma unroll
  for (int i = 0; i < IPT; ++i) p[i] = i * NT + t < a.most ? table[i * NT + t] : 0;
  const Row r = row_of(a, b);

  uint32_t key = 0;
  int ties = 0;
  if (r.e > 0)
    key = select<NT>(sh, r.e, [&](const auto& take) {
#pragma unroll
      for (int i = 0; i < IPT; ++i)
        if (i * NT + t >= r.lo && i * NT + t < r.hi) take(key_of(x[i]));
    }, ties);

  // Kept blocks to the front, evicted ones behind them, in order.  Every
  // thread has its values by the first barrier below.
  bool flag[IPT];
  int rank[IPT];
  auto may = [&](int i) { return r.e > 0 && i * NT + t >= r.lo && i * NT + t < r.hi; };
#pragma unroll
  for (int i = 0; i < IPT; ++i) flag[i] = may(i) && key_of(x[i]) == key;
  ranks<NT>(flag, sh.hist, sh.sums, rank);
#pragma unroll
  for (int i = 0; i < IPT; ++i) flag[i] = may(i) && (key_of(x[i]) < key || (flag[i] && rank[i] < ties));
  ranks<NT>(flag, sh.hist, sh.sums, rank);
#pragma unroll
  for (int i = 0; i < IPT; ++i) {
    const int j = i * NT + t;
    if (j >= a.most) break;
    table_out[j >= r.n ? j : flag[i] ? r.n - r.e + rank[i] : j - rank[i]] = p[i];
    if (j < r.n && !flag[i]) tot_out[j - rank[i]] = x[i];
    if (j >= r.n - r.e) tot_out[j] = 0.f;
  }
  if (t == 0) {
    a.blocks_out[b] = r.n - r.e;
    a.evicted[b] = r.e;
  }
}

// Rows of any length, read from memory in each step.  Totals may be rewritten
// in place (a kept block moves to the front, past what has been read).
__global__ __launch_bounds__(ET) void cache_evict_long_kernel(EvictArgs a) {
  __shared__ SelectLds sh;
  const int t = threadIdx.x, b = blockIdx.x;
  const float* tot = a.totals + (int64_t)b * a.most;
  const int32_t* table = a.table + (int64_t)b * a.most;
  float* tot_out = a.totals_out + (int64_t)b * a.most;
  int32_t* table_out = a.table_out + (int64_t)b * a.most;
  const Row r = row_of(a, b);
  uint32_t key = 0;
  int ties = 0;
  if (r.e > 0)
    key = select<ET>(sh, r.e, [&](const auto& take) {
      for (int j = r.lo + t; j < r.hi; j += ET) take(key_of(tot[j]));
    }, ties);

  int kept = 0, gone = 0, equal = 0;
  for (int j0 = 0; j0 < r.n; j0 += ET) {
    const int j = j0 + t;
    float x = 0.f;
    int32_t p = 0;
    bool may = false;
    uint32_t k = 0;
    if (j < r.n) {
      x = tot[j];
      p = table[j];
      k = key_of(x);
      may = r.e > 0 && j >= r.lo && j < r.hi;
    }
    int all;
    const int eq = scan<ET>(may && k == key, sh.sums, all);
    const bool out = may && (k < key || (k == key && equal + eq < ties));
    equal += all;
    const int rank = scan<ET>(out, sh.sums, all);
    if (j < r.n) {
      if (out) {
        table_out[r.n - r.e + gone + rank] = p;
      } else {
        const int to = kept + (t - rank);
        table_out[to] = p;
        tot_out[to] = x;
      }
    }
    gone += all;
    kept += min(ET, r.n - j0) - all;
  }
  __syncthreads();
  for (int j = r.n + t; j < a.most; j += ET) table_out[j] = table[j];
  for (int j = r.n - r.e + t; j < a.most; j += ET) tot_out[j] = 0.f;
  if (t == 0) {
    a.blocks_out[b] = r.n - r.e;
    a.evicted[b] = r.e;
  }
}

}  // namespace

extern "C" int spec_verify_evict(const float* totals, const int32_t* block_table, const int32_t* blocks, int B,
                                 int max_blocks, int budget, int keep_first, int keep_last, float* totals_out,
                                 int32_t* table_out, int32_t* blocks_out, int32_t* evicted, hipStream_t stream) {
  if (!totals || !block_table || !blocks || !totals_out || !table_out || !blocks_out || !evicted || B < 1 ||
      max_blocks < 1 || budget < 0 || keep_first < 0 || keep_last < 0)
    return SV_ERR_ARG;
  if (max_blocks > SV_MAX_BLOCKS || B > MAX_ITEMS / ET) return SV_ERR_UNSUPPORTED;
  const size_t n = (size_t)B * max_blocks * 4, nb = (size_t)B * 4;
  const Output out[] = {{{totals_out, n}, totals}, {{table_out, n}, block_table}, {{blocks_out, nb}, blocks},
                        {{evicted, nb}, nullptr}};
  const Array in[] = {{totals, n}, {block_table, n}, {blocks, nb}};
  if (outputs_overlap(out, in)) return SV_ERR_ARG;
  if (max_blocks > HELD_BLOCKS && table_out == block_table) return SV_ERR_UNSUPPORTED;
  const EvictArgs a{totals, block_table, blocks, totals_out, table_out, blocks_out, evicted, max_blocks, budget,
                    keep_first, keep_last};
  (void)hipGetLastError();
  const dim3 g(B);
  if (max_blocks <= 256) hipLaunchKernelGGL((cache_evict_kernel<256, 1>), g, dim3(256), 0, stream, a);
  else if (max_blocks <= 1024) hipLaunchKernelGGL((cache_evict_kernel<256, 4>), g, dim3(256), 0, stream, a);
  else if (max_blocks <= 4096) hipLaunchKernelGGL((cache_evict_kernel<1024, 4>), g, dim3(1024), 0, stream, a);
  else if (max_blocks <= 8192) hipLaunchKernelGGL((cache_evict_kernel<1024, 8>), g, dim3(1024), 0, stream, a);
  else if (max_blocks <= 12288) hipLaunchKernelGGL((cache_evict_kernel<1024, 12>), g, dim3(1024), 0, stream, a);
  else if (max_blocks <= HELD_BLOCKS) hipLaunchKernelGGL((cache_evict_kernel<1024, 16>), g, dim3(1024), 0, stream, a);
  else hipLaunchKernelGGL(cache_evict_long_kernel, g, dim3(ET), 0, stream, a);
  return hipGetLastError() == hipSuccess ? SV_OK : SV_ERR_HIP;
}
