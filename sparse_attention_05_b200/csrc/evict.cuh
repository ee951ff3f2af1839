// evict.cuh -- which cached tokens stay when a sequence's caches are trimmed.
//
// Of a sequence of n tokens the first `sink` and the last `recent` stay, and of those
// between them the keep - sink - recent with the most accumulated attention mass (ties
// to the lower slot). The order is that of the mass's bits made monotone; -0 counts as
// +0 and a NaN ranks below every number. A radix select over 11 + 11 + 10 bits finds the
// border key and how many of its ties stay, then one ordered sweep writes the slots.
#pragma once

#include "ptx.cuh"

namespace dsa {

constexpr int kEvictThreads = 512;
constexpr int kEvictBins = 2048;

struct EvictParams {
  const float* mass;         // [batch][ld]
  const int32_t* seqlens;    // [batch] or nullptr
  int32_t* kept;             // [batch][keep]
  int32_t* new_lens;         // [batch]
  int64_t ld;
  int32_t max_ctx, keep, sink, recent;
};

__device__ __forceinline__ uint32_t evict_key(float m) {
  if (m != m) return 0u;
  const uint32_t u = __float_as_uint(m + 0.0f);  // -0 + 0 = +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kEvictThreads) evict_select_kernel(const EvictParams p) {
  __shared__ int hist[kEvictBins];
  __shared__ int warp_sum[2][kEvictThreads / 32];
  __shared__ int found[2];
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int n = p.seqlens ? __ldg(p.seqlens + b) : p.max_ctx;
  int32_t* kept = p.kept + (int64_t)b * p.keep;
  if (n < 0 || n > p.max_ctx) {
    if (tid == 0) report_error(kErrBounds);
    n = 0;
  }
  if (tid == 0) p.new_lens[b] = min(n, p.keep);
  if (n <= p.keep) {
    for (int i = tid; i < p.keep; i += kEvictThreads) kept[i] = i < n ? i : -1;
    return;
  }
  const float* mass = p.mass + (int64_t)b * p.ld;
  const int begin = p.sink, end = n - p.recent;
  int want = p.keep - p.sink - p.recent;  // of [begin, end), which holds more than that
  for (int i = tid; i < p.sink; i += kEvictThreads) kept[i] = i;
  for (int i = tid; i < p.recent; i += kEvictThreads) kept[p.sink + want + i] = end + i;
  if (want == 0) return;
  // the border key: the want-th largest
  uint32_t border = 0;
  const int shifts[3] = {21, 10, 0}, widths[3] = {11, 11, 10};
  int left = want;
  for (int pass = 0; pass < 3; ++pass) {
    for (int i = tid; i < kEvictBins; i += kEvictThreads) hist[i] = 0;
    __syncthreads();
    const int shift = shifts[pass], width = widths[pass];
    for (int i = begin + tid; i < end; i += kEvictThreads) {
      const uint32_t key = evict_key(__ldg(mass + i));
      if (pass == 0 || (key >> (shift + width)) == border)
        atomicAdd(&hist[(key >> shift) & ((1 << width) - 1)], 1);
    }
    __syncthreads();
    // thread t sums the four bins from the top down; the bin where the count passes `left`
    int c[4], sum = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      c[j] = hist[kEvictBins - 1 - (tid * 4 + j)];
      sum += c[j];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum[0][warp] = incl;
    __syncthreads();
    int before = incl - sum;
    for (int w = 0; w < warp; ++w) before += warp_sum[0][w];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (before < left && before + c[j] >= left) {
        found[0] = kEvictBins - 1 - (tid * 4 + j);
        found[1] = left - before;
      }
      before += c[j];
    }
    __syncthreads();
    border = (border << width) | (uint32_t)found[0];
    left = found[1];
    __syncthreads();
  }
  // slots above the border, and the first `left` equal to it, in ascending order
  int above = 0, equal = 0;  // counts of the blocks swept so far
  for (int i0 = begin; i0 < end; i0 += kEvictThreads) {
    const int i = i0 + tid;
    const uint32_t key = i < end ? evict_key(__ldg(mass + i)) : 0u;
    const bool gt = i < end && key > border, eq = i < end && key == border;
    const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) {
      warp_sum[0][warp] = __popc(bg);
      warp_sum[1][warp] = __popc(be);
    }
    __syncthreads();
    int g0 = above, e0 = equal;
    for (int w = 0; w < kEvictThreads / 32; ++w) {
      if (w < warp) {
        g0 += warp_sum[0][w];
        e0 += warp_sum[1][w];
      }
      above += warp_sum[0][w];
      equal += warp_sum[1][w];
    }
    const uint32_t below = (1u << lane) - 1;
    const int rg = g0 + __popc(bg & below), re = e0 + __popc(be & below);
    if (gt || (eq && re < left)) kept[p.sink + rg + min(re, left)] = i;
    __syncthreads();
  }
}

}  // namespace dsa
