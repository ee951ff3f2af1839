// evict.cuh -- which cached tokens stay when a sequence's caches are trimmed.
//
// Of a sequence of n tokens the first `sink` and the last `recent` stay, and of those
// between them the keep - sink - recent with the most accumulated attention mass (ties
// to the lower slot). The order is that of the mass's bits made monotone; -0 counts as
// +0 and a NaN ranks below every number. A radix select over 11 + 11 + 10 bits finds the
// border key and how many of its ties stay, then one ordered sweep writes the slots.
//
// The mass is 4 B a slot, read once; what a call waits for is the chain of three
// histograms and a sweep. A cluster of up to eight CTAs takes a sequence, each a run of
// its slots with the keys held in shared memory; after each histogram every CTA adds up
// the cluster's bins for itself (a thread owns four bins: one 16-byte load per CTA), so a
// pass costs one cluster barrier. Histograms of the three passes lie apart, so no barrier
// protects their reuse.
#pragma once

#include "ptx.cuh"

namespace dsa {

constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kEvictBins = 2048;
constexpr int kEvictMaxKeys = 45056;  // keys a CTA holds in shared memory (176 KB)

struct EvictShared {
  int hist[3][kEvictBins];
  int warp_sum[kEvictWarps];
  int warp_above[kEvictWarps], warp_equal[kEvictWarps];
  int counts[2];                // this CTA's slots above and at the border
  int found[2];
};

struct EvictParams {
  const float* mass;         // [batch][ld]
  const int32_t* seqlens;    // [batch] or nullptr
  int32_t* kept;             // [batch][keep]
  int32_t* new_lens;         // [batch]
  int64_t ld;
  int32_t max_ctx, keep, sink, recent;
  int32_t splits;            // CTAs of a sequence's cluster
  int32_t held;              // keys of shared memory per CTA (0: the mass is read each time)
};

__device__ __forceinline__ uint32_t evict_key(float m) {
  if (m != m) return 0u;
  const uint32_t u = __float_as_uint(m + 0.0f);  // -0 + 0 = +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int4 ld_cluster_v4(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ int2 ld_cluster_v2(uint32_t addr) {
  int2 v;
  asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "r"(addr)
               : "memory");
  return v;
}

__global__ void __launch_bounds__(kEvictThreads, 2)
    evict_select_kernel(const EvictParams p) {
  extern __shared__ uint32_t keys[];
  __shared__ __align__(16) EvictShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / p.splits, rank = blockIdx.x % p.splits;
  int n = p.seqlens ? __ldg(p.seqlens + b) : p.max_ctx;
  int32_t* kept = p.kept + (int64_t)b * p.keep;
  const int gtid = rank * kEvictThreads + tid, gthreads = p.splits * kEvictThreads;
  if (n < 0 || n > p.max_ctx) {
    if (gtid == 0) report_error(kErrBounds);
    n = 0;
  }
  if (gtid == 0) p.new_lens[b] = min(n, p.keep);
  if (n <= p.keep) {
    for (int i = gtid; i < p.keep; i += gthreads) kept[i] = i < n ? i : -1;
    return;
  }
  const int want = p.keep - p.sink - p.recent;  // of [sink, n - recent), which holds more
  for (int i = gtid; i < p.sink; i += gthreads) kept[i] = i;
  for (int i = gtid; i < p.recent; i += gthreads) kept[p.sink + want + i] = n - p.recent + i;
  if (want == 0) return;
  // this CTA's run of the middle, a multiple of 32 slots but for the end
  const int middle = n - p.recent - p.sink;
  const int run = ((middle + p.splits - 1) / p.splits + 31) & ~31;
  const int begin = min(p.sink + rank * run, n - p.recent), end = min(begin + run, n - p.recent);
  const float* mass = p.mass + (int64_t)b * p.ld;
  const bool hold = p.held >= run;
  auto key_at = [&](int i) { return hold ? keys[i - begin] : evict_key(__ldg(mass + i)); };
  for (int i = tid; i < 3 * kEvictBins; i += kEvictThreads) (&sh.hist[0][0])[i] = 0;
  __syncthreads();
  // the border key: the want-th largest
  uint32_t border = 0;
  int left = want;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, width = pass == 2 ? 10 : 11;
    for (int i = begin + tid; i < end; i += kEvictThreads) {
      uint32_t key;
      if (pass == 0) {
        key = evict_key(__ldg(mass + i));
        if (hold) keys[i - begin] = key;
      } else {
        key = key_at(i);
      }
      if (pass == 0 || (key >> (shift + width)) == border)
        atomicAdd(&sh.hist[pass][(key >> shift) & ((1 << width) - 1)], 1);
    }
    cluster_sync_all();
    // thread t owns bins 4 t' .. 4 t' + 3 from the top down
    const int first = kEvictBins - 4 - tid * 4;
    int4 c = *reinterpret_cast<const int4*>(&sh.hist[pass][first]);
    const uint32_t mine = smem_u32(&sh.hist[pass][first]);
    for (int r = 1; r < p.splits; ++r) {
      const int peer = rank + r < p.splits ? rank + r : rank + r - p.splits;
      const int4 v = ld_cluster_v4(mapa_shared(mine, peer));
      c.x += v.x, c.y += v.y, c.z += v.z, c.w += v.w;
    }
    const int down[4] = {c.w, c.z, c.y, c.x};
    const int sum = c.x + c.y + c.z + c.w;
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) sh.warp_sum[warp] = incl;
    __syncthreads();
    int before = incl - sum;
    for (int w = 0; w < warp; ++w) before += sh.warp_sum[w];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (before < left && before + down[j] >= left) {
        sh.found[0] = first + 3 - j;
        sh.found[1] = left - before;
      }
      before += down[j];
    }
    __syncthreads();
    border = (border << width) | (uint32_t)sh.found[0];
    left = sh.found[1];
  }
  // slots above the border, and the first `left` equal to it, in ascending order: a warp
  // takes a run of the CTA's slots, counts them, and writes them behind those before it
  const int per = ((end - begin + kEvictWarps - 1) / kEvictWarps + 31) & ~31;
  const int w0 = min(begin + warp * per, end), w1 = min(w0 + per, end);
  int above = 0, equal = 0;
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const bool in = i0 + lane < w1;
    const uint32_t key = in ? key_at(i0 + lane) : 0u;
    above += __popc(__ballot_sync(0xffffffffu, in && key > border));
    equal += __popc(__ballot_sync(0xffffffffu, in && key == border));
  }
  if (lane == 0) {
    sh.warp_above[warp] = above;
    sh.warp_equal[warp] = equal;
  }
  __syncthreads();
  int g = 0, e = 0, all_g = 0, all_e = 0;
  for (int w = 0; w < kEvictWarps; ++w) {
    if (w < warp) g += sh.warp_above[w], e += sh.warp_equal[w];
    all_g += sh.warp_above[w], all_e += sh.warp_equal[w];
  }
  if (tid == 0) sh.counts[0] = all_g, sh.counts[1] = all_e;
  cluster_sync_all();
  for (int r = 0; r < rank; ++r) {
    const int2 v = ld_cluster_v2(mapa_shared(smem_u32(&sh.counts[0]), r));
    g += v.x, e += v.y;
  }
  const uint32_t lower = (1u << lane) - 1;
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    const bool in = i < w1;
    const uint32_t key = in ? key_at(i) : 0u;
    const bool gt = in && key > border, eq = in && key == border;
    const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
    const int rg = g + __popc(bg & lower), re = e + __popc(be & lower);
    if (gt || (eq && re < left)) kept[p.sink + rg + min(re, left)] = i;
    g += __popc(bg);
    e += __popc(be);
  }
  cluster_sync_all();  // no CTA leaves while another still reads its shared memory
}

}  // namespace dsa
